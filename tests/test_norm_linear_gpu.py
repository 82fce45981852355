"""Norm and projection in a row: what a call may alias, streams and graphs, and
calls that are refused before anything is written."""
import pytest
import torch

import beta_epilogue_amd as ge
import linear_ref as ref
from test_linear_gpu import _draw
from test_norm_gpu import _say

pytestmark = pytest.mark.gpu


def _inputs(M, N, K, q="e4m3", seed=3):
    g = torch.Generator().manual_seed(seed)
    bf = lambda r, c: _draw(g, r, c, torch.bfloat16).cuda()  # noqa: E731
    return dict(x=bf(M, K), residual=bf(M, K), weight=(1 + 0.3 * torch.randn(K, generator=g)).bfloat16().cuda(),
                B=_draw(g, N, K, ref.TORCH[q]).cuda(), scale_b=(torch.rand(N, generator=g) / 200).cuda(),
                bias=torch.randn(N, generator=g).cuda())


def test_refused_before_the_norm_writes():
    """A call that the projection would refuse leaves the residual stream as it
    was, although the norm alone would have been fine."""
    M, N, K = 20, 64, 64
    op = ge.FusedNormLinear(M, N, K, bias="f32", residual=True, add=True)
    t = _inputs(M, N, K)
    D = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    x0, r0, d0 = t["x"].clone(), t["residual"].clone(), D.clone()
    flat = torch.zeros(M * N + 4, dtype=torch.bfloat16, device="cuda")
    good = t | dict(D=D, H=t["x"], add=t["residual"])
    _say("case", M, N, K)
    for bad in (dict(D=D[:, :56]), dict(D=D.half()), dict(D=flat[4:].view(M, N)), dict(D=None), dict(bias=None),
                dict(bias=t["bias"].half()), dict(bias=torch.zeros(N + 1, device="cuda")[1:]), dict(add=None),
                dict(add=D.float()), dict(B=t["B"][:, :48]), dict(B=None), dict(scale_b=None),
                dict(scale_b=t["scale_b"].cpu()), dict(D=t["B"].view(torch.bfloat16))):
        with pytest.raises((ValueError, ge.GemmEpiError)):
            op(**(good | bad))
    torch.cuda.synchronize()
    assert torch.equal(t["x"], x0) and torch.equal(t["residual"], r0) and torch.equal(D, d0)
    with pytest.raises((ValueError, ge.GemmEpiError)):  # add without a plan for it
        ge.FusedNormLinear(M, N, K, residual=True)(t["x"], t["weight"], t["B"], t["scale_b"], D=D, H=t["x"],
                                                   residual=t["residual"], add=t["residual"])
    torch.cuda.synchronize()
    assert torch.equal(t["x"], x0) and torch.equal(D, d0)


@pytest.mark.parametrize("M", [3, 150])
def test_residual_stream_in_place(M):
    """h = x + residual written over x, then added to the projection and the
    sum written over it: equal to separate buffers bit for bit."""
    N = K = 256
    op = ge.FusedNormLinear(M, N, K, act="gelu", bias="f32", residual=True, add=True)
    t = _inputs(M, N, K, seed=M)
    D, H = (torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _say("case", M)
    op(**t, D=D, H=H, add=H)
    x = t.pop("x").clone()
    op(x, **t, D=x, H=x, add=x)
    torch.cuda.synchronize()
    assert torch.equal(x, D)


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("q", ["e4m3", "i8"])
def test_streams_and_graphs(M, q):
    """Calls of one plan on two streams at once and in two graphs, replayed in
    turn with eager calls between, equal the eager result bit for bit."""
    N, K = 264, 2064
    op = ge.FusedNormLinear(M, N, K, q=q, bias="f32", residual=True)
    t = _inputs(M, N, K, q)
    new = lambda: torch.empty(M, N, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    want = op(**t, D=new())
    outs = [new() for _ in range(8)]
    torch.cuda.synchronize()
    _say("case", M, q)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        op(**t, D=o, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs = []
    for o in outs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            op(**t, D=o)
        graphs.append((gr, o))
    for _ in range(3):
        for gr, o in graphs:
            o.zero_()
            torch.cuda.synchronize()
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want)
        assert torch.equal(op(**t, D=new()), want)
