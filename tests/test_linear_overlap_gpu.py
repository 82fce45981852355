"""Calls that overlap in time: the backward on two streams at once, with
activations, K slices and partial sums in its workspaces, from two host threads,
and in two graphs replayed in turn; the norm likewise."""
import threading

import pytest
import torch

import beta_epilogue_amd as ge
from test_linear_gpu import _draw, _say

pytestmark = pytest.mark.gpu


def _grad_case(act, tile, splits):
    M, N, K = 400, 264, 520
    g = torch.Generator().manual_seed(tile + splits)
    t = lambda r, c: _draw(g, r, c, torch.bfloat16).cuda()  # noqa: E731
    op = ge.FusedLinearGrad(M, N, K, act=act, da="bf16", db="f32", dbias="f32", tile=tile, splits=splits)
    ins = dict(dD=t(M, N), A=t(M, K), B=t(N, K), dB_in=torch.randn(N, K, generator=g).cuda())
    if act != "none":
        ins["Z"] = t(M, N)

    def new():
        o = dict(dA=torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), dB=torch.empty(N, K, device="cuda"),
                 dbias=torch.empty(N, device="cuda"))
        return o | (dict(dZ=torch.empty(M, N, dtype=torch.bfloat16, device="cuda")) if act != "none" else {})

    return op, ins, new


def _norm_case():
    g = torch.Generator().manual_seed(2)
    x, r = (_draw(g, 600, 3000, torch.bfloat16).cuda() for _ in range(2))
    w = torch.ones(3000, dtype=torch.bfloat16, device="cuda")
    op = ge.RmsNorm(600, 3000, y="i8", residual=True)

    def new():
        return dict(Y=torch.empty(600, 3000, dtype=torch.int8, device="cuda"), H=torch.empty_like(x),
                    scale=torch.empty(600, device="cuda"))

    return op, dict(x=x, weight=w, residual=r), new


CASES = {"gelu, 3 slices": lambda: _grad_case("gelu", 64, 3), "no activation": lambda: _grad_case("none", 128, 2),
         "relu, whole": lambda: _grad_case("relu", 128, 1), "norm": _norm_case}


@pytest.mark.parametrize("name", CASES)
def test_streams_threads_graphs(name):
    op, ins, new = CASES[name]()
    _say("case", name, getattr(op, "workspace_bytes", 0))
    want = new()
    op(**ins, **want)
    outs = [new() for _ in range(8)]
    torch.cuda.synchronize()
    same = lambda o: all(torch.equal(o[k], want[k]) for k in want)  # noqa: E731

    def wipe():
        for o in outs:
            for v in o.values():
                v.zero_()
        torch.cuda.synchronize()

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        op(**ins, **o, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(map(same, outs))
    wipe()

    def work(k):
        for o in outs[k::2]:
            op(**ins, **o, stream=streams[k])

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(map(same, outs))
    wipe()
    graphs = []
    for o in outs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            op(**ins, **o)
        graphs.append((gr, o))
    for _ in range(3):
        wipe()
        for gr, o in graphs:
            gr.replay()
        eager = new()
        op(**ins, **eager)
        torch.cuda.synchronize()
        assert same(eager) and all(same(o) for _, o in graphs)
