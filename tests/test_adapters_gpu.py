"""The linear layer with low-rank adapters on the GPU against a plain 64-bit
form.  Bounds (linear_ref's, and): the inner products u are sums of K terms in
fp32, rounded once to 16 bits; their error times |up| and rank further fp32
terms come on top of z.  Each case prints its name before the GPU step."""
import pytest
import torch

import beta_epilogue_amd as ge
import linear_ref as ref
from test_linear_gpu import ACTS, NAN, Out, _draw, _say, _strided

pytestmark = pytest.mark.gpu

TORCH = ref.TORCH


def plain(A, B, ids, down, up, scale, act, bias, residual, dtype):
    """(D, Z, bound of D, bound of Z)."""
    a, b, K, rank = ref.f64(A), ref.f64(B), A.shape[1], down.shape[1]
    z, S = a @ b.T, a.abs() @ b.abs().T
    extra = torch.zeros_like(z)
    for g in range(down.shape[0]):
        at = (ids == g).nonzero()[:, 0]
        if at.numel() == 0:
            continue
        s, d, u = float(scale[g]), ref.f64(down[g]), ref.f64(up[g])
        inner, size = s * (a[at] @ d.T), abs(s) * (a[at].abs() @ d.abs().T)
        z[at] += inner @ u.T
        e = (K + 2) * ref.U * size
        e = e + ref.half_step(inner.abs() + e, dtype)
        extra[at] += e @ u.abs().T
        S[at] += (inner.abs() + e) @ u.abs().T
    if bias is not None:
        z, S = z + ref.f64(bias), S + ref.f64(bias).abs()
    d = ref.act(z, act)
    if residual is not None:
        d = d + ref.f64(residual)
    ez = (K + rank + 4) * ref.U * S + extra
    r = ref.f64(residual).abs() if residual is not None else 0.0
    ed = 1.13 * ez + z.abs() * 2.0 ** -21 + ref.U * (z.abs() + r)
    return d, z, ed + ref.half_step(d.abs() + ed, dtype), ez + ref.half_step(z.abs() + ez, dtype)


def some_ids(g, M, G, kind):
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if kind == "one":
        return torch.full((M,), G - 1, dtype=torch.int32)
    ids = torch.randint(0, G, (M,), generator=g)
    if kind == "runs":  # prompts one after the other
        ids = ids[torch.randint(0, min(M, 5), (M,), generator=g).sort().values]
    wrong = torch.tensor([-1, G, (1 << 31) - 1, -(1 << 31)])
    return torch.where(torch.rand(M, generator=g) < 0.15, wrong[torch.randint(0, 4, (M,), generator=g)], ids).to(torch.int32)


def run(M, N, K, rank, G, ab="bf16", act="none", bias=None, res=False, z=False, pad=0, splits=0, variant=-1, seed=1,
        kind="mixed", inplace=False):
    g = torch.Generator().manual_seed(seed)
    T = TORCH[ab]
    A, B = _draw(g, M, K, T), _draw(g, N, K, T, K ** -0.5)
    ids = some_ids(g, M, G, kind)
    down = _draw(g, G * rank, K, T, K ** -0.5).view(G, rank, K)
    up = _draw(g, G * N, rank, T, rank ** -0.5).view(G, N, rank)
    scale = torch.rand(G, generator=g) * 2 - 0.5
    for e in range(G):  # adapters that no row has are not read into any result
        if not (ids == e).any():
            down[e], up[e], scale[e] = NAN, NAN, NAN
    b = _draw(g, 1, N, TORCH[bias])[0] if bias else None
    R = _draw(g, M, N, T) if res else None
    ld = lambda c, on=True: c + pad if pad and on else 0  # noqa: E731
    op = ge.AdapterLinear(M, N, K, rank, G, ab=ab, act=act, bias=bias, residual=res, z=z, lda=ld(K), ldb=ld(K), ldd=ld(N),
                          ldr=ld(N, res), ldz=ld(N, z), splits=splits, variant=variant)
    D, Z = Out(M, N, T, N + pad), (Out(M, N, T, N + pad) if z else None)
    Rd = _strided(R, pad) if res else None
    if inplace:
        D.t.copy_(Rd)
        Rd = D.t
    plan = op.plan
    _say("case", M, N, K, "rank", rank, "of", G, ab, act, kind, "pad", pad, plan["name"], "splits", plan["splits"])
    ws = torch.full((plan["workspace_bytes"],), 0xff, dtype=torch.uint8, device="cuda")  # NaN wherever it is not written
    there = torch.cat([torch.zeros(1, dtype=torch.int32), ids]).cuda()[1:]  # (not 16-byte aligned)
    op(_strided(A, pad), _strided(B, pad), there, down.cuda(), up.cuda(), scale.cuda(), D=D.t,
       bias=b.cuda() if bias else None, residual=Rd, Z=Z.t if z else None, workspace=ws)
    torch.cuda.synchronize()
    assert D.intact() and (Z is None or Z.intact()), "a guard was overwritten"
    d, zr, bd, bz = plain(A, B, ids, down, up, scale, act, b, R, T)
    ref.check("D", D.t, d, bd)
    if z:
        ref.check("Z", Z.t, zr, bz)
    op.close()
    return plan


@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("ab", ["bf16", "f16"])
def test_few_rows(M, ab):
    names = ge.linear_variant_names()
    for rank, G in ((8, 1), (16, 70), (40, 3), (64, 5), (128, 20)):
        plan = run(M, 264, 656, rank, G, ab, act="silu", bias="f32", res=True, z=True, seed=M + rank,
                   variant=names.index("linear_rows"))
        assert plan["name"] == "linear_rows"


@pytest.mark.parametrize("N,K", [(8, 8), (8, 4104), (24, 1040), (4104, 32), (1032, 8200)])
@pytest.mark.parametrize("M", [1, 3, 40])
def test_few_rows_sizes(M, N, K):
    run(M, N, K, 16, 4)
    run(M, N, K, 72, 2, "f16", res=True)


TILES = [n for n in ge.linear_variant_names() if n.split("_")[1] in ("f16", "bf16")]


@pytest.mark.parametrize("name", TILES)
@pytest.mark.parametrize("kind", ["mixed", "runs", "one", "none"])
def test_every_tile(name, kind):
    ab, v = name.split("_")[1], ge.linear_variant_names().index(name)
    run(333, 328, 272, 16, 5, ab, act="gelu", bias="f32", res=True, z=True, variant=v, kind=kind)
    run(333, 328, 136, 72, 9, ab, variant=v, kind=kind, pad=16)
    run(270, 264, 1168, 24, 40, ab, act="silu", bias=ab, res=True, variant=v, kind=kind, splits=3)


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 56, 64, 96, 128])
@pytest.mark.parametrize("M", [65, 130, 1100])
def test_ranks(M, rank):
    run(M, 136, 328, rank, 6, kind="runs", bias="bf16")
    run(M, 136, 328, rank, 200, kind="mixed")


@pytest.mark.parametrize("rank,G", [(16, 2), (24, 1), (32, 2), (64, 2), (128, 2)])
@pytest.mark.parametrize("kind", ["mixed", "runs", "none"])
def test_up_to_two_adapters(rank, G, kind):
    """Their rows are not sorted."""
    run(701, 264, 520, rank, G, kind=kind, seed=rank)
    run(1040, 72, 2056, rank, G, "f16", kind=kind, seed=rank + 1)


@pytest.mark.parametrize("M,rank,G", [(1500, 8, 1024), (300, 16, 1000), (70, 128, 600), (2200, 64, 257), (8200, 8, 300)])
@pytest.mark.parametrize("name", TILES)
def test_many_adapters(M, rank, G, name):
    run(M, 72, 72, rank, G, name.split("_")[1], kind="mixed", seed=G, variant=ge.linear_variant_names().index(name))


@pytest.mark.parametrize("M,N,K", [(65, 8, 8), (65, 264, 16), (257, 520, 1032), (1001, 256, 40), (300, 2552, 24),
                                   (65, 16, 8200), (2100, 64, 4104)])
@pytest.mark.parametrize("kind", ["mixed", "runs"])
def test_sizes(M, N, K, kind):
    run(M, N, K, 16, 7, act="relu", bias="f32", res=True, kind=kind)
    run(M, N, K, 64, 3, "f16", kind=kind)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [7, 100])
def test_activations(act, M):
    run(M, 136, 264, 16, 4, "f16", act=act, bias="f32", res=True, z=True)


@pytest.mark.parametrize("M", [7, 200])
def test_strides_and_in_place(M):
    run(M, 264, 512, 16, 4, act="gelu", bias="f32", res=True, inplace=True)
    run(M, 264, 512, 16, 4, res=True, inplace=True, pad=8, splits=2)
    run(M, 264, 512, 32, 4, res=True, z=True, pad=32)


def test_the_plan_counts_the_adapters():
    """The K tiles that a tile's adapters add fall on its first K slice, so many adapters
    want fewer slices and smaller tiles than the projection alone, or few-row kernels."""
    for M, N, K, rank, G in ((512, 1024, 8192, 8, 300), (64, 512, 4096, 32, 48)):
        alone, many = ge.FusedLinear(M, N, K).plan, ge.AdapterLinear(M, N, K, rank, G).plan
        assert many["splits"] < alone["splits"] and many["tile_m"] <= alone["tile_m"], (alone, many)


def test_without_adapters_it_is_the_linear_layer():
    g = torch.Generator().manual_seed(2)
    for M in (16, 300):
        A, B = _draw(g, M, 512, torch.bfloat16).cuda(), _draw(g, 264, 512, torch.bfloat16).cuda()
        D, want = (torch.zeros(M, 264, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
        down = torch.full((2, 16, 512), NAN, dtype=torch.bfloat16, device="cuda")
        up = torch.full((2, 264, 16), NAN, dtype=torch.bfloat16, device="cuda")
        _say("case without", M)
        ge.AdapterLinear(M, 264, 512, 16, 2)(A, B, ids, down, up, torch.full((2,), NAN, device="cuda"), D=D)
        ge.FusedLinear(M, 264, 512)(A, B, D=want)
        assert torch.equal(D, want)


def test_special_values():
    """A NaN or an infinity of one row, or of one adapter, stays with its rows."""
    for M in (12, 200):
        A = torch.ones(M, 64, dtype=torch.bfloat16)
        B, down, up = (torch.ones(*s, dtype=torch.bfloat16) for s in ((64, 64), (3, 16, 64), (3, 64, 16)))
        A[1, 3] = NAN
        down[1, 2, 5], up[2, 7, 3] = NAN, float("inf")
        ids = torch.zeros(M, dtype=torch.int32)
        ids[4], ids[5], ids[6] = 1, 2, -1
        D = torch.zeros(M, 64, dtype=torch.bfloat16, device="cuda")
        _say("case special", M)
        ge.AdapterLinear(M, 64, 64, 16, 3)(A.cuda(), B.cuda(), ids.cuda(), down.cuda(), up.cuda(),
                                           torch.full((3,), 0.5, device="cuda"), D=D)
        D = D.cpu().float()
        assert torch.isnan(D[1]).all() and torch.isnan(D[4]).all() and (D[6] == 64).all()
        assert D[5, 7] == float("inf") and (D[5, :7] == 64 + 512).all() and (D[5, 8:] == 64 + 512).all()
        rest = [i for i in range(M) if i not in (1, 4, 5, 6)]
        assert (D[rest] == 64 + 512).all()


@pytest.mark.parametrize("M", [7, 150])
def test_inner_products_of_fp16(M):
    """Below fp16's normal range they are off by half of a subnormal step (2^-25), beyond its
    largest value infinite, in their own rows only."""
    N, K, rank, G, T = 72, 64, 16, 3, torch.float16
    g = torch.Generator().manual_seed(M)
    A, B = _draw(g, M, K, T), torch.zeros(N, K, dtype=T)
    down, up = _draw(g, G * rank, K, T, K ** -0.5).view(G, rank, K), _draw(g, G * N, rank, T, 100.0).view(G, N, rank)
    ids = (torch.arange(M) % G).to(torch.int32)
    for scale in (1e-4, 1e-6, 2.0 ** -24):
        D = torch.empty(M, N, dtype=T, device="cuda")
        s = torch.full((G,), scale)
        _say("case small inner products", M, scale)
        op = ge.AdapterLinear(M, N, K, rank, G, ab="f16")
        op(A.cuda(), B.cuda(), ids.cuda(), down.cuda(), up.cuda(), s.cuda(), D=D)
        want, _, bound, _ = plain(A, B, ids, down, up, s, "none", None, None, T)
        ref.check("D", D, want, bound)
    s = torch.tensor([1.0, 1e6, 1.0])
    up = (up / 1e4).to(T)
    op(A.cuda(), B.cuda(), ids.cuda(), down.cuda(), up.cuda(), s.cuda(), D=D)
    want, _, bound, _ = plain(A, B, ids, down, up, s, "none", None, None, T)
    near = ids != 1
    ref.check("D", D[near.cuda()], want[near], bound[near])
    assert not torch.isfinite(D[1].float()).all()


def test_behind_the_norm():
    """Norm, projection with adapters, and an expert layer's sort of its result,
    as a program would run them, on two streams and in two graphs."""
    g = torch.Generator().manual_seed(9)
    M, N, K, rank, G = 130, 136, 264, 16, 5
    x, w = _draw(g, M, K, torch.bfloat16).cuda(), torch.ones(K, dtype=torch.bfloat16, device="cuda")
    B = _draw(g, N, K, torch.bfloat16, K ** -0.5).cuda()
    down, up = _draw(g, G * rank, K, torch.bfloat16, 0.1).view(G, rank, K).cuda(), _draw(g, G * N, rank, torch.bfloat16).view(
        G, N, rank).cuda()
    scale, ids = torch.rand(G, generator=g).cuda(), some_ids(g, M, G, "runs").cuda()
    experts = torch.randint(0, 4, (M, 2), generator=g).cuda()
    norm, linear = ge.RmsNorm(M, K), ge.AdapterLinear(M, N, K, rank, G, act="silu", splits=2)
    sort = ge.ExpertSort(M, 2, 4, cols=N)
    assert linear.workspace_bytes > 0

    def new():
        e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(Y=e(M, K), D=e(M, N), S=e(2 * M, N), off=i(5), rows=i(M, 2))

    def call(o, stream=None):
        norm(x, w, Y=o["Y"], stream=stream)
        linear(o["Y"], B, ids, down, up, scale, D=o["D"], stream=stream)
        sort(experts, o["D"], offsets=o["off"], rows=o["rows"], Y=o["S"], stream=stream)

    _say("case behind the norm")
    want = new()
    call(want)
    torch.cuda.synchronize()
    d, _, bd, _ = plain(want["Y"].cpu(), B.cpu(), ids.cpu(), down.cpu(), up.cpu(), scale.cpu(), "silu", None, None,
                        torch.bfloat16)
    ref.check("D", want["D"], d, bd)
    same = lambda o: all(torch.equal(o[n], want[n]) for n in want)  # noqa: E731
    outs = [new() for _ in range(6)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        call(o, streams[i % 2])
    torch.cuda.synchronize()
    assert all(map(same, outs))
    graphs = []
    for o in outs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(o)
        graphs.append(gr)
    for _ in range(3):
        for o in outs[:2]:
            for t in o.values():
                t.zero_()
        eager = new()
        for gr in graphs:
            gr.replay()
        call(eager)
        torch.cuda.synchronize()
        assert same(eager) and all(map(same, outs[:2]))


@pytest.mark.parametrize("M,G", [(2100, 5), (9000, 70), (2100, 2)])
def test_sorted_rows_on_streams_and_in_graphs(M, G):
    """Many rows, whose inner products take a sort (but for two adapters): two
    streams, and two graphs replayed in turn with eager calls between."""
    g = torch.Generator().manual_seed(M)
    N, K, rank = 72, 136, 16
    b = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    A, B, down, up = b(M, K), b(N, K), b(G, rank, K), b(G, N, rank)
    scale, ids = torch.rand(G, generator=g).cuda(), some_ids(g, M, G, "mixed").cuda()
    op = ge.AdapterLinear(M, N, K, rank, G)
    _say("case sorted rows, streams and graphs", M, G, op.plan["name"])
    new = lambda: torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    call = lambda d, stream=None: op(A, B, ids, down, up, scale, D=d, stream=stream)  # noqa: E731
    want = call(new())
    d, _, bd, _ = plain(A.cpu(), B.cpu(), ids.cpu(), down.cpu(), up.cpu(), scale.cpu(), "none", None, None, torch.bfloat16)
    ref.check("D", want, d, bd)
    outs = [new() for _ in range(6)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        call(o, streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs = []
    for o in outs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(o)
        graphs.append(gr)
    for _ in range(3):
        for o in outs[:2]:
            o.zero_()
        for gr in graphs:
            gr.replay()
        eager = call(new())
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in (eager, *outs[:2]))


def test_refusals():
    M, N, K, rank, G = 16, 64, 128, 16, 2
    b = dict(dtype=torch.bfloat16, device="cuda")
    op = ge.AdapterLinear(M, N, K, rank, G, residual=True)
    D = torch.zeros(M, N, **b)
    good = dict(A=torch.zeros(M, K, **b), B=torch.zeros(N, K, **b), ids=torch.zeros(M, dtype=torch.int32, device="cuda"),
                down=torch.zeros(G, rank, K, **b), up=torch.zeros(G, N, rank, **b), scale=torch.ones(G, device="cuda"), D=D,
                residual=torch.zeros(M, N, **b))
    op(**good)
    for bad in (dict(ids=None), dict(ids=good["ids"].long()), dict(ids=good["ids"][:4]), dict(down=good["up"]), dict(up=None),
                dict(up=good["up"][:1]), dict(scale=good["scale"].half()), dict(scale=None), dict(residual=None), dict(Z=D),
                dict(D=good["A"]), dict(A=good["A"].half()), dict(B=good["B"].cpu()),
                dict(up=good["up"].transpose(1, 2).contiguous().transpose(1, 2)),
                dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, ge.GemmEpiError)):
            op(**(good | bad))


@pytest.mark.parametrize("name", TILES)
@pytest.mark.parametrize("splits", [1, 2])
def test_adapters_that_are_not_finite(name, splits):
    """An infinity or a NaN in some adapters' up reaches their rows only, in every
    kernel: the others' rows are what they are without it, bit for bit."""
    ab, v = name.split("_")[1], ge.linear_variant_names().index(name)
    M, N, K, rank, G = 300, 264, 136, 24, 6
    g = torch.Generator().manual_seed(3)
    T = TORCH[ab]
    A, B = _draw(g, M, K, T).cuda(), _draw(g, N, K, T, K ** -0.5).cuda()
    ids = some_ids(g, M, G, "mixed")
    down, up = _draw(g, G * rank, K, T, K ** -0.5).view(G, rank, K).cuda(), _draw(g, G * N, rank, T).view(G, N, rank).cuda()
    bad = up.clone()
    bad[2, 7, 3], bad[2, N - 1, rank - 1], bad[5, 0, 0] = float("inf"), -float("inf"), NAN
    op = ge.AdapterLinear(M, N, K, rank, G, ab=ab, variant=v, splits=splits)
    D, want = torch.zeros(M, N, dtype=T, device="cuda"), torch.zeros(M, N, dtype=T, device="cuda")
    scale = torch.ones(G, device="cuda")
    _say("case not finite", name, splits)
    op(A, B, ids.cuda(), down, up, scale, D=want)
    op(A, B, ids.cuda(), down, bad, scale, D=D)
    theirs = (ids == 2) | (ids == 5)
    assert torch.equal(D[~theirs], want[~theirs])
    assert torch.isnan(D[ids == 5][:, 0]).all() and torch.isfinite(D[ids == 5][:, 1:]).all()
    assert not torch.isfinite(D[ids == 2][:, 7]).any() and not torch.isfinite(D[ids == 2][:, N - 1]).any()
    assert torch.isfinite(D[ids == 2][:, 8:N - 1]).all()
    # (their finite columns: the same sums in another order)
    d, _, bd, _ = plain(A.cpu(), B.cpu(), ids, down.cpu(), up.cpu(), torch.ones(G), "none", None, None, T)
    rest = torch.ones(N, dtype=torch.bool)
    rest[[0, 7, N - 1]] = False
    ref.check("D", D[theirs][:, rest], d[theirs][:, rest], bd[theirs][:, rest])
