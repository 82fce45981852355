"""Tokens sorted by expert and brought back, on the GPU against plain forms
(tests/experts_ref.py, which derives the bounds).  Each case prints its name
before the GPU step."""
import pytest
import torch

import beta_epilogue_amd as ge
import experts_ref as ref
import linear_ref
from test_linear_gpu import NAN, Out, _draw, _say, _strided

pytestmark = pytest.mark.gpu

TORCH = linear_ref.TORCH


def _ids(g, T, k, E, kind="some"):
    if kind == "one":
        return torch.full((T, k), E - 1, dtype=torch.int64)
    if kind == "none":
        return torch.full((T, k), -1, dtype=torch.int64)
    ids = torch.randint(0, E, (T, k), generator=g)  # (the same expert twice in a token, too)
    if kind == "some":
        wrong = torch.tensor([-1, E, -(1 << 40), (1 << 32), (1 << 32) + E - 1, -(1 << 63), (1 << 63) - 1])
        bad = torch.rand(T, k, generator=g) < 0.2
        ids = torch.where(bad, wrong[torch.randint(0, len(wrong), (T, k), generator=g)], ids)
    return ids


def run_sort(T, k, E, cols, x="bf16", ids="i64", kind="some", scale=False, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    choice = _ids(g, T, k, E, kind)
    if ids == "i32":
        choice = choice.clamp(-(1 << 31), (1 << 31) - 1).to(torch.int32)
    offsets, rows = ref.sort(choice, E)
    n = int(offsets[-1])
    op = ge.ExpertSort(T, k, E, cols=cols, x=x, ids=ids, scale=scale, ldx=cols + pad if pad else 0,
                       ldy=cols + 2 * pad if pad else 0)
    _say("case sort", T, k, E, cols, x, ids, kind, "ws", op.workspace_bytes)
    off = torch.full((E + 1 + 2,), 77, dtype=torch.int32, device="cuda")
    rw = torch.full((T + 2, k), 77, dtype=torch.int32, device="cuda")
    more, X, Y, st = {}, None, None, None
    if cols:
        X = _draw(g, T, cols, TORCH[x])
        Y = Out(T * k, cols, TORCH[x], cols + 2 * pad)
        more = dict(X=_strided(X, pad), Y=Y.t)
    if scale:
        sc = torch.rand(T, generator=g)
        st = torch.full((T * k,), 7.0, device="cuda")
        more.update(scale=sc.cuda(), scale_out=st)
    op(choice.cuda(), offsets=off[1:E + 2], rows=rw[1:T + 1], **more)
    torch.cuda.synchronize()
    assert torch.equal(off.cpu()[1:E + 2], offsets) and off[0] == 77 and off[-1] == 77
    assert torch.equal(rw.cpu()[1:T + 1], rows) and (rw[0] == 77).all() and (rw[-1] == 77).all()
    token = torch.full((T * k,), -1)
    flat = rows.reshape(-1)
    token[flat[flat >= 0].long()] = torch.arange(T * k)[flat >= 0] // k
    if cols:
        assert Y.intact()
        got = Y.t.cpu().float()
        assert torch.equal(got[:n], X.float()[token[:n]])
        assert (got[n:] == -80.0).all(), "rows behind the last were written"
    if scale:
        assert torch.equal(st.cpu()[:n], sc[token[:n]]) and (st.cpu()[n:] == 7.0).all()
    op.close()


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (16, 8, 64), (63, 1, 2), (64, 1, 1024), (65, 3, 13),
                                   (512, 8, 128), (4096, 1, 16), (4097, 1, 16), (8192, 1, 16), (8193, 1, 1024), (683, 6, 1000), (5000, 8, 256),
                                   (20, 64, 100), (12345, 5, 33)])
def test_sort(T, k, E):
    run_sort(T, k, E, 64, kind="some", seed=T)
    run_sort(T, k, E, 0, kind="all", ids="i32", seed=T)


@pytest.mark.parametrize("kind", ["one", "none"])
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (37, 4, 6), (2050, 4, 64)])
def test_sort_one_expert_or_none(kind, T, k, E):
    run_sort(T, k, E, 128, kind=kind)
    run_sort(T, k, E, 128, kind=kind, ids="i32", pad=32)


@pytest.mark.parametrize("x,cols", [("bf16", 8), ("f16", 1032), ("f32", 4), ("f32", 2052), ("e4m3", 16), ("i8", 4112)])
def test_sort_types_and_strides(x, cols):
    run_sort(100, 3, 7, cols, x=x, scale=x in ("e4m3", "i8"))
    run_sort(1001, 3, 7, cols, x=x, scale=True, pad=16, ids="i32")


def run_combine(T, k, cols, x="bf16", weights=True, res=False, pad=0, inplace=False, E=6, kind="some", seed=0):
    g = torch.Generator().manual_seed(seed)
    _, rows = ref.sort(_ids(g, T, k, E, kind), E)
    DT = TORCH[x]
    Y = _draw(g, T * k, cols, DT)
    n = int((rows >= 0).sum())
    Y[n:] = NAN  # rows that nobody has
    w = torch.randn(T, k, generator=g) if weights else None
    if weights:
        w[rows < 0] = NAN
    R = _draw(g, T, cols, DT) if res else None
    op = ge.ExpertCombine(T, k, cols, x=x, weights=weights, residual=res, ldy=cols + pad if pad else 0,
                          ldd=cols + 2 * pad if pad else 0, ldr=cols + 2 * pad if pad and res else 0)
    D = Out(T, cols, DT, cols + 2 * pad)
    Rd = _strided(R, 2 * pad) if res else None
    if inplace:
        D.t.copy_(Rd)
        Rd = D.t
    _say("case combine", T, k, cols, x, weights, res, pad)
    op(_strided(Y, pad), rows.cuda(), w.cuda() if weights else None, D=D.t, residual=Rd)
    torch.cuda.synchronize()
    assert D.intact()
    d, bound = ref.combine(Y, rows, w, R)
    linear_ref.check("D", D.t, d, bound + linear_ref.half_step(d.abs() + bound, DT))
    op.close()


@pytest.mark.parametrize("T,k,cols", [(1, 1, 8), (1, 8, 4096), (37, 4, 520), (1001, 3, 1032), (300, 64, 16), (4100, 5, 256),
                                      (33, 9, 8192)])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_combine(T, k, cols, x):
    run_combine(T, k, cols, x, seed=T)
    run_combine(T, k, cols, x, weights=False, res=True, seed=T)


@pytest.mark.parametrize("kind", ["one", "none"])
def test_combine_one_expert_or_none(kind):
    run_combine(77, 4, 264, kind=kind, res=kind == "one")


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_combine_strides_and_in_place(x):
    run_combine(65, 3, 264, x, res=True, pad=16)
    run_combine(65, 3, 264, x, res=True, pad=16, inplace=True)
    run_combine(65, 3, 264, x, res=True, inplace=True)


def run_combine_grad(T, k, cols, x="bf16", pad=0, E=6, kind="some", seed=0):
    g = torch.Generator().manual_seed(seed)
    _, rows = ref.sort(_ids(g, T, k, E, kind), E)
    DT = TORCH[x]
    n = int((rows >= 0).sum())
    Y, dD, w = _draw(g, T * k, cols, DT), _draw(g, T, cols, DT), torch.randn(T, k, generator=g)
    Y[n:] = NAN
    w[rows < 0] = NAN
    op = ge.ExpertCombineGrad(T, k, cols, x=x, ldd=cols + pad if pad else 0, ldy=cols + 2 * pad if pad else 0,
                              ldg=cols + 3 * pad if pad else 0)
    dY = Out(T * k, cols, DT, cols + 3 * pad)
    dw = torch.full((T + 2, k), 77.0, device="cuda")
    _say("case combine_grad", T, k, cols, x, pad, kind)
    op(_strided(dD, pad), _strided(Y, 2 * pad), rows.cuda(), w.cuda(), dY=dY.t, dweights=dw[1:T + 1])
    torch.cuda.synchronize()
    assert dY.intact() and (dw[0] == 77).all() and (dw[-1] == 77).all()
    dy, dwr, bound = ref.combine_grad(dD, Y, rows, w)
    assert (dY.t.cpu()[n:].float() == -80.0).all(), "rows behind the last were written"
    linear_ref.check("dY", dY.t[:n], dy[:n], ref.rounded(dy[:n], DT, 1))
    linear_ref.check("dweights", dw[1:T + 1], dwr, bound)
    op.close()


@pytest.mark.parametrize("T,k,cols", [(1, 1, 8), (1, 8, 4096), (37, 4, 520), (1001, 3, 1032), (100, 64, 16), (2500, 5, 256),
                                      (2048, 2, 1000), (33, 9, 8192)])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_combine_grad(T, k, cols, x):
    run_combine_grad(T, k, cols, x, seed=T)


@pytest.mark.parametrize("kind", ["one", "none"])
def test_combine_grad_one_expert_or_none(kind):
    run_combine_grad(77, 4, 264, kind=kind)
    run_combine_grad(2100, 3, 264, kind=kind, pad=8)


def test_gradient_against_differences():
    """<dY, y'> and <dweights, w'> are the derivative of <dD, D> along (y', w'),
    which is linear in each: differences of whole steps, in 64 bits."""
    g = torch.Generator().manual_seed(3)
    T, k, cols, E = 50, 3, 64, 4
    _, rows = ref.sort(_ids(g, T, k, E), E)
    n = int((rows >= 0).sum())
    Y, Yp, dD = (_draw(g, m, cols, torch.float32) for m in (T * k, T * k, T))
    w, wp = torch.randn(T, k, generator=g), torch.randn(T, k, generator=g)
    grad = ge.ExpertCombineGrad(T, k, cols, x="f32")
    dY, dw = torch.zeros(T * k, cols, device="cuda"), torch.zeros(T, k, device="cuda")
    _say("case differences")
    grad(dD.cuda(), Y.cuda(), rows.cuda(), w.cuda(), dY=dY, dweights=dw)
    value = lambda y, v: (linear_ref.f64(dD) * ref.combine(y, rows, v)[0]).sum()  # noqa: E731
    y64, w64 = Y.double(), w.double()
    along_y = (value(y64 + Yp, w64) - value(y64 - Yp, w64)) / 2
    along_w = (value(y64, w64 + wp) - value(y64, w64 - wp)) / 2
    got_y = (linear_ref.f64(dY)[:n] * Yp.double()[:n]).sum()
    got_w = (linear_ref.f64(dw) * wp.double()).sum()
    # every term is off by at most (cols + 2) U of its size (bound of dweights; dY by U)
    size_y = (linear_ref.f64(dY)[:n].abs() * Yp.double()[:n].abs()).sum()
    size_w = (ref.combine_grad(dD, Y, rows, w)[2] * wp.double().abs()).sum()
    assert abs(got_y - along_y) <= 2 * linear_ref.U * size_y + 1e-12 * abs(along_y)
    assert abs(got_w - along_w) <= size_w + 1e-12 * abs(along_w)


def test_sort_gradient_is_combine():
    """The gradient of <G, Y> with Y[rows[t][j]] = X[t] is the sum of G's rows."""
    g = torch.Generator().manual_seed(4)
    T, k, cols, E = 70, 4, 40, 9
    ids = _ids(g, T, k, E)
    offsets, rows = (torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda"))
    G, dX = _draw(g, T * k, cols, torch.float32), torch.zeros(T, cols, device="cuda")
    _say("case sort gradient")
    ge.ExpertSort(T, k, E)(ids.cuda(), offsets=offsets, rows=rows)
    ge.ExpertCombine(T, k, cols, x="f32", weights=False)(G.cuda(), rows, D=dX)
    for t in range(T):
        want = sum((G[r] for r in rows.cpu()[t].tolist() if r >= 0), torch.zeros(cols)).double()
        assert (dX.cpu()[t].double() - want).abs().max() <= 2 * (k + 1) * linear_ref.U * G.abs().max() * k


def test_rows_outside_the_batch_add_nothing():
    T, k, cols = 8, 2, 64
    Y = torch.ones(T * k, cols, dtype=torch.bfloat16, device="cuda")
    rows = torch.arange(T * k, dtype=torch.int32).reshape(T, k)
    rows[3, 1], rows[4, 0], rows[5] = T * k, (1 << 31) - 1, -(1 << 31)
    D = torch.zeros(T, cols, dtype=torch.bfloat16, device="cuda")
    _say("case rows outside")
    ge.ExpertCombine(T, k, cols, weights=False)(Y, rows.cuda(), D=D)
    assert D[:, 0].tolist() == [2, 2, 2, 1, 1, 0, 2, 2]


def test_far_rows():
    """Rows more than 4 GiB into their tensors."""
    T, k, E, cols, ld = 70000, 2, 3, 16, 32768
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("less than 40 GiB of device memory free")
    g = torch.Generator().manual_seed(6)
    ids = _ids(g, T, k, E, "all")
    _, rows = ref.sort(ids, E)
    X = _draw(g, T, cols, torch.bfloat16)
    big = torch.zeros(T * k, ld, dtype=torch.bfloat16, device="cuda")
    Y = big[:, :cols]
    off, rw = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
    _say("case far rows")
    ge.ExpertSort(T, k, E, cols=cols, ldy=ld)(ids.cuda(), X.cuda(), offsets=off, rows=rw, Y=Y)
    assert torch.equal(rw.cpu(), rows) and torch.equal(Y[rw.reshape(-1).long()].cpu(), X.repeat_interleave(k, 0))
    D = torch.zeros(T, cols, dtype=torch.bfloat16, device="cuda")
    ge.ExpertCombine(T, k, cols, weights=False, ldy=ld)(Y, rw, D=D)
    assert torch.equal(D.cpu(), (2 * X.float()).bfloat16())
    dw = torch.zeros(T, k, device="cuda")
    w = torch.full((T, k), 0.5, device="cuda")
    dD = torch.ones(T, cols, dtype=torch.bfloat16, device="cuda")
    dY = torch.zeros_like(big)[:, :cols]
    ge.ExpertCombineGrad(T, k, cols, ldy=ld, ldg=ld)(dD, Y, rw, w, dY=dY, dweights=dw)
    assert (dY == 0.5).all()
    want = X.double().sum(1)
    bound = (cols + 2) * linear_ref.U * X.double().abs().sum(1)
    assert ((dw.cpu().double() - want[:, None]).abs() <= bound[:, None]).all()


def test_streams_and_graphs():
    """Two streams at once and two graphs replayed in turn give what one call
    gives, with rows of their own and a workspace each."""
    g = torch.Generator().manual_seed(8)
    T, k, E, cols = 3000, 4, 40, 256  # three chunks of the sort
    ids = _ids(g, T, k, E).cuda()
    X, w = _draw(g, T, cols, torch.bfloat16).cuda(), torch.rand(T, k, generator=g).cuda()
    sort, back = ge.ExpertSort(T, k, E, cols=cols), ge.ExpertCombine(T, k, cols)
    grad = ge.ExpertCombineGrad(T, k, cols)
    assert sort.workspace_bytes > 0

    def new():
        z = lambda *s, **d: torch.zeros(*s, device="cuda", **d)  # noqa: E731
        b = dict(dtype=torch.bfloat16)
        return dict(offsets=z(E + 1, dtype=torch.int32), rows=z(T, k, dtype=torch.int32), Y=z(T * k, cols, **b),
                    D=z(T, cols, **b), dY=z(T * k, cols, **b), dw=z(T, k))

    def run(o, stream=None):
        sort(ids, X, offsets=o["offsets"], rows=o["rows"], Y=o["Y"], stream=stream)
        back(o["Y"], o["rows"], w, D=o["D"], stream=stream)
        grad(o["D"], o["Y"], o["rows"], w, dY=o["dY"], dweights=o["dw"], stream=stream)

    _say("case streams and graphs")
    want = new()
    run(want)
    torch.cuda.synchronize()
    same = lambda o: all(torch.equal(o[n], want[n]) for n in want)  # noqa: E731
    outs = [new() for _ in range(6)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        run(o, streams[i % 2])
    torch.cuda.synchronize()
    assert all(map(same, outs))
    graphs = []
    for o in outs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            run(o)
        graphs.append(gr)
    for _ in range(3):
        for o in outs[:2]:
            for v in o.values():
                v.zero_()
        eager = new()
        for gr in graphs:
            gr.replay()
        run(eager)
        torch.cuda.synchronize()
        assert same(eager) and all(map(same, outs[:2]))


def test_refusals():
    T, k, E, cols = 8, 2, 4, 64
    ids = torch.zeros(T, k, dtype=torch.int64, device="cuda")
    off, rows = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
    X = torch.zeros(T, cols, dtype=torch.bfloat16, device="cuda")
    Y = torch.zeros(T * k, cols, dtype=torch.bfloat16, device="cuda")
    sort = ge.ExpertSort(T, k, E, cols=cols)
    for bad in (dict(ids=ids.int()), dict(ids=ids[:4]), dict(X=X[:4]), dict(X=X.float()), dict(Y=Y[:4]), dict(X=None),
                dict(Y=None), dict(rows=off), dict(scale=torch.zeros(T, device="cuda")), dict(ids=ids.cpu())):
        with pytest.raises((ValueError, ge.GemmEpiError)):
            sort(**(dict(ids=ids, X=X, offsets=off, rows=rows, Y=Y) | bad))
    flat = torch.zeros(T * cols * k + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ge.GemmEpiError):  # not at a 16-byte boundary
        sort(ids, X, offsets=off, rows=rows, Y=flat[1:1 + T * k * cols].view(T * k, cols))
    with pytest.raises(ge.GemmEpiError):  # Y begins where X does
        sort(ids, Y[:T], offsets=off, rows=rows, Y=Y)
    back = ge.ExpertCombine(T, k, cols, residual=True)
    w, D = torch.zeros(T, k, device="cuda"), torch.zeros_like(X)
    for bad in (dict(weights=None), dict(residual=None), dict(D=Y[:T]), dict(weights=w.half()), dict(rows=rows.long())):
        with pytest.raises((ValueError, ge.GemmEpiError)):
            back(**(dict(Y=Y, rows=rows, weights=w, D=D, residual=X) | bad))
    grad = ge.ExpertCombineGrad(T, k, cols)
    dY, dw = torch.zeros_like(Y), torch.zeros_like(w)
    for bad in (dict(dY=Y), dict(dweights=w), dict(weights=None), dict(dD=Y)):
        with pytest.raises((ValueError, ge.GemmEpiError)):
            grad(**(dict(dD=X, Y=Y, rows=rows, weights=w, dY=dY, dweights=dw) | bad))
    with pytest.raises(ge.GemmEpiError):
        ge.ExpertSort(5000, 2, E)(torch.zeros(5000, 2, dtype=torch.int64, device="cuda"), offsets=off,
                                  rows=torch.zeros(5000, 2, dtype=torch.int32, device="cuda"),
                                  workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
