"""The root-mean-square norm and its backward on the GPU against plain 64-bit
forms (tests/linear_ref.py), and the norm in front of the linear layer."""
import sys

import pytest
import torch

import beta_epilogue_amd as ge
import linear_ref as ref
from test_linear_gpu import NAN, Out, _draw, _strided

pytestmark = pytest.mark.gpu

EPS = 1e-6
QMAX = {"e4m3": 448.0, "i8": 127.0}


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def run_norm(rows, cols, x="bf16", y=None, res=False, weight=None, pad=0, seed=1, eps=EPS, X=None, R=None, keep_h=True):
    y, weight = y or x, weight or x
    g = torch.Generator().manual_seed(seed)
    chan = torch.exp(torch.randn(1, cols, generator=g))
    X = (torch.randn(rows, cols, generator=g) * chan).to(ref.TORCH[x]) if X is None else X
    R = (_draw(g, rows, cols, ref.TORCH[x], 2.0) if R is None else R) if res else None
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(ref.TORCH[weight])
    ld = cols + pad if pad else 0
    op = ge.RmsNorm(rows, cols, x=x, y=y, weight=weight, residual=res, eps=eps, ldx=ld, ldy=ld, ldr=ld if res else 0,
                    ldh=ld if res else 0)
    Y = Out(rows, cols, ref.TORCH[y], ld)
    H = Out(rows, cols, ref.TORCH[x], ld) if res and keep_h else None
    scale = torch.empty(rows, device="cuda") if y in QMAX else None
    _say("case", rows, cols, x, y, "res", res, "pad", pad)
    op(_strided(X, pad), w.cuda(), residual=_strided(R, pad) if res else None, Y=Y.t, H=H.t if H else None, scale=scale)
    torch.cuda.synchronize()
    assert Y.intact()
    h, s, want = ref.rmsnorm(X, w, eps, R)
    rel = ref.norm_rel(cols)
    size = (h.abs() + ref.U * h.abs()) * s * ref.f64(w).abs()
    if H is not None:
        assert H.intact()
        assert torch.equal(H.t.cpu(), (X.float() + R.float()).to(X.dtype)), "H is x + residual rounded once"
    if y in QMAX:
        sc = ref.f64(scale)
        top = want.abs().amax(dim=1).clamp_min(0)
        ref.check("scale", scale, (top / QMAX[y]).clamp_min(2.0 ** -126), (rel + 4 * ref.U) * top / QMAX[y] + 2.0 ** -149)
        got = ref.f64(Y.t) * sc[:, None]
        # half a step: e4m3 2^-4 of the value, at least half its smallest step 2^-9; int8 half a scale
        q = (want / sc[:, None]).abs()
        step = torch.maximum(q * 2.0 ** -4, torch.full_like(q, 2.0 ** -10)) if y == "e4m3" else torch.full_like(q, 0.5)
        bound = (step * (1 + 2.0 ** -20) + q * (rel + 6 * ref.U)) * sc[:, None]
        assert (got - want).abs().le(bound).all(), float(((got - want).abs() - bound).max())
        assert float(ref.f64(Y.t).abs().max()) <= QMAX[y]
    else:
        ref.check("Y", Y.t, want, rel * size + ref.half_step(want.abs() + rel * size, ref.TORCH[y]))
    op.close()


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 511), (9, 512), (7, 513), (4, 1000), (6, 1024), (3, 1025), (5, 2048),
          (2, 2051), (3, 4096), (2, 4099), (3, 8192), (2, 8193), (2, 16384), (1, 16383), (1000, 40)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f16", "e4m3"), ("f32", "i8"), ("f32", "f32"), ("bf16", "e4m3"),
                                 ("f16", "f16"), ("bf16", "i8")])
def test_norm(rows, cols, x, y):
    run_norm(rows, cols, x, y, res=True, seed=rows + cols)


@pytest.mark.parametrize("x,y", [("bf16", "e4m3"), ("f16", "i8"), ("f32", "f32"), ("f32", "e4m3"), ("f16", "f16")])
@pytest.mark.parametrize("cols", [33, 256, 1300, 5000, 9000])
def test_norm_strides_and_weights(cols, x, y):
    run_norm(5, cols, x, y, res=False, weight="f32", pad=3)
    run_norm(5, cols, x, y, res=True, pad=8, keep_h=False)
    run_norm(5, cols, x, y, res=True, pad=1)


def test_norm_eps():
    """Rows of tiny values, where eps decides; an all-zero row; eps 0."""
    X = torch.full((4, 96), 1e-4, dtype=torch.bfloat16)
    X[1] = 0
    X[2, 5:] = 0
    for y in ("bf16", "e4m3", "i8"):
        run_norm(4, 96, "bf16", y, X=X, eps=1e-6)
    run_norm(3, 96, "bf16", "bf16", X=X[[0, 2, 3]], eps=0.0)
    scale = torch.empty(4, device="cuda")
    Y = torch.empty(4, 96, dtype=torch.int8, device="cuda")
    ge.RmsNorm(4, 96, y="i8")(X.cuda(), torch.ones(96, dtype=torch.bfloat16, device="cuda"), Y=Y, scale=scale)
    assert (Y[1] == 0).all() and float(scale[1]) == 2.0 ** -126


@pytest.mark.parametrize("cols", [100, 3000])
@pytest.mark.parametrize("y", ["bf16", "e4m3", "i8"])
def test_norm_special_values(cols, y):
    """A NaN or an infinity stays in its row, which shows it."""
    X = torch.ones(4, cols, dtype=torch.bfloat16)
    X[1, cols // 2] = NAN
    X[2, 1] = float("inf")
    Y = torch.zeros(4, cols, dtype=ref.TORCH[y], device="cuda")
    scale = torch.zeros(4, device="cuda") if y != "bf16" else None
    _say("case", cols, y)
    ge.RmsNorm(4, cols, y=y)(X.cuda(), torch.ones(cols, dtype=torch.bfloat16, device="cuda"), Y=Y, scale=scale)
    v = Y.cpu().float()
    if scale is not None:
        v = v * scale.cpu()[:, None]
    assert torch.isnan(v[1]).any() and torch.isnan(v[2]).any()
    assert (v[0] - 1).abs().max() < 2.0 ** -4 and (v[3] - 1).abs().max() < 2.0 ** -4
    if scale is not None:
        assert not torch.isfinite(scale[1:3]).any() and torch.isfinite(scale[[0, 3]]).all()


def test_norm_in_place():
    g = torch.Generator().manual_seed(2)
    for cols in (300, 4100):
        X, R = _draw(g, 6, cols, torch.bfloat16), _draw(g, 6, cols, torch.bfloat16)
        w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
        op = ge.RmsNorm(6, cols, residual=True)
        want_y, want_h = (torch.empty(6, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        op(X.cuda(), w, residual=R.cuda(), Y=want_y, H=want_h)
        x, r = X.cuda(), R.cuda()
        op(x, w, residual=r, Y=x, H=r)
        assert torch.equal(x, want_y) and torch.equal(r, want_h)


def test_norm_refusals():
    op = ge.RmsNorm(4, 64, residual=True, y="e4m3")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    good = dict(x=bf(4, 64), weight=bf(64), residual=bf(4, 64), H=bf(4, 64), scale=torch.zeros(4, device="cuda"),
                Y=torch.zeros(4, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn))
    op(**good)
    for bad in (dict(x=bf(4, 65)), dict(weight=bf(63)), dict(residual=None), dict(scale=None), dict(Y=bf(4, 64)),
                dict(x=bf(4, 64).float()), dict(H=good["weight"].expand(4, 64)), dict(scale=good["scale"].double())):
        with pytest.raises((ValueError, ge.GemmEpiError)):
            op(**(good | bad))
    same = ge.RmsNorm(4, 64, residual=True)
    x, r = bf(4, 64), bf(4, 64)
    with pytest.raises(ge.GemmEpiError):
        same(x, bf(64), residual=r, Y=x, H=x)
    torch.cuda.synchronize()


# --- backward --------------------------------------------------------------
def run_grad(rows, cols, x="bf16", weight=None, dweight="f32", dh_in=False, pad=0, seed=1, alias=None):
    weight = weight or x
    g = torch.Generator().manual_seed(seed)
    T = ref.TORCH[x]
    H, dY, I = (_draw(g, rows, cols, T, s) for s in (2.0, 1.0, 1.0))
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(ref.TORCH[weight])
    ld = cols + pad if pad else 0
    op = ge.RmsNormGrad(rows, cols, x=x, weight=weight, dweight=dweight, eps=EPS, ldy=ld, ldh=ld, ldi=ld, ldo=ld)
    Hd, dYd, Id = _strided(H, pad), _strided(dY, pad), _strided(I, pad) if dh_in else None
    out = Out(rows, cols, T, ld)
    dH = out.t if alias is None else {"H": Hd, "dY": dYd, "I": Id}[alias]
    dw = torch.empty(cols, dtype=ref.TORCH[dweight], device="cuda") if dweight else None
    _say("case", rows, cols, x, "pad", pad, "ws", op.workspace_bytes)
    op(dYd, Hd, w.cuda(), dH_in=Id, dH=dH, dweight=dw)
    torch.cuda.synchronize()
    assert out.intact()
    dh, dwr, bound, sw = ref.rmsnorm_grad(dY, H, w, EPS, I if dh_in else None)
    ref.check("dH", dH, dh, bound + ref.half_step(dh.abs() + bound, T))
    if dweight:
        e = (ref.norm_rel(cols) + (rows + 8) * ref.U) * sw
        ref.check("dweight", dw, dwr, e + ref.half_step(dwr.abs() + e, ref.TORCH[dweight]))
    op.close()


@pytest.mark.parametrize("rows,cols", SHAPES + [(1300, 520), (600, 3000), (300, 9001), (700, 6143), (3, 6145),
                                            (300, 12288), (2, 12289)])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
def test_grad(rows, cols, x):
    run_grad(rows, cols, x, dh_in=cols % 2 == 0, seed=cols)


def test_grad_forms():
    run_grad(40, 600, "bf16", weight="f32", dweight="bf16")
    run_grad(40, 1600, "f16", dweight=None, dh_in=True)
    for cols in (77, 1111, 5001, 12000):
        run_grad(33, cols, "bf16", dh_in=True, pad=5)
    for alias in ("H", "dY", "I"):
        run_grad(20, 2500, "bf16", dh_in=True, alias=alias)


def test_grad_against_differences():
    """Central differences of the 64-bit sum(dY * y) and sum(dY * y) + sum(dH_in
    * h); fp32 tensors, so the bound is that of the fp32 arithmetic plus the
    differences' own h^2 = 1e-8."""
    rows, cols = 6, 80
    g = torch.Generator().manual_seed(9)
    H, dY, I = (torch.randn(rows, cols, generator=g) for _ in range(3))
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    dH, dw = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda")
    ge.RmsNormGrad(rows, cols, x="f32")(dY.cuda(), H.cuda(), w.cuda(), dH_in=I.cuda(), dH=dH, dweight=dw)
    h64, w64 = H.double(), w.double()

    def f(h, w):
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * w
        return (dY.double() * y).sum() + (I.double() * h).sum()

    for grad, at in ((dH, 0), (dw, 1)):
        u = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        plus, minus = [h64, w64], [h64, w64]
        plus[at], minus[at] = plus[at] + 1e-4 * u, minus[at] - 1e-4 * u
        diff = float(f(*plus) - f(*minus)) / 2e-4
        got = float((ref.f64(grad) * u).sum())
        assert abs(got - diff) <= 1e-5 * float((ref.f64(grad).abs() * u.abs()).sum()) + 1e-6


def test_grad_graph_and_streams():
    rows, cols = 700, 1500
    g = torch.Generator().manual_seed(3)
    H, dY = (_draw(g, rows, cols, torch.bfloat16).cuda() for _ in range(2))
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    op = ge.RmsNormGrad(rows, cols)
    new = lambda: (torch.empty_like(H), torch.empty(cols, device="cuda"))  # noqa: E731
    dH, dw = new()
    op(dY, H, w, dH=dH, dweight=dw)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        o, gr = new(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            op(dY, H, w, dH=o[0], dweight=o[1])
        graphs.append((gr, o))
    for _ in range(3):
        for gr, o in graphs:
            o[0].zero_(), o[1].zero_()
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(o[0], dH) and torch.equal(o[1], dw)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [new() for _ in range(6)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        op(dY, H, w, dH=o[0], dweight=o[1], stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o[0], dH) and torch.equal(o[1], dw) for o in outs)


# --- together --------------------------------------------------------------
@pytest.mark.parametrize("q", ["e4m3", "i8"])
@pytest.mark.parametrize("M", [1, 33, 200])
def test_norm_linear(M, q):
    """The norm into 8 bits and the projection that reads it: equal to the two
    calls with kept buffers bit for bit, and within the 8-bit operands' own
    rounding of the 64-bit result (half a step of each element of the norm)."""
    N, K = 136, 1040
    g = torch.Generator().manual_seed(M)
    X, R = _draw(g, M, K, torch.bfloat16), _draw(g, M, K, torch.bfloat16)
    w = (1 + 0.3 * torch.randn(K, generator=g)).bfloat16()
    B, sb = _draw(g, N, K, ref.TORCH[q]), torch.rand(N, generator=g) / 200
    bias, add = torch.randn(N, generator=g), _draw(g, M, N, torch.bfloat16)
    op = ge.FusedNormLinear(M, N, K, q=q, act="silu", bias="f32", residual=True, add=True)
    D, H = (torch.empty(M, n, dtype=torch.bfloat16, device="cuda") for n in (N, K))
    _say("case", M, q)
    op(X.cuda(), w.cuda(), B.cuda(), sb.cuda(), D=D, residual=R.cuda(), H=H, bias=bias.cuda(), add=add.cuda())
    assert torch.equal(H.cpu(), (X.float() + R.float()).bfloat16())
    Q, s = torch.empty(M, K, dtype=torch.uint8, device="cuda").view(ref.TORCH[q]), torch.empty(M, device="cuda")
    op.norm(X.cuda(), w.cuda(), residual=R.cuda(), Y=Q, scale=s)
    D2 = op.linear(Q, B.cuda(), scale_a=s, scale_b=sb.cuda(), bias=bias.cuda(), residual=add.cuda(),
                   D=torch.empty_like(D))
    assert torch.equal(D, D2)
    d, z, S = ref.linear(Q, B, "silu", bias, s, sb, add)
    bd, _ = ref.linear_bounds(d, z, S, K, q, torch.bfloat16, M > 64 and q == "e4m3", add)
    ref.check("D", D, d, bd)
    _, _, y = ref.rmsnorm(X, w, 1e-6, R)
    sc = ref.f64(s)[:, None]
    half = torch.maximum(y.abs() * 2.0 ** -4, sc * 2.0 ** -10) if q == "e4m3" else 0.5 * sc.expand_as(y)
    b64 = ref.f64(B) * sb.double()[:, None]
    far = 1.2 * (half * 1.001) @ b64.abs().T + bd
    want, _, _ = ref.linear(y.float(), b64.float(), "silu", bias, residual=add)
    assert ((ref.f64(D) - want).abs() <= far).all()


def test_training_step_together():
    """Forward and backward of norm -> linear with kept tensors, gradients
    against 64-bit automatic differentiation of the same block; bf16 tensors:
    each of the five roundings on the way (Y, Z, dZ, dY, dH) moves a result by
    at most 2^-8 of the sums of absolute values, 3% of the largest in all."""
    M, N, K = 70, 72, 264
    g = torch.Generator().manual_seed(21)
    X, R = _draw(g, M, K, torch.bfloat16), _draw(g, M, K, torch.bfloat16)
    w = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16()
    W = _draw(g, N, K, torch.bfloat16, K ** -0.5)
    b, dD = 0.2 * torch.randn(N, generator=g), _draw(g, M, N, torch.bfloat16)
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    Y, H, D, Z = bf(M, K), bf(M, K), bf(M, N), bf(M, N)
    wd, Wd, dDd = w.cuda(), W.cuda(), dD.cuda()
    ge.RmsNorm(M, K, residual=True)(X.cuda(), wd, residual=R.cuda(), Y=Y, H=H)
    ge.FusedLinear(M, N, K, act="gelu", bias="f32", z=True)(Y, Wd, bias=b.cuda(), D=D, Z=Z)
    dZ, dY, dH = bf(M, N), bf(M, K), bf(M, K)
    dW, db, dw = (torch.empty(*s, device="cuda") for s in ((N, K), (N,), (K,)))
    ge.FusedLinearGrad(M, N, K, act="gelu", da="bf16", db="f32", dbias="f32")(
        dDd, Y, Wd, Z=Z, dZ=dZ, dA=dY, dB=dW, dbias=db)
    ge.RmsNormGrad(M, K)(dY, H, wd, dH=dH, dweight=dw)
    x, w6, W6, b6 = (t.double().requires_grad_() for t in (X, w, W, b))
    h = x + R.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * w6
    out = ref.act(y @ W6.T + b6, "gelu")
    out.backward(dD.double())
    for name, got, want in (("D", D, out.detach()), ("dH", dH, x.grad), ("dweight", dw, w6.grad), ("dW", dW, W6.grad),
                            ("dbias", db, b6.grad)):
        assert float((ref.f64(got) - want).abs().max()) <= 0.03 * float(want.abs().max()), name


def test_norm_more_rows_than_one_grid_direction():
    """2^26 rows and a few: four to a workgroup of 256 threads, which would be
    2^32 threads in one direction of the grid."""
    rows, n = (1 << 26) + 64, 64
    g = torch.Generator().manual_seed(5)
    X, w = torch.randn(n, 8, generator=g).to(torch.bfloat16).cuda(), torch.ones(8, dtype=torch.bfloat16, device="cuda")
    want = torch.empty_like(X)
    _say("case", rows, 8)
    ge.RmsNorm(n, 8)(X, w, Y=want)
    many = X.repeat(rows // n, 1)
    Y = torch.zeros_like(many)
    ge.RmsNorm(rows, 8)(many, w, Y=Y)
    assert (Y.view(-1, n, 8) == want).all()


def test_offsets_beyond_32_bits():
    """Tensors of 4.4 GB: every 256 rows give what they give alone, bit for
    bit; dweight sums 2 x 10^3 terms in a workgroup and 10^3 workgroups."""
    rep, cols = 2100, 4096
    g = torch.Generator().manual_seed(6)
    x, r, dy, i = (torch.randn(256, cols, generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    out = []
    for n in (1, rep):
        X, R = x.repeat(n, 1), r.repeat(n, 1)
        Y = torch.zeros(256 * n, cols, dtype=torch.int8, device="cuda")
        scale = torch.zeros(256 * n, device="cuda")
        _say("case", 256 * n, cols)
        ge.RmsNorm(256 * n, cols, y="i8", residual=True)(X, w, Y=Y, residual=R, H=X, scale=scale)
        dW = torch.zeros(cols, device="cuda")
        ge.RmsNormGrad(256 * n, cols)(dy.repeat(n, 1), X, w, dH=R, dH_in=i.repeat(n, 1), dweight=dW)
        out.append((Y, scale, X, R, dW))
    for big, base in zip(out[1][:4], out[0][:4]):
        assert (big.view((rep,) + base.shape) == base).all()
    h = out[0][2].double()
    terms = dy.double() * h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)
    bound = rep * terms.abs().sum(0) * 3100 * 2.0 ** -24
    assert ((out[1][4].double() - rep * terms.sum(0)).abs() <= bound).all()
