"""The root-mean-square norm and its backward far from 1: rows whose statistics
lie near the ends of fp32's range, rows of zeros, a small or no eps, NaN with a
payload.  The forms and bounds are those of tests/linear_ref.py: no
intermediate of either kernel leaves fp32's normal range at these magnitudes,
so the relative bounds hold as they stand."""
import pytest
import torch

import beta_epilogue_amd as ge
import linear_ref as ref
from test_linear_gpu import _draw
from test_norm_gpu import _say, run_norm

pytestmark = pytest.mark.gpu


def _grad(H, dY, w, eps, dh_in=None, x="bf16"):
    rows, cols = H.shape
    dH = torch.empty(rows, cols, dtype=ref.TORCH[x], device="cuda")
    dw = torch.empty(cols, device="cuda")
    op = ge.RmsNormGrad(rows, cols, x=x, weight="f32", eps=eps)
    op(dY.cuda(), H.cuda(), w.cuda(), dH=dH, dweight=dw, dH_in=dh_in.cuda() if dh_in is not None else None)
    torch.cuda.synchronize()
    return dH, dw


# Row sizes of one and several waves a row, with whole and cut groups.
COLS = [7, 96, 700, 2051, 4097, 9000]


@pytest.mark.parametrize("rms,eps", [(5e15, 1e-6), (1e13, 1e-6), (1e-14, 0.0), (1e-11, 1e-24)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_grad_magnitudes(cols, x, rms, eps):
    """dH = s (g - xhat mean(g xhat)) is of ordinary size (s times g) although
    s^3 is not a normal fp32 number."""
    rows = 5
    g = torch.Generator().manual_seed(cols)
    T = ref.TORCH[x]
    H, dY = _draw(g, rows, cols, T, rms), _draw(g, rows, cols, T)
    dY = (dY.float() + 3 * H.float() / rms).to(T)  # (so that the mean of g xhat is not small)
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    _say("case", cols, x, rms, eps)
    dH, dw = _grad(H, dY, w, eps, x=x)
    dh, dwr, bound, sw = ref.rmsnorm_grad(dY, H, w, eps)
    ref.check("dH", dH, dh, bound + ref.half_step(dh.abs() + bound, T))
    e = (ref.norm_rel(cols) + (rows + 8) * ref.U) * sw
    ref.check("dweight", dw, dwr, e + ref.half_step(dwr.abs() + e, torch.float32))


@pytest.mark.parametrize("eps", [1e-6, 1e-30])
@pytest.mark.parametrize("cols", COLS)
def test_grad_zero_rows(cols, eps):
    """A row of zeros (padding) has dH = dH_in + g / sqrt(eps), for the
    smallest eps too, and adds nothing to dweight."""
    g = torch.Generator().manual_seed(cols)
    H, dY, I = (_draw(g, 6, cols, torch.float32) for _ in range(3))
    H[1], H[4] = 0, 0
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    _say("case", cols, eps)
    dH, dw = _grad(H, dY, w, eps, I, "f32")
    dh, dwr, bound, sw = ref.rmsnorm_grad(dY, H, w, eps, I)
    ref.check("dH", dH, dh, bound + ref.half_step(dh.abs() + bound, torch.float32))
    e = (ref.norm_rel(cols) + 14 * ref.U) * sw
    ref.check("dweight", dw, dwr, e + ref.half_step(dwr.abs() + e, torch.float32))


@pytest.mark.parametrize("rms,eps", [(5e15, 1e-6), (1e-14, 0.0), (1e-11, 1e-24)])
@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("bf16", "e4m3"), ("bf16", "i8"), ("f32", "f32"), ("f32", "i8")])
@pytest.mark.parametrize("cols", [96, 2051, 9000])
def test_norm_magnitudes(cols, x, y, rms, eps):
    X = _draw(torch.Generator().manual_seed(cols), 5, cols, ref.TORCH[x], rms)
    run_norm(5, cols, x, y, X=X, eps=eps)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("y", ["bf16", "e4m3", "i8"])
def test_zero_rows_without_eps(cols, y):
    """eps 0: a row of zeros gives zeros (with the least scale), and its
    neighbours what they give alone."""
    g = torch.Generator().manual_seed(cols)
    X = _draw(g, 4, cols, torch.bfloat16)
    X[1], X[3] = 0, 0
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")

    def run(x):
        n = x.shape[0]
        Y = torch.full((n, cols), 5.0).to(ref.TORCH[y]).cuda()
        scale = torch.full((n,), 5.0, device="cuda") if y != "bf16" else None
        ge.RmsNorm(n, cols, y=y, eps=0.0)(x.cuda(), w, Y=Y, scale=scale)
        torch.cuda.synchronize()
        return Y.float(), scale

    _say("case", cols, y)
    Y, scale = run(X)
    alone, s = run(X[[0, 2]])
    assert (Y[[1, 3]] == 0).all() and torch.equal(Y[[0, 2]], alone)
    if scale is not None:
        assert (scale[[1, 3]] == 2.0 ** -126).all() and torch.equal(scale[[0, 2]], s)


@pytest.mark.parametrize("cols", COLS)
def test_grad_zero_rows_without_eps(cols):
    """eps 0 stands for 2^-149: a row of zeros whose dY is 0 (padding) has dH =
    dH_in, and another g 2^74.5, the formula's value; neither adds to dweight."""
    g = torch.Generator().manual_seed(cols)
    H, dY, I = (_draw(g, 5, cols, torch.float32) for _ in range(3))
    H[1], H[3] = 0, 0
    dY[1] = 0
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    _say("case", cols)
    dH, dw = _grad(H, dY, w, 0.0, I, "f32")
    dh, dwr, bound, sw = ref.rmsnorm_grad(dY, H, w, 2.0 ** -149, I)
    assert torch.equal(dH[1].cpu(), I[1])
    ref.check("dH", dH, dh, bound + ref.half_step(dh.abs() + bound, torch.float32))
    e = (ref.norm_rel(cols) + 13 * ref.U) * sw
    ref.check("dweight", dw, dwr, e + ref.half_step(dwr.abs() + e, torch.float32))


@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_int8_of_nan_with_payload(cols, x):
    """int8 values that would be NaN are 0, whatever bits the NaN has: in an
    fp32 weight, and in an fp32 x."""
    nan = torch.tensor([0x7fc01234, 0x7f800055], dtype=torch.int32).view(torch.float32)  # quiet, signalling
    w = torch.ones(cols)
    X = torch.ones(3, cols, dtype=ref.TORCH[x])
    Y, scale = torch.full((3, cols), 9, dtype=torch.int8, device="cuda"), torch.zeros(3, device="cuda")
    op = ge.RmsNorm(3, cols, x=x, y="i8", weight="f32")
    _say("case", cols, x)
    for v in nan:
        bad = w.clone()
        bad[cols // 2] = v
        op(X.cuda(), bad.cuda(), Y=Y.fill_(9), scale=scale)
        assert (Y == 0).all() and torch.isnan(scale).all()
        if x == "f32":
            Z = X.clone()
            Z[1, cols // 2] = v
            op(Z.cuda(), w.cuda(), Y=Y.fill_(9), scale=scale)
            assert (Y[1] == 0).all() and torch.isnan(scale[1]) and (Y[[0, 2]] == 127).all()
