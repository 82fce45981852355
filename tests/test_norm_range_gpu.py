"""The root-mean-square norm and its backward far from 1: rows whose statistics
lie near the ends of fp32's range, rows of zeros, a small or no eps.  The forms and bounds are those of tests/linear_ref.py: no
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
