"""The linear layer's backward of a forward with alpha: dA and dB carry it,
dbias and dZ do not, against the 64-bit formulas and against differences.
Bounds as in test_linear_gpu.run_grad, times |alpha|; the product with alpha and
the sum with dB_in are two further fp32 roundings, inside its 4 u."""
import pytest
import torch

import beta_epilogue_amd as ge
import linear_ref as ref
from beta_epilogue_amd import layers
from test_linear_gpu import ACTS, Out, _draw, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile,splits", [(0, 0), (64, 1), (64, 3), (128, 1), (128, 3), (256, 1), (256, 3)])
@pytest.mark.parametrize("ab,alpha", [("bf16", 0.5), ("f16", -1.7)])
def test_grad_alpha(ab, alpha, tile, splits):
    M, N, K = 333, 328, 456
    g = torch.Generator().manual_seed(tile + splits)
    T = ref.TORCH[ab]
    dD, Z = _draw(g, M, N, T), _draw(g, M, N, T, 1.5)
    A, B, C = _draw(g, M, K, T), _draw(g, N, K, T, K ** -0.5), torch.randn(N, K, generator=g)
    op = ge.FusedLinearGrad(M, N, K, ab=ab, act="gelu", da=ab, db="f32", dbias="f32", tile=tile, splits=splits)
    dA, dB, dZ, db = Out(M, K, T), Out(N, K, torch.float32), Out(M, N, T), Out(1, N, torch.float32)
    _say("case", ab, alpha, tile, splits)
    op(dD.cuda(), A.cuda(), B.cuda(), Z=Z.cuda(), dB_in=C.cuda(), dZ=dZ.t, dA=dA.t, dB=dB.t, dbias=db.t[0],
       alpha=alpha)
    torch.cuda.synchronize()
    assert all(o.intact() for o in (dA, dB, dZ, db))
    f = float(torch.tensor(alpha, dtype=torch.float32))
    z, dz = ref.f64(Z), ref.f64(dZ.t)
    exact = ref.f64(dD) * ref.act_slope(z, "gelu")
    err = ref.f64(dD).abs() * (1 + z.abs()) * 2.0 ** -20
    ref.check("dZ", dZ.t, exact, err + ref.half_step(exact.abs() + err, T))
    a, b = ref.f64(A), ref.f64(B)
    want, S = f * (dz @ b), abs(f) * (dz.abs() @ b.abs())
    ref.check("dA", dA.t, want, (N + 4) * ref.U * S + ref.half_step(want.abs() + N * ref.U * S, T))
    want, S = f * (dz.T @ a) + C.double(), abs(f) * (dz.abs().T @ a.abs()) + C.double().abs()
    ref.check("dB", dB.t, want, (M + 4) * ref.U * S + ref.half_step(want.abs() + M * ref.U * S, torch.float32))
    want, e = exact.sum(0), err.sum(0) + (M + 4) * ref.U * (exact.abs() + err).sum(0)
    ref.check("dbias", db.t[0], want, e + ref.half_step(want.abs() + e, torch.float32))


@pytest.mark.parametrize("act", ACTS)
def test_grad_alpha_against_differences(act):
    """Forward with alpha = 0.75 and its backward: central differences of
    sum(dD * act(alpha A B^T + b)), with the bound of
    test_linear_gpu.test_grad_against_differences."""
    M, N, K, alpha = 40, 48, 56, 0.75
    g = torch.Generator().manual_seed(12)
    A, B = _draw(g, M, K, torch.bfloat16), _draw(g, N, K, torch.bfloat16, K ** -0.5)
    b, dD = torch.randn(N, generator=g), _draw(g, M, N, torch.bfloat16)
    bf, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(device="cuda")
    D, Z = torch.empty(M, N, **bf), torch.empty(M, N, **bf)
    _say("case", act)
    ge.FusedLinear(M, N, K, act=act, bias="f32", z=True)(A.cuda(), B.cuda(), bias=b.cuda(), D=D, Z=Z, alpha=alpha)
    a, w, bb = ref.f64(A), ref.f64(B), b.double()
    shift = ref.f64(Z) - (alpha * (a @ w.T) + bb)  # the forward at which Z is exact
    if act == "relu":  # no difference may step over the kink
        dD = torch.where(ref.f64(Z).abs() < 0.02, torch.zeros_like(dD), dD)
    dA, dB, db = torch.empty(M, K, **f32), torch.empty(N, K, **f32), torch.empty(N, **f32)
    kw = {} if act == "none" else dict(Z=Z, dZ=torch.empty(M, N, **bf))
    ge.FusedLinearGrad(M, N, K, act=act, da="f32", db="f32", dbias="f32")(dD.cuda(), A.cuda(), B.cuda(), dA=dA, dB=dB,
                                                                      dbias=db, alpha=alpha, **kw)

    def f(a, w, bb):
        return (ref.f64(dD) * ref.act(alpha * (a @ w.T) + bb + shift, act)).sum()

    dz = (ref.f64(dD) * ref.act_slope(ref.f64(Z), act)).abs()
    h = 1e-4
    for grad, at, size in ((dA, 0, dz @ w.abs()), (dB, 1, dz.T @ a.abs()), (db, 2, dz.sum(0))):
        u = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        plus, minus = [a, w, bb], [a, w, bb]
        plus[at], minus[at] = plus[at] + h * u, minus[at] - h * u
        diff = float(f(*plus) - f(*minus)) / (2 * h)
        got = float((ref.f64(grad) * u).sum())
        assert abs(got - diff) <= 2.0 ** -8 * float((size * u.abs()).sum()), (act, at, got, diff)


def test_alpha_one_is_the_default():
    """Of the binding's call and of the C entry point without an alpha."""
    M, N, K = 130, 136, 264
    g = torch.Generator().manual_seed(1)
    dD, A, B = (_draw(g, *s, torch.bfloat16).cuda() for s in ((M, N), (M, K), (N, K)))
    op = ge.FusedLinearGrad(M, N, K, da="bf16", db="f32")
    out = [(torch.empty_like(A), torch.empty(N, K, device="cuda")) for _ in range(4)]
    op(dD, A, B, dA=out[0][0], dB=out[0][1])
    op(dD, A, B, dA=out[1][0], dB=out[1][1], alpha=1.0)
    ws = torch.empty(max(op.workspace_bytes, 1), dtype=torch.uint8, device="cuda")
    assert layers.lib().gemm_epi_linear_grad_run(
        op.handle, dD.data_ptr(), A.data_ptr(), B.data_ptr(), None, None, None, out[2][0].data_ptr(),
        out[2][1].data_ptr(), None, ws.data_ptr(), op.workspace_bytes, torch.cuda.current_stream().cuda_stream) == 0
    op(dD, A, B, dA=out[3][0], dB=out[3][1], alpha=2.0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in out[1:3] for a, b in zip(out[0], o))
    assert torch.equal(out[3][1], 2 * out[0][1])
