"""The activations' far negative side, held to relative bounds: values go in
through the bias (A is zero) and come out in fp32.

In units of 2^-24 a rounding costs 1 and v_exp and v_rcp 2 each.
gelu, z = -a: E's argument a^2 / 2 log2(e) has 3 roundings (a^2, the constant,
their product), which E turns into 3 a^2 / 2; the polynomial in t, with t's own 3
amplified by at most 2.2 and the coefficients' cancellation 1.7, 12; E, its two
products and the one with z 5: 1.5 a^2 + 20 with what t adds as a factor, and the
fit's 8.8e-7.  gelu_tanh: the argument 2 u log2(e) has 8 roundings, each |2 u|;
sigmoid and product 7.  silu: 2 roundings of |z|, then 7."""
import pytest
import torch

import beta_epilogue_amd as ge
import linear_ref as ref
from test_linear_gpu import _say

pytestmark = pytest.mark.gpu

BOUND = {"gelu": lambda z: (1.5 * z * z + 20) * ref.U + 8.8e-7,
         "gelu_tanh": lambda z: (8 * (2 * 0.79788456 * z * (1 + 0.044715 * z * z)).abs() + 8) * ref.U,
         "silu": lambda z: (2 * z.abs() + 8) * ref.U}
LOW = {"gelu": -12.5, "gelu_tanh": -9.0, "silu": -80.0}  # (results are normal fp32 numbers)


@pytest.mark.parametrize("M", [2, 70])  # the few-row kernel and a tile kernel
@pytest.mark.parametrize("act", sorted(LOW))
def test_negative_tail(act, M):
    N, K = 8192, 64
    z = torch.linspace(LOW[act], 3.0, N)
    zero = lambda r: torch.zeros(r, K, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    D = torch.empty(M, N, device="cuda")
    op = ge.FusedLinear(M, N, K, d="f32", act=act, bias="f32")
    _say("case", act, M, op.plan["name"])
    op(zero(M), zero(N), bias=z.cuda(), D=D)
    want = ref.act(z.double(), act)
    rel = (ref.f64(D) - want).abs() / want.abs()
    off = (rel / BOUND[act](z.double())).max()
    print(act, "largest share of the bound", float(off))
    assert (D == D[0]).all() and float(off) <= 1
