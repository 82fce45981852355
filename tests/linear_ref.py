"""Plain 64-bit forms of the linear layer and the norm on the CPU, and the
error bounds that the GPU tests hold the kernels to.

u = 2^-24 is fp32's rounding.  Every bound is a sum of

* the accumulator's: a sum of n products in any order is off by at most
  n u S with S = sum |a||b| (the e4m3 MFMA keeps fewer bits of a group of
  products: 1e-3 S, the bar of the GEMM's 16-bit outputs; int8 sums are exact
  and their conversion to fp32 is off by u);
* the fp32 steps behind it, one u of their operands each;
* an activation's: |act(z)| is off by |z| 2^-21 (its exponent's argument is
  off by a few u |z|, which the function's own slope damps; the fitted tail of
  gelu is off by 1e-6 relative, of at most 0.17), and an error e of z becomes
  at most 1.13 e (the largest slope);
* half a step of the output's type, eps / 2 of the value (plus half of its
  smallest subnormal).
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
         "i8": torch.int8}


def f64(t):
    """Stored values as float64 on the CPU."""
    t = t.detach().cpu()
    return t.to(torch.float32).double() if t.dtype == torch.float8_e4m3fn else t.double()


def half_step(v, dtype):
    return v.abs() * HALF_STEP[dtype] + TINY[dtype]


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        p = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * 2 * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def linear(A, B, act_name="none", bias=None, scale_a=None, scale_b=None, residual=None, alpha=1.0):
    """(D, Z, S): D and Z in 64 bits, S = |scales| * sum |a||b| + |bias|."""
    a, b = f64(A), f64(B)
    s = torch.full((1, 1), float(torch.tensor(alpha, dtype=torch.float32)), dtype=torch.float64)
    if scale_a is not None:
        s = s * f64(scale_a)[:, None]
    if scale_b is not None:
        s = s * f64(scale_b)
    z = s * (a @ b.T)
    S = s.abs() * (a.abs() @ b.abs().T)
    if bias is not None:
        z = z + f64(bias)
        S = S + f64(bias).abs()
    d = act(z, act_name)
    if residual is not None:
        d = d + f64(residual)
    return d, z, S


def linear_bounds(d, z, S, K, ab, dtype, fp8_mfma, residual=None):
    """Bounds on |D - d| and |Z - z|."""
    acc = 1e-3 if fp8_mfma else (2 * U if ab == "i8" else K * U)
    ez = (acc + 4 * U) * S
    r = f64(residual).abs() if residual is not None else 0.0
    ed = 1.13 * ez + z.abs() * 2.0 ** -21 + U * (z.abs() + r)
    return ed + half_step(d.abs() + ed, dtype), ez + half_step(z.abs() + ez, dtype)


def check(name, got, want, bound):
    got = f64(got)
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError("%s: %d of %d outside their bounds, first at %d: got %r want %r bound %r" % (
            name, int(bad.sum()), bad.numel(), i, float(got.reshape(-1)[i]), float(want.reshape(-1)[i]),
            float(bound.expand_as(want).reshape(-1)[i])))


def rmsnorm(x, w, eps, residual=None):
    """(h, s, y) in 64 bits."""
    h = f64(x)
    if residual is not None:
        h = h + f64(residual)
    s = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32)))
    return h, s, h * s * f64(w)


def norm_rel(cols):
    """Relative error of the fp32 row statistics: a thread adds at most
    cols / 64 + 8 squares, the joins 10 more, the mean, root and quotient 6,
    halved by the root; y has 3 roundings of its own (h, * s, * w)."""
    return (cols / 64 + 32) * U


def rmsnorm_grad(dy, h, w, eps, dh_in=None):
    """(dh, dw, bound of dh without the output's rounding, sum |dy h s|)."""
    dy, h, w = f64(dy), f64(h), f64(w)
    s = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32)))
    g = dy * w
    dh = s * g - h * s ** 3 * (g * h).mean(dim=1, keepdim=True)
    size = s * g.abs() + h.abs() * s ** 3 * (g * h).abs().mean(dim=1, keepdim=True)
    if dh_in is not None:
        dh = dh + f64(dh_in)
        size = size + f64(dh_in).abs()
    return dh, (dy * h * s).sum(dim=0), 4 * norm_rel(h.shape[1]) * size, (dy * h * s).abs().sum(dim=0)
