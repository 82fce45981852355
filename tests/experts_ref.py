"""Plain 64-bit forms of a mixture of experts' operators on the CPU, and the
bounds that the GPU tests hold the kernels to (U, half steps and ``check`` as in
linear_ref):

* combine: a chain of k + 1 fp32 steps is off by at most (k + 1) U times the sum
  of its terms' sizes, and D is rounded once;
* its gradient: dY is one fp32 product, rounded once; dweights is a sum of n
  products in some order, off by at most n U sum |d||y|.
"""
from __future__ import annotations

import torch

from linear_ref import U, f64, half_step


def sort(ids, experts):
    """(offsets, rows) as nested lists: a stable order by expert."""
    groups = [[] for _ in range(experts)]
    T, k = ids.shape
    for t, choice in enumerate(ids.tolist()):
        for j, e in enumerate(choice):
            if 0 <= e < experts:
                groups[e].append(t * k + j)
    offsets, rows, n = [0], torch.full((T * k,), -1, dtype=torch.int32), 0
    for g in groups:
        for i in g:
            rows[i] = n
            n += 1
        offsets.append(n)
    return torch.tensor(offsets, dtype=torch.int32), rows.reshape(T, k)


def combine(Y, rows, weights=None, residual=None):
    """(D, bound without the output's rounding)."""
    y, r = f64(Y), rows.long()
    w = torch.ones(rows.shape, dtype=torch.float64) if weights is None else f64(weights)
    T, k = rows.shape
    d = torch.zeros(T, y.shape[1], dtype=torch.float64) if residual is None else f64(residual)
    size = d.abs()
    for j in range(k):
        t = (r[:, j] >= 0).nonzero()[:, 0]
        term = w[t, j][:, None] * y[r[t, j]]
        d[t] += term
        size[t] += term.abs()
    return d, (k + 1) * U * size


def combine_grad(dD, Y, rows, weights):
    """(dY, dweights, bound of dweights); rows of dY that no choice has: NaN."""
    d, y, r, w = f64(dD), f64(Y), rows.long(), f64(weights)
    dy = torch.full(y.shape, float("nan"), dtype=torch.float64)
    dw = torch.zeros(rows.shape, dtype=torch.float64)
    size = torch.zeros_like(dw)
    for j in range(rows.shape[1]):
        t = (r[:, j] >= 0).nonzero()[:, 0]
        dy[r[t, j]] = w[t, j][:, None] * d[t]
        dw[t, j] = (d[t] * y[r[t, j]]).sum(1)
        size[t, j] = (d[t] * y[r[t, j]]).abs().sum(1)
    return dy, dw, (y.shape[1] + 2) * U * size


def rounded(v, dtype, steps=0.0):
    """Half a step of the output, and `steps` of fp32, around v."""
    e = v.abs() * steps * U
    return e + half_step(v.abs() + e, dtype)
