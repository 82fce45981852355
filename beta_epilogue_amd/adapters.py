"""Thin Python binding of the linear layer with low-rank adapters
(include/gemm_epi_adapters.h).

A plan object as in ``layers``: a handle for one problem shape, torch tensors
checked against it, nothing computed in Python.
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPES, _check, gemm_epi_plan
from . import layers
from .layers import ACTIVATIONS, TORCH_DTYPES, _code, _i32, _Plan, gemm_epi_linear_desc


class gemm_epi_adapter_linear_desc(ctypes.Structure):
    _fields_ = [("linear", gemm_epi_linear_desc), ("rank", _i32), ("adapters", _i32)]


_bound = None


def lib():
    """The loaded shared library, with this module's entry points declared."""
    global _bound
    if _bound is None:
        L = layers.lib()
        P, I, N = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        D = ctypes.POINTER(gemm_epi_adapter_linear_desc)
        for name, args in (("create", [D, ctypes.POINTER(P)]), ("create_variant", [D, I, ctypes.POINTER(P)]),
                           ("destroy", [P]), ("run", [P] * 12 + [N, P]), ("get_plan", [P, ctypes.POINTER(gemm_epi_plan)])):
            f = getattr(L, "gemm_epi_adapter_linear_" + name)
            f.argtypes, f.restype = args, I
        _bound = L
    return _bound


class AdapterLinear(_Plan):
    """D = act(A . B^T + bias + scale[g] (A . down[g]^T) . up[g]^T) + residual, where
    g = ids[m] is the adapter of row m (none outside 0 .. adapters - 1).

    A is M x K, B (the shared weight) N x K, ids M int32, down adapters x rank x K,
    up adapters x N x rank, scale adapters (fp32), D, residual and Z M x N.  ab: f16
    or bf16, the type of all of them but bias (its type, or None).  rank: a
    multiple of 8, at most 128.  Everything else is as in ``FusedLinear``.
    """

    _op = "adapter_linear"

    def __init__(self, M, N, K, rank, adapters, *, ab="bf16", act="none", bias=None, residual=False, z=False, lda=0,
                 ldb=0, ldd=0, ldr=0, ldz=0, splits=0, variant=-1):
        lib()
        code = _code(DTYPES, ab, "type")
        super().__init__(gemm_epi_adapter_linear_desc(gemm_epi_linear_desc(
            M, N, K, lda, ldb, ldd, ldr, ldz, code, code, _code(DTYPES, bias, "type"),
            _code(ACTIVATIONS, act, "activation"), int(residual), int(z), 0, 0, splits), rank, adapters), variant)
        ab, bias = TORCH_DTYPES[ab], TORCH_DTYPES[bias] if bias else None
        m, v = self._matrix, self._vector
        self._specs = (m("A", ab, M, K, lda or K), m("B", ab, N, K, ldb or K), v("ids", torch.int32, M),
                       ("down", ab, (adapters, rank, K), (rank * K, K, 1)),
                       ("up", ab, (adapters, N, rank), (N * rank, rank, 1)), v("scale", torch.float32, adapters),
                       v("bias", bias, N), m("residual", ab, M, N, ldr or N), m("D", ab, M, N, ldd or N),
                       m("Z", ab, M, N, ldz or N))
        self.workspace_bytes = self.plan["workspace_bytes"]

    @property
    def plan(self) -> dict:
        p = gemm_epi_plan()
        _check(lib().gemm_epi_adapter_linear_get_plan(self.handle, ctypes.byref(p)), "gemm_epi_adapter_linear_get_plan")
        return {k: getattr(p, k) for k, _ in p._fields_ if k != "name"} | {"name": p.name.decode()}

    def __call__(self, A, B, ids, down, up, scale, *, D, bias=None, residual=None, Z=None, stream=None,
                 workspace=None):
        ptr = self._ptr
        a, b, i, dn, u, sc, bs, r, d, z = self._specs
        raw, s = self._stream(stream)
        ws, nbytes, keep = self._workspace(self.workspace_bytes, workspace, s)
        code = self._run(self.handle, ptr(A, a), ptr(B, b), ptr(ids, i), ptr(down, dn), ptr(up, u), ptr(scale, sc),
                         ptr(bias, bs), ptr(residual, r), ptr(D, d), ptr(Z, z), ws, nbytes, raw)
        if code:
            _check(code, "gemm_epi_adapter_linear_run")
        return D
