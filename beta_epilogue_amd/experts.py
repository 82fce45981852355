"""Thin Python binding of a mixture of experts' operators
(include/gemm_epi_experts.h): tokens sorted by expert and their results brought
back.

Plan objects as in ``layers``: a handle for one problem shape, torch tensors
checked against it, nothing computed in Python.  T tokens choose top_k experts
each; a choice outside 0 .. experts - 1 is none.  R = tokens * top_k rows lie
sorted by expert, those of expert e at offsets[e] .. offsets[e + 1] - 1; rows
behind offsets[experts] are neither read nor written.
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPES, _check
from . import layers
from .layers import TORCH_DTYPES, _code, _f32, _i32, _i64, _Plan

IDS_DTYPES = {"i32": torch.int32, "i64": torch.int64}


class gemm_epi_expert_sort_desc(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("cols", _i64), ("ldx", _i64), ("ldy", _i64), ("top_k", _i32), ("experts", _i32),
                ("ids_bits", _i32), ("x_dtype", _i32), ("scale", _i32)]


class gemm_epi_expert_combine_desc(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("cols", _i64), ("ldy", _i64), ("ldd", _i64), ("ldr", _i64), ("top_k", _i32),
                ("x_dtype", _i32), ("weights", _i32), ("residual", _i32)]


class gemm_epi_expert_combine_grad_desc(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("cols", _i64), ("ldd", _i64), ("ldy", _i64), ("ldg", _i64), ("top_k", _i32),
                ("x_dtype", _i32)]


_bound = None


def lib():
    """The loaded shared library, with this module's entry points declared."""
    global _bound
    if _bound is None:
        L = layers.lib()
        P, I, N = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        for op, desc in (("expert_sort", gemm_epi_expert_sort_desc),
                         ("expert_combine", gemm_epi_expert_combine_desc),
                         ("expert_combine_grad", gemm_epi_expert_combine_grad_desc)):
            create, destroy = getattr(L, "gemm_epi_%s_create" % op), getattr(L, "gemm_epi_%s_destroy" % op)
            create.argtypes, create.restype = [ctypes.POINTER(desc), ctypes.POINTER(P)], I
            destroy.argtypes, destroy.restype = [P], I
        L.gemm_epi_expert_sort_run.argtypes = [P] * 9 + [N, P]
        L.gemm_epi_expert_combine_run.argtypes = [P] * 7
        L.gemm_epi_expert_combine_grad_run.argtypes = [P] * 8
        for op in ("expert_sort", "expert_combine", "expert_combine_grad"):
            getattr(L, "gemm_epi_%s_run" % op).restype = I
        L.gemm_epi_expert_sort_workspace.argtypes, L.gemm_epi_expert_sort_workspace.restype = [P], N
        _bound = L
    return _bound


class _ExpertPlan(_Plan):
    """A plan whose entry points this module declares."""

    def __init__(self, *a, **k):
        lib()
        super().__init__(*a, **k)


class ExpertSort(_ExpertPlan):
    """Tokens sorted by expert: offsets, rows and Y[rows[t][j]] = X[t].

    ids (tokens x top_k, i32 or i64) are the experts that each token chose, as
    from ``torch.topk``.  offsets (experts + 1, int32) receives where each
    expert's rows begin, rows (tokens x top_k, int32) the row of every choice,
    -1 for none; within an expert the choices keep their order.  cols > 0: the
    rows of X (tokens x cols, type x: f16, bf16, f32, e4m3 or i8) are moved
    into Y (tokens * top_k x cols), with scale: one fp32 scale per row too
    (``RmsNorm``'s into 8 bits).  Its gradient is ``ExpertCombine`` without
    weights.  At most 64 choices per token and 1024 experts.
    """

    _op = "expert_sort"

    def __init__(self, tokens, top_k, experts, *, cols=0, x="bf16", ids="i64", scale=False, ldx=0, ldy=0):
        ids = _code(IDS_DTYPES, ids, "type of ids")
        super().__init__(gemm_epi_expert_sort_desc(tokens, cols, ldx, ldy, top_k, experts,
                                                   64 if ids is torch.int64 else 32,
                                                   _code(DTYPES, x, "type") if cols else 0, int(scale)))
        m, v, R = self._matrix, self._vector, tokens * top_k
        x = TORCH_DTYPES[x] if cols else None
        self._specs = (m("ids", ids, tokens, top_k, top_k), m("X", x, tokens, cols, ldx or cols),
                       v("offsets", torch.int32, experts + 1), m("rows", torch.int32, tokens, top_k, top_k),
                       m("Y", x, R, cols, ldy or cols), v("scale", torch.float32, tokens),
                       v("scale_out", torch.float32, R))
        self.workspace_bytes = lib().gemm_epi_expert_sort_workspace(self.handle)

    def __call__(self, ids, X=None, *, offsets, rows, Y=None, scale=None, scale_out=None, stream=None,
                 workspace=None):
        ptr = self._ptr
        si, sx, so, sr, sy, ss, st = self._specs
        raw, s = self._stream(stream)
        ws, nbytes, keep = self._workspace(self.workspace_bytes, workspace, s)
        code = self._run(self.handle, ptr(ids, si), ptr(X, sx), ptr(scale, ss), ptr(offsets, so), ptr(rows, sr),
                         ptr(Y, sy), ptr(scale_out, st), ws, nbytes, raw)
        if code:
            _check(code, "gemm_epi_expert_sort_run")
        return Y


class ExpertCombine(_ExpertPlan):
    """D[t] = residual[t] + sum over j of weights[t][j] Y[rows[t][j]].

    Y has tokens * top_k rows (``ExpertSort``'s order), rows is the sort's,
    weights (tokens x top_k, fp32) the router's.  A choice without a row adds
    nothing.  Sums are fp32 in the order of the choices.  weights=False: every weight
    is 1, which is the gradient of the sort's X (residual: what reaches X by
    other ways).  x: the type of Y, D and residual (f16, bf16 or f32).
    """

    _op = "expert_combine"

    def __init__(self, tokens, top_k, cols, *, x="bf16", weights=True, residual=False, ldy=0, ldd=0, ldr=0):
        super().__init__(gemm_epi_expert_combine_desc(tokens, cols, ldy, ldd, ldr, top_k, _code(DTYPES, x, "type"),
                                                      int(weights), int(residual)))
        x, m = TORCH_DTYPES[x], self._matrix
        self._specs = (m("Y", x, tokens * top_k, cols, ldy or cols), m("rows", torch.int32, tokens, top_k, top_k),
                       m("weights", torch.float32, tokens, top_k, top_k), m("residual", x, tokens, cols, ldr or cols),
                       m("D", x, tokens, cols, ldd or cols))

    def __call__(self, Y, rows, weights=None, *, D, residual=None, stream=None):
        ptr = self._ptr
        sy, sr, sw, sx, sd = self._specs
        code = self._run(self.handle, ptr(Y, sy), ptr(rows, sr), ptr(weights, sw), ptr(residual, sx), ptr(D, sd),
                         self._stream(stream)[0])
        if code:
            _check(code, "gemm_epi_expert_combine_run")
        return D


class ExpertCombineGrad(_ExpertPlan):
    """The gradients of ``ExpertCombine``: dY[rows[t][j]] = weights[t][j] dD[t]
    and dweights[t][j] = dD[t] . Y[rows[t][j]] (fp32; 0 for a choice without a
    row).  The residual's gradient is dD.
    """

    _op = "expert_combine_grad"

    def __init__(self, tokens, top_k, cols, *, x="bf16", ldd=0, ldy=0, ldg=0):
        super().__init__(gemm_epi_expert_combine_grad_desc(tokens, cols, ldd, ldy, ldg, top_k,
                                                           _code(DTYPES, x, "type")))
        x, m, R = TORCH_DTYPES[x], self._matrix, tokens * top_k
        self._specs = (m("dD", x, tokens, cols, ldd or cols), m("Y", x, R, cols, ldy or cols),
                       m("rows", torch.int32, tokens, top_k, top_k), m("weights", torch.float32, tokens, top_k, top_k),
                       m("dY", x, R, cols, ldg or cols), m("dweights", torch.float32, tokens, top_k, top_k))

    def __call__(self, dD, Y, rows, weights, *, dY, dweights, stream=None):
        ptr = self._ptr
        sd, sy, sr, sw, sg, sv = self._specs
        code = self._run(self.handle, ptr(dD, sd), ptr(Y, sy), ptr(rows, sr), ptr(weights, sw), ptr(dY, sg),
                         ptr(dweights, sv), self._stream(stream)[0])
        if code:
            _check(code, "gemm_epi_expert_combine_grad_run")
        return dY
