"""Thin Python binding of a mixture of experts' operators
(include/gemm_epi_experts.h): tokens sorted by expert, the experts' linear
layers and the results brought back.

Plan objects as in ``layers``: a handle for one problem shape, torch tensors
checked against it, nothing computed in Python.  T tokens choose top_k experts
each; a choice outside 0 .. experts - 1 is none.  R = tokens * top_k rows lie
sorted by expert, those of expert e at offsets[e] .. offsets[e + 1] - 1; rows
behind offsets[experts] are neither read nor written.
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPES, _check, gemm_epi_plan
from . import layers
from .layers import ACTIVATIONS, TORCH_DTYPES, _code, _i32, _i64, _Plan

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


class gemm_epi_expert_linear_desc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("N", _i64), ("K", _i64), ("lda", _i64), ("ldd", _i64), ("ldu", _i64), ("ldz", _i64),
                ("experts", _i32), ("ab_dtype", _i32), ("d_dtype", _i32), ("bias_dtype", _i32), ("act", _i32),
                ("mul", _i32), ("z", _i32), ("scale_a", _i32), ("scale_b", _i32)]


class gemm_epi_expert_linear_grad_desc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("N", _i64), ("K", _i64), ("experts", _i32), ("ab_dtype", _i32), ("act", _i32),
                ("mul", _i32), ("da_dtype", _i32), ("db_dtype", _i32), ("dbias_dtype", _i32), ("tile", _i32)]


_DESCS = {"expert_sort": gemm_epi_expert_sort_desc, "expert_combine": gemm_epi_expert_combine_desc,
          "expert_combine_grad": gemm_epi_expert_combine_grad_desc, "expert_linear": gemm_epi_expert_linear_desc,
          "expert_linear_grad": gemm_epi_expert_linear_grad_desc}

_bound = None


def lib():
    """The loaded shared library, with this module's entry points declared."""
    global _bound
    if _bound is None:
        L = layers.lib()
        P, I, N = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        for op, desc in _DESCS.items():
            create, destroy = getattr(L, "gemm_epi_%s_create" % op), getattr(L, "gemm_epi_%s_destroy" % op)
            create.argtypes, create.restype = [ctypes.POINTER(desc), ctypes.POINTER(P)], I
            destroy.argtypes, destroy.restype = [P], I
        L.gemm_epi_expert_sort_run.argtypes = [P] * 9 + [N, P]
        L.gemm_epi_expert_combine_run.argtypes = [P] * 7
        L.gemm_epi_expert_combine_grad_run.argtypes = [P] * 8
        L.gemm_epi_expert_linear_run.argtypes = [P] * 11
        L.gemm_epi_expert_linear_grad_run.argtypes = [P] * 14 + [N, P]
        for op in _DESCS:
            getattr(L, "gemm_epi_%s_run" % op).restype = I
        for op in ("expert_sort", "expert_linear_grad"):
            f = getattr(L, "gemm_epi_%s_workspace" % op)
            f.argtypes, f.restype = [P], N
        f = L.gemm_epi_expert_linear_create_variant
        f.argtypes, f.restype = [ctypes.POINTER(gemm_epi_expert_linear_desc), I, ctypes.POINTER(P)], I
        L.gemm_epi_expert_linear_get_plan.argtypes = [P, ctypes.POINTER(gemm_epi_plan)]
        L.gemm_epi_expert_linear_get_plan.restype = I
        L.gemm_epi_expert_linear_variant_count.argtypes, L.gemm_epi_expert_linear_variant_count.restype = [], I
        L.gemm_epi_expert_linear_variant_name.argtypes = [I]
        L.gemm_epi_expert_linear_variant_name.restype = ctypes.c_char_p
        _bound = L
    return _bound


def expert_linear_variant_names() -> list:
    """Names of the experts' linear layer's kernels, by variant number."""
    L = lib()
    return [L.gemm_epi_expert_linear_variant_name(i).decode() for i in range(L.gemm_epi_expert_linear_variant_count())]


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


class ExpertLinear(_ExpertPlan):
    """D[r] = act(scale_a[r] * scale_b[e] * (A[r] . B[e]^T) + bias[e]) * U[r] for
    the rows r of every expert e.

    A is rows x K (``ExpertSort``'s Y), B experts x N x K (packed), bias and
    scale_b experts x N, scale_a rows, D, U and Z rows x N; rows is the batch's
    capacity, tokens * top_k.  ab: f16, bf16, e4m3 or i8; d (of D, U and Z):
    f16, bf16 or f32.  bias: its type, or None; mul, z, scale_a, scale_b:
    whether the call has U, Z and the scales.  Z receives the pre-activation,
    which ``ExpertLinearGrad`` takes.  e4m3 with a 16-bit d sums with fewer bits than fp32
    in the tile kernels (where large products cancel, off by 0.0006 of the sum of |a||b|).  A gated layer is two calls: U = ExpertLinear
    of one weight, then act and mul with the other.  variant forces a kernel.
    """

    _op = "expert_linear"

    def __init__(self, rows, experts, N, K, *, ab="bf16", d=None, act="none", bias=None, mul=False, z=False,
                 scale_a=False, scale_b=False, lda=0, ldd=0, ldu=0, ldz=0, variant=-1):
        d = d or (ab if ab in ("f16", "bf16") else "bf16")
        super().__init__(gemm_epi_expert_linear_desc(
            rows, N, K, lda, ldd, ldu, ldz, experts, _code(DTYPES, ab, "type"), _code(DTYPES, d, "type"),
            _code(DTYPES, bias, "type"), _code(ACTIVATIONS, act, "activation"), int(mul), int(z), int(scale_a),
            int(scale_b)), variant)
        ab, d, bias = TORCH_DTYPES[ab], TORCH_DTYPES[d], TORCH_DTYPES[bias] if bias else None
        m, v = self._matrix, self._vector
        self._specs = (m("A", ab, rows, K, lda or K), ("B", ab, (experts, N, K), (N * K, K, 1)),
                       v("offsets", torch.int32, experts + 1), m("bias", bias, experts, N, N),
                       v("scale_a", torch.float32, rows), m("scale_b", torch.float32, experts, N, N),
                       m("U", d, rows, N, ldu or N), m("D", d, rows, N, ldd or N), m("Z", d, rows, N, ldz or N))

    @property
    def plan(self) -> dict:
        p = gemm_epi_plan()
        _check(lib().gemm_epi_expert_linear_get_plan(self.handle, ctypes.byref(p)), "gemm_epi_expert_linear_get_plan")
        return {k: getattr(p, k) for k, _ in p._fields_ if k != "name"} | {"name": p.name.decode()}

    def __call__(self, A, B, offsets, *, D, bias=None, scale_a=None, scale_b=None, U=None, Z=None, stream=None):
        ptr = self._ptr
        a, b, o, bs, sa, sb, u, d, z = self._specs
        code = self._run(self.handle, ptr(A, a), ptr(B, b), ptr(offsets, o), ptr(bias, bs), ptr(scale_a, sa),
                         ptr(scale_b, sb), ptr(U, u), ptr(D, d), ptr(Z, z), self._stream(stream)[0])
        if code:
            _check(code, "gemm_epi_expert_linear_run")
        return D


class ExpertLinearGrad(_ExpertPlan):
    """The gradients of ``ExpertLinear`` without scales.

    g = dD * U, dZ = g * act'(Z), dU = dD * act(Z), dA[r] = dZ[r] . B[e], and over
    every expert's rows dB[e] = dB_in[e] + dZ^T . A, dbias[e] = the column sums of
    dZ.  All tensors are packed; dD, Z, U, dZ, dU, A and B have type ab (f16 or
    bf16).  da, db, dbias: the gradients' types, None for one not wanted.
    Without an activation and mul dD takes dZ's place and Z and dZ are not given.
    With db the whole of A and of dZ must be below 2 GiB each; a larger batch is several
    calls, each on a range of rows with ``offsets`` less its first row and dB_in = the dB
    before (dbias adds up).
    tile (64, 128 or 256) forces the products' tile.
    """

    _op = "expert_linear_grad"

    def __init__(self, rows, experts, N, K, *, ab="bf16", act="none", mul=False, da=None, db=None, dbias=None, tile=0):
        super().__init__(gemm_epi_expert_linear_grad_desc(
            rows, N, K, experts, _code(DTYPES, ab, "type"), _code(ACTIVATIONS, act, "activation"), int(mul),
            _code(DTYPES, da, "type"), _code(DTYPES, db, "type"), _code(DTYPES, dbias, "type"), tile))
        ab = TORCH_DTYPES[ab]
        da, db, dbias = (TORCH_DTYPES[t] if t else None for t in (da, db, dbias))
        m, E = self._matrix, experts
        w = (N * K, K, 1)
        self._specs = (m("dD", ab, rows, N, N), m("A", ab, rows, K, K), ("B", ab, (E, N, K), w),
                       self._vector("offsets", torch.int32, E + 1), m("Z", ab, rows, N, N), m("U", ab, rows, N, N),
                       ("dB_in", db, (E, N, K), w), m("dZ", ab, rows, N, N), m("dU", ab, rows, N, N),
                       m("dA", da, rows, K, K), ("dB", db, (E, N, K), w), m("dbias", dbias, E, N, N))
        self._wants = (da is not None, db is not None)
        self.workspace_bytes = lib().gemm_epi_expert_linear_grad_workspace(self.handle)

    def __call__(self, dD, A, B, offsets, *, Z=None, U=None, dB_in=None, dZ=None, dU=None, dA=None, dB=None,
                 dbias=None, stream=None, workspace=None):
        ptr = self._ptr
        sd, sa, sb, so, sz, su, sc, gz, gu, ga, gb, gs = self._specs
        wants_a, wants_b = self._wants
        raw, s = self._stream(stream)
        ws, nbytes, keep = self._workspace(self.workspace_bytes, workspace, s)
        # (an operand that the wanted gradients do not need is not passed on)
        code = self._run(self.handle, ptr(dD, sd), ptr(A if wants_b else None, sa), ptr(B if wants_a else None, sb),
                         ptr(offsets, so), ptr(Z, sz), ptr(U, su), ptr(dB_in, sc), ptr(dZ, gz), ptr(dU, gu),
                         ptr(dA, ga), ptr(dB, gb), ptr(dbias, gs), ws, nbytes, raw)
        if code:
            _check(code, "gemm_epi_expert_linear_grad_run")
