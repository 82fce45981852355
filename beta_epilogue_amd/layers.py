"""Thin Python binding of the linear layer and the norm
(include/gemm_epi_linear.h, include/gemm_epi_norm.h).

As in the package's ``FusedGemm``, a plan object holds a handle for one
problem shape and its call marshals torch tensors: data pointers and the
current stream go to the C entry points, nothing is computed in Python.
Tensors are checked against the plan (device, type, shape and strides).  A
plan's workspace is allocated per call from torch's caching allocator on the
call's stream, so calls on different streams and captured graphs never share
one; ``workspace=`` passes a uint8 tensor of the caller's instead.
"""
from __future__ import annotations

import ctypes
import torch

from . import DTYPES, _check, gemm_epi_plan
from . import lib as _load

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
TORCH_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
                "e4m3": torch.float8_e4m3fn, "i8": torch.int8}

_i64, _i32, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class gemm_epi_linear_desc(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("lda", _i64), ("ldb", _i64), ("ldd", _i64),
                ("ldr", _i64), ("ldz", _i64), ("ab_dtype", _i32), ("d_dtype", _i32), ("bias_dtype", _i32),
                ("act", _i32), ("residual", _i32), ("z", _i32), ("scale_a", _i32), ("scale_b", _i32),
                ("splits", _i32)]


class gemm_epi_linear_grad_desc(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("ab_dtype", _i32), ("act", _i32), ("da_dtype", _i32),
                ("db_dtype", _i32), ("dbias_dtype", _i32)]


class gemm_epi_rmsnorm_desc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("ldx", _i64), ("ldr", _i64), ("ldh", _i64), ("ldy", _i64),
                ("x_dtype", _i32), ("y_dtype", _i32), ("weight_dtype", _i32), ("residual", _i32), ("eps", _f32)]


class gemm_epi_rmsnorm_grad_desc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("ldy", _i64), ("ldh", _i64), ("ldi", _i64), ("ldo", _i64),
                ("x_dtype", _i32), ("weight_dtype", _i32), ("dweight_dtype", _i32), ("eps", _f32)]


_bound = None


def lib():
    """The loaded shared library, with this module's entry points declared."""
    global _bound
    if _bound is None:
        L = _load()
        _bind(L)
        _bound = L
    return _bound


def _bind(L):
    """Argument types of the entry points."""
    P, I, N = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    for op, desc in (("linear", gemm_epi_linear_desc), ("linear_grad", gemm_epi_linear_grad_desc),
                     ("rmsnorm", gemm_epi_rmsnorm_desc), ("rmsnorm_grad", gemm_epi_rmsnorm_grad_desc)):
        create, destroy = getattr(L, "gemm_epi_%s_create" % op), getattr(L, "gemm_epi_%s_destroy" % op)
        create.argtypes, create.restype = [ctypes.POINTER(desc), ctypes.POINTER(P)], I
        destroy.argtypes, destroy.restype = [P], I
    L.gemm_epi_linear_create_variant.argtypes = [ctypes.POINTER(gemm_epi_linear_desc), I, ctypes.POINTER(P)]
    L.gemm_epi_linear_create_variant.restype = I
    L.gemm_epi_linear_run.argtypes = [P] * 9 + [_f32, P, N, P]
    L.gemm_epi_linear_grad_run.argtypes = [P] * 11 + [N, P]
    L.gemm_epi_rmsnorm_run.argtypes = [P] * 8
    L.gemm_epi_rmsnorm_grad_run.argtypes = [P] * 8 + [N, P]
    for op in ("linear", "linear_grad", "rmsnorm", "rmsnorm_grad"):
        getattr(L, "gemm_epi_%s_run" % op).restype = I
    L.gemm_epi_linear_get_plan.argtypes = [P, ctypes.POINTER(gemm_epi_plan)]
    L.gemm_epi_linear_get_plan.restype = I
    L.gemm_epi_linear_variant_count.argtypes, L.gemm_epi_linear_variant_count.restype = [], I
    L.gemm_epi_linear_variant_name.argtypes, L.gemm_epi_linear_variant_name.restype = [I], ctypes.c_char_p
    for op in ("linear_grad", "rmsnorm_grad"):
        f = getattr(L, "gemm_epi_%s_workspace" % op)
        f.argtypes, f.restype = [P], N


def linear_variant_names() -> list:
    """Names of the linear layer's kernels, by variant number."""
    return [lib().gemm_epi_linear_variant_name(i).decode() for i in range(lib().gemm_epi_linear_variant_count())]


class _Plan:
    """A handle of one shape; subclasses set _op and call it."""

    _op = ""

    def __init__(self, desc, variant=-1):
        self.handle = None
        self.desc = desc
        h = ctypes.c_void_p()
        if variant == -1:
            where = "gemm_epi_%s_create" % self._op
            _check(getattr(lib(), where)(ctypes.byref(desc), ctypes.byref(h)), where)
        else:
            where = "gemm_epi_%s_create_variant" % self._op
            _check(getattr(lib(), where)(ctypes.byref(desc), variant, ctypes.byref(h)), where)
        self.handle = h.value
        self.device = torch.cuda.current_device()
        self._run = getattr(lib(), "gemm_epi_%s_run" % self._op)

    def _ptr(self, name, t, dtype, rows, cols, ld):
        """The data pointer of a tensor that fits the plan (None: absent).
        rows 0: a vector of cols values."""
        if t is None:
            return None
        if t.device.type != "cuda" or t.device.index != self.device:
            raise ValueError("%s is on %s, the plan on cuda:%d" % (name, t.device, self.device))
        if t.dtype is not dtype:
            raise ValueError("%s has type %s, the plan %s" % (name, t.dtype, dtype))
        if rows == 0:
            if t.shape != (cols,) or (cols > 1 and t.stride(0) != 1):
                raise ValueError("%s must be a packed vector of %d values" % (name, cols))
        elif t.shape != (rows, cols) or (rows > 1 and t.stride(0) != ld) or (cols > 1 and t.stride(1) != 1):
            raise ValueError("%s must be %d x %d with row stride %d: got %s with strides %s"
                             % (name, rows, cols, ld, tuple(t.shape), t.stride()))
        return t.data_ptr()

    def _stream(self, stream):
        """The hipStream_t of a call, and the stream (None: the current one)."""
        if stream is None:
            return torch.cuda.current_stream().cuda_stream, None
        if hasattr(stream, "cuda_stream"):
            if stream.device.index != self.device:
                raise ValueError("the stream is on %s, the plan on cuda:%d" % (stream.device, self.device))
            return stream.cuda_stream, stream
        return stream, torch.cuda.ExternalStream(stream or 0)

    def _workspace(self, nbytes, workspace, stream):
        """Pointer, size and owner of a call's workspace."""
        if workspace is not None:
            if workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or \
                    workspace.device.type != "cuda" or workspace.device.index != self.device:
                raise ValueError("workspace must be a packed uint8 tensor on cuda:%d" % self.device)
            return workspace.data_ptr(), workspace.numel(), workspace
        if nbytes == 0:
            return None, 0, None
        return self._scratch(nbytes, torch.uint8, stream)

    def _scratch(self, n, dtype, stream):
        """n values of scratch memory that belongs to the call's stream."""
        if stream is None:
            t = torch.empty(n, dtype=dtype, device=self._dev())
        else:
            with torch.cuda.stream(stream):
                t = torch.empty(n, dtype=dtype, device=self._dev())
        return t.data_ptr(), t.numel() * t.element_size(), t

    def _dev(self):
        return torch.device("cuda", self.device)

    def close(self):
        if self.handle:
            getattr(lib(), "gemm_epi_%s_destroy" % self._op)(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _code(table, key, what):
    if key not in table:
        raise ValueError("unknown %s %r (one of %s)" % (what, key, ", ".join(str(k) for k in table if k)))
    return table[key]


class FusedLinear(_Plan):
    """D = act(alpha * scale_a[m] * scale_b[n] * (A . B^T) + bias) + residual.

    A is M x K, B (the weight) N x K, D, residual and Z M x N, all row-major;
    lda .. ldz are row strides in elements (0: packed).  ab: f16, bf16, e4m3 or
    i8; d (of D, residual and Z): f16, bf16 or f32.  bias: its type, or None;
    residual, z, scale_a, scale_b: whether the call has them.  Z receives the
    pre-activation, which ``FusedLinearGrad`` takes.  M of at most 64 runs the
    few-row kernel.  variant and splits force a kernel and a K split.
    """

    _op = "linear"

    def __init__(self, M, N, K, *, ab="bf16", d=None, act="none", bias=None, residual=False, z=False,
                 scale_a=False, scale_b=False, lda=0, ldb=0, ldd=0, ldr=0, ldz=0, splits=0, variant=-1):
        d = d or (ab if ab in ("f16", "bf16") else "bf16")
        super().__init__(gemm_epi_linear_desc(
            M, N, K, lda, ldb, ldd, ldr, ldz, _code(DTYPES, ab, "type"), _code(DTYPES, d, "type"),
            _code(DTYPES, bias, "type"), _code(ACTIVATIONS, act, "activation"), int(residual), int(z),
            int(scale_a), int(scale_b), splits), variant)
        self._ab, self._d = TORCH_DTYPES[ab], TORCH_DTYPES[d]
        self._bias = TORCH_DTYPES[bias] if bias else None
        self._mnk = (M, N, K)
        self._ld = (lda or K, ldb or K, ldd or N, ldr or N, ldz or N)
        self._ws = self.plan["workspace_bytes"]

    @property
    def plan(self) -> dict:
        p = gemm_epi_plan()
        _check(lib().gemm_epi_linear_get_plan(self.handle, ctypes.byref(p)), "gemm_epi_linear_get_plan")
        return {k: getattr(p, k) for k, _ in p._fields_ if k != "name"} | {"name": p.name.decode()}

    def __call__(self, A, B, *, D, bias=None, scale_a=None, scale_b=None, residual=None, Z=None, alpha=1.0,
                 stream=None, workspace=None):
        M, N, K = self._mnk
        lda, ldb, ldd, ldr, ldz = self._ld
        ptr, d, f32 = self._ptr, self._d, torch.float32
        raw, s = self._stream(stream)
        ws, nbytes, keep = self._workspace(self._ws, workspace, s)
        _check(self._run(self.handle, ptr("A", A, self._ab, M, K, lda), ptr("B", B, self._ab, N, K, ldb),
                         ptr("bias", bias, self._bias, 0, N, 0), ptr("scale_a", scale_a, f32, 0, M, 0),
                         ptr("scale_b", scale_b, f32, 0, N, 0), ptr("residual", residual, d, M, N, ldr),
                         ptr("D", D, d, M, N, ldd), ptr("Z", Z, d, M, N, ldz), alpha, ws, nbytes, raw),
               "gemm_epi_linear_run")
        return D


class FusedLinearGrad(_Plan):
    """The gradients of a linear layer.

    dZ = dD * act'(Z), dA = dZ . B, dB = dB_in + dZ^T . A, dbias = the column
    sums of dZ.  All tensors are packed; dD, Z, dZ, A and B have type ab (f16
    or bf16).  da, db, dbias: the gradients' types, None for one not wanted.
    Without an activation dD takes dZ's place and Z and dZ are not given.  The
    residual's gradient is dD.
    """

    _op = "linear_grad"

    def __init__(self, M, N, K, *, ab="bf16", act="none", da=None, db=None, dbias=None):
        super().__init__(gemm_epi_linear_grad_desc(
            M, N, K, _code(DTYPES, ab, "type"), _code(ACTIVATIONS, act, "activation"), _code(DTYPES, da, "type"),
            _code(DTYPES, db, "type"), _code(DTYPES, dbias, "type")))
        self._ab, self._mnk = TORCH_DTYPES[ab], (M, N, K)
        self._t = tuple(TORCH_DTYPES[t] if t else None for t in (da, db, dbias))
        self.workspace_bytes = lib().gemm_epi_linear_grad_workspace(self.handle)

    def __call__(self, dD, A=None, B=None, *, Z=None, dB_in=None, dZ=None, dA=None, dB=None, dbias=None,
                 stream=None, workspace=None):
        M, N, K = self._mnk
        ptr, ab = self._ptr, self._ab
        da_t, db_t, dbias_t = self._t
        raw, s = self._stream(stream)
        ws, nbytes, keep = self._workspace(self.workspace_bytes, workspace, s)
        # (an operand that the wanted gradients do not need is not passed on)
        _check(self._run(self.handle, ptr("dD", dD, ab, M, N, N), ptr("A", A if db_t else None, ab, M, K, K),
                         ptr("B", B if da_t else None, ab, N, K, K), ptr("Z", Z, ab, M, N, N),
                         ptr("dB_in", dB_in, db_t, N, K, K), ptr("dZ", dZ, ab, M, N, N),
                         ptr("dA", dA, da_t, M, K, K), ptr("dB", dB, db_t, N, K, K),
                         ptr("dbias", dbias, dbias_t, 0, N, 0), ws, nbytes, raw), "gemm_epi_linear_grad_run")


class RmsNorm(_Plan):
    """Y = h / sqrt(mean(h^2) + eps) * weight, h = x + residual.

    x (of x, residual and H): f16, bf16 or f32; y: the same type, or e4m3 or i8
    with one fp32 scale per row (the linear layer's scale_a); weight: x's type
    or f32.  H, if given, receives h rounded.  ldx .. ldy: row strides in
    elements (0: packed); at most 16384 columns.
    """

    _op = "rmsnorm"

    def __init__(self, rows, cols, *, x="bf16", y=None, weight=None, residual=False, eps=1e-6, ldx=0, ldr=0, ldh=0,
                 ldy=0):
        y, weight = y or x, weight or x
        super().__init__(gemm_epi_rmsnorm_desc(rows, cols, ldx, ldr, ldh, ldy, _code(DTYPES, x, "type"),
                                               _code(DTYPES, y, "type"), _code(DTYPES, weight, "type"),
                                               int(residual), eps))
        self._t = (TORCH_DTYPES[x], TORCH_DTYPES[y], TORCH_DTYPES[weight])
        self._shape = (rows, cols)
        self._ld = (ldx or cols, ldr or cols, ldh or cols, ldy or cols)

    def __call__(self, x, weight, *, Y, residual=None, H=None, scale=None, stream=None):
        R, C = self._shape
        ldx, ldr, ldh, ldy = self._ld
        xt, yt, wt = self._t
        ptr = self._ptr
        raw, _ = self._stream(stream)
        _check(self._run(self.handle, ptr("x", x, xt, R, C, ldx), ptr("residual", residual, xt, R, C, ldr),
                         ptr("weight", weight, wt, 0, C, 0), ptr("Y", Y, yt, R, C, ldy), ptr("H", H, xt, R, C, ldh),
                         ptr("scale", scale, torch.float32, 0, R, 0), raw), "gemm_epi_rmsnorm_run")
        return Y


class RmsNormGrad(_Plan):
    """The gradients of the norm: dH (of x and of the residual alike, with
    dH_in, the gradient that reaches h by other ways, added) and dweight.

    x: the type of dY, H, dH_in and dH; dweight: its type, None if not wanted.
    """

    _op = "rmsnorm_grad"

    def __init__(self, rows, cols, *, x="bf16", weight=None, dweight="f32", eps=1e-6, ldy=0, ldh=0, ldi=0, ldo=0):
        weight = weight or x
        super().__init__(gemm_epi_rmsnorm_grad_desc(rows, cols, ldy, ldh, ldi, ldo, _code(DTYPES, x, "type"),
                                                    _code(DTYPES, weight, "type"), _code(DTYPES, dweight, "type"),
                                                    eps))
        self._t = (TORCH_DTYPES[x], TORCH_DTYPES[weight], TORCH_DTYPES[dweight] if dweight else None)
        self._shape = (rows, cols)
        self._ld = (ldy or cols, ldh or cols, ldi or cols, ldo or cols)
        self.workspace_bytes = lib().gemm_epi_rmsnorm_grad_workspace(self.handle)

    def __call__(self, dY, H, weight, *, dH, dH_in=None, dweight=None, stream=None, workspace=None):
        R, C = self._shape
        ldy, ldh, ldi, ldo = self._ld
        xt, wt, dwt = self._t
        ptr = self._ptr
        raw, s = self._stream(stream)
        ws, nbytes, keep = self._workspace(self.workspace_bytes, workspace, s)
        _check(self._run(self.handle, ptr("dY", dY, xt, R, C, ldy), ptr("H", H, xt, R, C, ldh),
                         ptr("weight", weight, wt, 0, C, 0), ptr("dH_in", dH_in, xt, R, C, ldi),
                         ptr("dH", dH, xt, R, C, ldo), ptr("dweight", dweight, dwt, 0, C, 0), ws, nbytes, raw),
               "gemm_epi_rmsnorm_grad_run")
        return dH


class FusedNormLinear:
    """A pre-norm projection in 8 bits: ``RmsNorm`` of x (+ residual) into an
    8-bit operand with row scales, then ``FusedLinear`` of it.

    x: f16, bf16 or f32 (M x K); q: e4m3 or i8, the type of the norm's output
    and of B, whose column scales are scale_b.  H (if given) receives x +
    residual; the linear layer's own residual is ``add``.
    """

    def __init__(self, M, N, K, *, x="bf16", q="e4m3", d="bf16", weight=None, act="none", bias=None, residual=False,
                 add=False, eps=1e-6):
        if q not in ("e4m3", "i8"):
            raise ValueError("q must be e4m3 or i8")
        self.norm = RmsNorm(M, K, x=x, y=q, weight=weight, residual=residual, eps=eps)
        self.linear = FusedLinear(M, N, K, ab=q, d=d, act=act, bias=bias, residual=add, scale_a=True, scale_b=True)
        self._mk, self._q = (M, K), TORCH_DTYPES[q]

    def __call__(self, x, weight, B, scale_b, *, D, residual=None, H=None, bias=None, add=None, stream=None):
        M, K = self._mk
        _, s = self.norm._stream(stream)
        _, _, q = self.norm._scratch(M * K, torch.uint8, s)
        _, _, scale = self.norm._scratch(M, torch.float32, s)
        q = q.view(self._q).view(M, K)
        self.norm(x, weight, Y=q, residual=residual, H=H, scale=scale, stream=stream)
        return self.linear(q, B, D=D, bias=bias, scale_a=scale, scale_b=scale_b, residual=add, stream=stream)

    def close(self):
        self.norm.close()
        self.linear.close()
