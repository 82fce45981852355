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

from . import DTYPES, GEMM_EPI_ERR_ALIGNMENT, GEMM_EPI_ERR_INVALID_ARG, GemmEpiError, _check, gemm_epi_plan
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
                ("db_dtype", _i32), ("dbias_dtype", _i32), ("tile", _i32), ("splits", _i32)]


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
    L.gemm_epi_linear_grad_run_alpha.argtypes = [P] * 10 + [_f32, P, N, P]
    L.gemm_epi_linear_grad_run_alpha.restype = I
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


# The current stream's hipStream_t.  torch's own raw accessor where there is
# one: 0.1 us, against 2.5 us for a torch.cuda.Stream object, of a call's 6 us.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


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
        self._device = torch.device("cuda", self.device)
        self._run = getattr(lib(), "gemm_epi_%s_run" % self._op)

    @staticmethod
    def _matrix(name, dtype, rows, cols, ld):
        """What a tensor argument has to be: name, type, shape and strides."""
        return name, dtype, (rows, cols), (ld, 1)

    @staticmethod
    def _vector(name, dtype, n):
        return name, dtype, (n,), (1,)

    def _ptr(self, t, spec):
        """The data pointer of a tensor that fits the plan (None: absent)."""
        if t is None:
            return None
        _, dtype, shape, strides = spec
        if t.get_device() == self.device and t.dtype is dtype and t.shape == shape and t.stride() == strides:
            return t.data_ptr()
        return self._ptr_or_raise(t, *spec)

    def _ptr_or_raise(self, t, name, dtype, shape, strides):
        if t.device.type != "cuda" or t.device.index != self.device:
            raise ValueError("%s is on %s, the plan on cuda:%d" % (name, t.device, self.device))
        if t.dtype is not dtype:
            raise ValueError("%s has type %s, the plan %s" % (name, t.dtype, dtype))
        # (the stride of an extent of one has no meaning)
        if t.shape != shape or any(n > 1 and got != want for n, got, want in zip(shape, t.stride(), strides)):
            raise ValueError("%s must have shape %s with strides %s: got %s with strides %s"
                             % (name, shape, strides, tuple(t.shape), t.stride()))
        return t.data_ptr()

    def _stream(self, stream):
        """The hipStream_t of a call, and the stream (None: the current one)."""
        if stream is None:
            return _current_stream(self.device), None
        if hasattr(stream, "cuda_stream"):
            if stream.device.index != self.device:
                raise ValueError("the stream is on %s, the plan on cuda:%d" % (stream.device, self.device))
            return stream.cuda_stream, stream
        return stream, torch.cuda.ExternalStream(stream or 0, device=self._device)

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
            t = torch.empty(n, dtype=dtype, device=self._device)
        else:
            with torch.cuda.stream(stream):
                t = torch.empty(n, dtype=dtype, device=self._device)
        return t.data_ptr(), t.numel() * t.element_size(), t

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
    pre-activation, which ``FusedLinearGrad`` takes (with the same alpha; it has
    no scales).  Few rows (decoding) run a kernel of their own.  variant and
    splits force a kernel and a K split.
    """

    _op = "linear"

    def __init__(self, M, N, K, *, ab="bf16", d=None, act="none", bias=None, residual=False, z=False,
                 scale_a=False, scale_b=False, lda=0, ldb=0, ldd=0, ldr=0, ldz=0, splits=0, variant=-1):
        d = d or (ab if ab in ("f16", "bf16") else "bf16")
        super().__init__(gemm_epi_linear_desc(
            M, N, K, lda, ldb, ldd, ldr, ldz, _code(DTYPES, ab, "type"), _code(DTYPES, d, "type"),
            _code(DTYPES, bias, "type"), _code(ACTIVATIONS, act, "activation"), int(residual), int(z),
            int(scale_a), int(scale_b), splits), variant)
        ab, d, bias = TORCH_DTYPES[ab], TORCH_DTYPES[d], TORCH_DTYPES[bias] if bias else None
        m, v = self._matrix, self._vector
        self._specs = (m("A", ab, M, K, lda or K), m("B", ab, N, K, ldb or K), v("bias", bias, N),
                       v("scale_a", torch.float32, M), v("scale_b", torch.float32, N),
                       m("residual", d, M, N, ldr or N), m("D", d, M, N, ldd or N), m("Z", d, M, N, ldz or N))
        self._ws = self.plan["workspace_bytes"]

    @property
    def plan(self) -> dict:
        p = gemm_epi_plan()
        _check(lib().gemm_epi_linear_get_plan(self.handle, ctypes.byref(p)), "gemm_epi_linear_get_plan")
        return {k: getattr(p, k) for k, _ in p._fields_ if k != "name"} | {"name": p.name.decode()}

    def __call__(self, A, B, *, D, bias=None, scale_a=None, scale_b=None, residual=None, Z=None, alpha=1.0,
                 stream=None, workspace=None):
        ptr = self._ptr
        a, b, bs, sa, sb, r, d, z = self._specs
        raw, s = self._stream(stream)
        ws, nbytes, keep = self._workspace(self._ws, workspace, s)
        code = self._run(self.handle, ptr(A, a), ptr(B, b), ptr(bias, bs), ptr(scale_a, sa), ptr(scale_b, sb),
                         ptr(residual, r), ptr(D, d), ptr(Z, z), alpha, ws, nbytes, raw)
        if code:
            _check(code, "gemm_epi_linear_run")
        return D


class FusedLinearGrad(_Plan):
    """The gradients of a linear layer.

    dZ = dD * act'(Z), dA = alpha dZ . B, dB = dB_in + alpha dZ^T . A, dbias =
    the column sums of dZ, for a forward of this alpha without scales.  All
    tensors are packed; dD, Z, dZ, A and B have type ab (f16 or bf16).  da, db,
    dbias: the gradients' types, None for one not wanted.  Without an activation
    dD takes dZ's place and Z and dZ are not given.  The residual's gradient is
    dD.  tile (64, 128 or 256) and splits force the products' tile and K split.
    """

    _op = "linear_grad"

    def __init__(self, M, N, K, *, ab="bf16", act="none", da=None, db=None, dbias=None, tile=0, splits=0):
        super().__init__(gemm_epi_linear_grad_desc(
            M, N, K, _code(DTYPES, ab, "type"), _code(ACTIVATIONS, act, "activation"), _code(DTYPES, da, "type"),
            _code(DTYPES, db, "type"), _code(DTYPES, dbias, "type"), tile, splits))
        ab = TORCH_DTYPES[ab]
        da, db, dbias = (TORCH_DTYPES[t] if t else None for t in (da, db, dbias))
        m, v = self._matrix, self._vector
        self._specs = (m("dD", ab, M, N, N), m("A", ab, M, K, K), m("B", ab, N, K, K), m("Z", ab, M, N, N),
                       m("dB_in", db, N, K, K), m("dZ", ab, M, N, N), m("dA", da, M, K, K), m("dB", db, N, K, K),
                       v("dbias", dbias, N))
        self._wants = (da is not None, db is not None)
        self._run = lib().gemm_epi_linear_grad_run_alpha
        self.workspace_bytes = lib().gemm_epi_linear_grad_workspace(self.handle)

    def __call__(self, dD, A=None, B=None, *, Z=None, dB_in=None, dZ=None, dA=None, dB=None, dbias=None,
                 alpha=1.0, stream=None, workspace=None):
        ptr = self._ptr
        g, a, b, z, c, gz, ga, gb, gbias = self._specs
        wants_a, wants_b = self._wants
        raw, s = self._stream(stream)
        ws, nbytes, keep = self._workspace(self.workspace_bytes, workspace, s)
        # (an operand that the wanted gradients do not need is not passed on)
        code = self._run(self.handle, ptr(dD, g), ptr(A if wants_b else None, a), ptr(B if wants_a else None, b),
                         ptr(Z, z), ptr(dB_in, c), ptr(dZ, gz), ptr(dA, ga), ptr(dB, gb), ptr(dbias, gbias), alpha,
                         ws, nbytes, raw)
        if code:
            _check(code, "gemm_epi_linear_grad_run_alpha")


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
        x, m = TORCH_DTYPES[x], self._matrix
        self._specs = (m("x", x, rows, cols, ldx or cols), m("residual", x, rows, cols, ldr or cols),
                       self._vector("weight", TORCH_DTYPES[weight], cols),
                       m("Y", TORCH_DTYPES[y], rows, cols, ldy or cols), m("H", x, rows, cols, ldh or cols),
                       self._vector("scale", torch.float32, rows))

    def __call__(self, x, weight, *, Y, residual=None, H=None, scale=None, stream=None):
        ptr = self._ptr
        sx, sr, sw, sy, sh, ss = self._specs
        code = self._run(self.handle, ptr(x, sx), ptr(residual, sr), ptr(weight, sw), ptr(Y, sy), ptr(H, sh),
                         ptr(scale, ss), self._stream(stream)[0])
        if code:
            _check(code, "gemm_epi_rmsnorm_run")
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
        x, m = TORCH_DTYPES[x], self._matrix
        self._specs = (m("dY", x, rows, cols, ldy or cols), m("H", x, rows, cols, ldh or cols),
                       self._vector("weight", TORCH_DTYPES[weight], cols), m("dH_in", x, rows, cols, ldi or cols),
                       m("dH", x, rows, cols, ldo or cols),
                       self._vector("dweight", TORCH_DTYPES[dweight] if dweight else None, cols))
        self.workspace_bytes = lib().gemm_epi_rmsnorm_grad_workspace(self.handle)

    def __call__(self, dY, H, weight, *, dH, dH_in=None, dweight=None, stream=None, workspace=None):
        ptr = self._ptr
        sy, sh, sw, si, so, sd = self._specs
        raw, s = self._stream(stream)
        ws, nbytes, keep = self._workspace(self.workspace_bytes, workspace, s)
        code = self._run(self.handle, ptr(dY, sy), ptr(H, sh), ptr(weight, sw), ptr(dH_in, si), ptr(dH, so),
                         ptr(dweight, sd), ws, nbytes, raw)
        if code:
            _check(code, "gemm_epi_rmsnorm_grad_run")
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
        self._bias, self._add = bias is not None, bool(add)
        self._scale_at = (M * K + 255) // 256 * 256
        self._scratch_bytes = self._scale_at + 4 * M

    def __call__(self, x, weight, B, scale_b, *, D, residual=None, H=None, bias=None, add=None, stream=None):
        norm, linear = self.norm, self.linear
        # what the projection would refuse, before the norm writes H
        ptr = linear._ptr
        _, sb, sbias, _, sscale, sadd, sd, _ = linear._specs
        b, bs, sc, r, d = ptr(B, sb), ptr(bias, sbias), ptr(scale_b, sscale), ptr(add, sadd), ptr(D, sd)
        if b is None or d is None or sc is None or (bs is None) == self._bias or (r is None) == self._add:
            self._refuse(GEMM_EPI_ERR_INVALID_ARG, "B, D and scale_b are required; bias and add as the plan says")
        if (b | d | sc | (bs or 0) | (r or 0)) & 15:
            self._refuse(GEMM_EPI_ERR_ALIGNMENT, "a tensor is not 16-byte aligned")
        if d in (b, bs, sc):
            self._refuse(GEMM_EPI_ERR_INVALID_ARG, "D may not be an operand")
        raw, s = norm._stream(stream)
        q, _, keep = norm._scratch(self._scratch_bytes, torch.uint8, s)  # the operand, then its row scales
        scale = q + self._scale_at
        sx, sr, sw, _, sh, _ = norm._specs
        code = norm._run(norm.handle, ptr(x, sx), ptr(residual, sr), ptr(weight, sw), q, ptr(H, sh), scale, raw)
        if code:
            _check(code, "gemm_epi_rmsnorm_run")
        ws, nbytes, keep_ws = linear._workspace(linear._ws, None, s)
        code = linear._run(linear.handle, q, b, bs, scale, sc, r, d, None, 1.0, ws, nbytes, raw)
        if code:
            _check(code, "gemm_epi_linear_run")
        return D

    @staticmethod
    def _refuse(code, text):
        raise GemmEpiError(code, "gemm_epi_linear_run", text)

    def close(self):
        self.norm.close()
        self.linear.close()
