"""The linear layer's and the norm's entry points without a GPU: exports,
static validation before any device query, and the host-side refusals."""
import ctypes
import os
import re

import pytest
import torch

import beta_epilogue_amd as ge
from beta_epilogue_amd import layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OK, INVALID, UNSUPPORTED, ALIGN, DEVICE = (ge.GEMM_EPI_OK, ge.GEMM_EPI_ERR_INVALID_ARG, ge.GEMM_EPI_ERR_UNSUPPORTED,
                                           ge.GEMM_EPI_ERR_ALIGNMENT, ge.GEMM_EPI_ERR_DEVICE)


@pytest.mark.parametrize("header", ["gemm_epi_linear.h", "gemm_epi_norm.h"])
def test_exports(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_epi_\w+)\s*\(", text)))
    assert len(names) >= 7
    lib = ctypes.CDLL(ge.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), "missing export " + n


@pytest.mark.parametrize("header", ["gemm_epi_linear.h", "gemm_epi_norm.h"])
def test_headers_are_c(header, tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "%s"\nint main(void) { return 0; }\n' % header)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                   check=True)


def _create(op, desc, **fields):
    d = desc()
    for k, v in fields.items():
        setattr(d, k, v)
    h = ctypes.c_void_p(99)
    rc = getattr(layers.lib(), "gemm_epi_%s_create" % op)(ctypes.byref(d), ctypes.byref(h))
    if rc == OK:
        getattr(layers.lib(), "gemm_epi_%s_destroy" % op)(h)
    else:
        assert h.value is None and ge.last_error()
    return rc


T = ge.DTYPES
LINEAR = dict(M=100, N=256, K=512, ab_dtype=T["bf16"], d_dtype=T["bf16"])
LINEAR_BAD = [
    (dict(M=0), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID),
    (dict(ab_dtype=0), INVALID), (dict(ab_dtype=T["f32"]), INVALID), (dict(ab_dtype=99), INVALID),
    (dict(ab_dtype=T["e5m2"]), UNSUPPORTED), (dict(ab_dtype=T["u8"]), UNSUPPORTED),
    (dict(d_dtype=T["i32"]), INVALID), (dict(d_dtype=T["e4m3"]), INVALID), (dict(d_dtype=0), INVALID),
    (dict(bias_dtype=T["i8"]), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(residual=2), INVALID), (dict(z=-1), INVALID), (dict(scale_a=3), INVALID), (dict(splits=-1), INVALID),
    (dict(K=516), ALIGN), (dict(N=252), ALIGN), (dict(ab_dtype=T["e4m3"], K=520), ALIGN),
    (dict(lda=500), INVALID), (dict(lda=516), ALIGN), (dict(ldb=-8), INVALID), (dict(ldd=260), ALIGN),
    (dict(ldr=256), INVALID), (dict(ldz=256), INVALID), (dict(residual=1, ldr=255), INVALID),
    (dict(lda=1 << 40), UNSUPPORTED), (dict(K=1 << 40), UNSUPPORTED), (dict(N=1 << 40), UNSUPPORTED),
    (dict(M=1 << 40), UNSUPPORTED), (dict(ldd=1 << 62), UNSUPPORTED), (dict(M=(1 << 63) - 1), UNSUPPORTED),
    (dict(ab_dtype=T["i8"], K=1 << 17), UNSUPPORTED),  # 2^17 products of up to 2^14 in an int32
]


@pytest.mark.parametrize("bad,code", LINEAR_BAD, ids=[str(b[0]) for b in LINEAR_BAD])
def test_linear_validation(bad, code):
    assert _create("linear", layers.gemm_epi_linear_desc, **(LINEAR | bad)) == code, ge.last_error()


GRAD = dict(M=100, N=256, K=512, ab_dtype=T["bf16"], da_dtype=T["bf16"], db_dtype=T["f32"], dbias_dtype=T["f32"])
GRAD_BAD = [
    (dict(M=0), INVALID), (dict(K=-5), INVALID), (dict(ab_dtype=0), INVALID), (dict(ab_dtype=T["e4m3"]), UNSUPPORTED),
    (dict(act=9), INVALID), (dict(da_dtype=T["i32"]), INVALID), (dict(dbias_dtype=T["e4m3"]), INVALID),
    (dict(da_dtype=0, db_dtype=0, dbias_dtype=0), INVALID), (dict(N=250), ALIGN), (dict(K=500, N=256), ALIGN),
    (dict(M=1 << 62), UNSUPPORTED), (dict(N=1 << 40, da_dtype=0, db_dtype=0), UNSUPPORTED),
    (dict(tile=32), INVALID), (dict(splits=-2), INVALID), (dict(K=1 << 22), UNSUPPORTED),
    (dict(M=1 << 20, N=1 << 12), UNSUPPORTED),  # an operand of 2 GiB or more
    (dict(N=(1 << 26) + 8, da_dtype=0, db_dtype=0), UNSUPPORTED),  # more threads than a launch has
]


@pytest.mark.parametrize("bad,code", GRAD_BAD, ids=[str(b[0]) for b in GRAD_BAD])
def test_linear_grad_validation(bad, code):
    assert _create("linear_grad", layers.gemm_epi_linear_grad_desc, **(GRAD | bad)) == code, ge.last_error()


NORM = dict(rows=4, cols=100, x_dtype=T["bf16"], y_dtype=T["e4m3"], weight_dtype=T["bf16"], eps=1e-6)
NORM_BAD = [
    (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(cols=16385), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(x_dtype=0), INVALID), (dict(x_dtype=T["i8"]), UNSUPPORTED), (dict(weight_dtype=T["f16"]), UNSUPPORTED),
    (dict(ldx=99), INVALID), (dict(ldx=-100), INVALID), (dict(ldx=1 << 62), INVALID),
]


@pytest.mark.parametrize("bad,code", NORM_BAD + [
    (dict(y_dtype=T["f16"]), UNSUPPORTED), (dict(y_dtype=T["e5m2"]), UNSUPPORTED), (dict(y_dtype=17), INVALID),
    (dict(residual=2), INVALID), (dict(ldr=100), INVALID), (dict(ldh=100), INVALID)], ids=lambda v: str(v))
def test_rmsnorm_validation(bad, code):
    assert _create("rmsnorm", layers.gemm_epi_rmsnorm_desc, **(NORM | bad)) == code, ge.last_error()


@pytest.mark.parametrize("bad,code", [(({"ldy": 99} if "ldx" in b else b), c) for b, c in NORM_BAD] + [
    (dict(dweight_dtype=T["i32"]), INVALID)], ids=lambda v: str(v))
def test_rmsnorm_grad_validation(bad, code):
    good = {k: v for k, v in NORM.items() if k != "y_dtype"}
    assert _create("rmsnorm_grad", layers.gemm_epi_rmsnorm_grad_desc, **(good | bad)) == code, ge.last_error()


def test_valid_problems_stop_at_the_device():
    """With no GPU every valid problem passes validation and ends at the device
    query, never on another path."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for more in ({}, dict(M=1), dict(ab_dtype=T["e4m3"], d_dtype=T["f32"], scale_a=1, scale_b=1), dict(lda=520, ldd=264),
                 dict(residual=1, ldr=264, z=1, ldz=512, act=4, bias_dtype=T["f16"], splits=3)):
        assert _create("linear", layers.gemm_epi_linear_desc, **(LINEAR | more)) == DEVICE
    assert _create("linear_grad", layers.gemm_epi_linear_grad_desc, **GRAD) == DEVICE
    assert _create("linear_grad", layers.gemm_epi_linear_grad_desc, **(GRAD | dict(da_dtype=0, db_dtype=0))) == DEVICE
    assert _create("rmsnorm", layers.gemm_epi_rmsnorm_desc, **(NORM | dict(residual=1, ldr=101))) == DEVICE
    assert _create("rmsnorm_grad", layers.gemm_epi_rmsnorm_grad_desc,
                   **{k: v for k, v in NORM.items() if k != "y_dtype"}) == DEVICE


def test_null_arguments():
    L = layers.lib()
    h = ctypes.c_void_p()
    for op in ("linear", "linear_grad", "rmsnorm", "rmsnorm_grad"):
        assert getattr(L, "gemm_epi_%s_create" % op)(None, ctypes.byref(h)) == INVALID
        assert getattr(L, "gemm_epi_%s_destroy" % op)(None) == OK
    assert L.gemm_epi_linear_create(ctypes.byref(layers.gemm_epi_linear_desc()), None) == INVALID
    assert L.gemm_epi_linear_run(None, 16, 16, None, None, None, None, 16, None, 1.0, None, 0, None) == INVALID
    assert L.gemm_epi_linear_grad_run(None, 16, 16, 16, None, None, None, 16, 16, None, None, 0, None) == INVALID
    assert L.gemm_epi_rmsnorm_run(None, 16, None, 16, 16, None, None, None) == INVALID
    assert L.gemm_epi_rmsnorm_grad_run(None, 16, 16, 16, None, 16, None, None, 0, None) == INVALID
    assert L.gemm_epi_linear_get_plan(None, ctypes.byref(ge.gemm_epi_plan())) == INVALID
    assert L.gemm_epi_linear_grad_workspace(None) == -1 and L.gemm_epi_rmsnorm_grad_workspace(None) == -1


NAMES = 20


def test_variant_table():
    names = ge.linear_variant_names()
    assert len(set(names)) == len(names) == NAMES and names[-1] == "linear_rows"
    assert layers.lib().gemm_epi_linear_variant_name(-1) is None
    assert layers.lib().gemm_epi_linear_variant_name(NAMES) is None
    d = layers.gemm_epi_linear_desc(**LINEAR)
    h = ctypes.c_void_p()
    create = layers.lib().gemm_epi_linear_create_variant
    assert create(ctypes.byref(d), NAMES, ctypes.byref(h)) == INVALID
    assert create(ctypes.byref(d), names.index("linear_f16_256x256"), ctypes.byref(h)) == UNSUPPORTED
    assert create(ctypes.byref(d), names.index("linear_rows"), ctypes.byref(h)) == UNSUPPORTED  # 100 rows


def test_unknown_names_are_refused():
    with pytest.raises(ValueError):
        ge.FusedLinear(1, 8, 8, ab="f64")
    with pytest.raises(ValueError):
        ge.FusedLinear(1, 8, 8, act="swish")
    with pytest.raises(ValueError):
        ge.FusedNormLinear(1, 16, 16, q="bf16")
