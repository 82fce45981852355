"""The experts' entry points without a GPU: exports, static validation before
any device query, and the host-side refusals."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import beta_epilogue_amd as ge
from beta_epilogue_amd import experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = "gemm_epi_experts.h"
OK, INVALID, UNSUPPORTED, ALIGN, DEVICE = (ge.GEMM_EPI_OK, ge.GEMM_EPI_ERR_INVALID_ARG, ge.GEMM_EPI_ERR_UNSUPPORTED,
                                           ge.GEMM_EPI_ERR_ALIGNMENT, ge.GEMM_EPI_ERR_DEVICE)
T = ge.DTYPES


def test_exports():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", HEADER)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_epi_\w+)\s*\(", text)))
    assert len(names) >= 10
    lib = ctypes.CDLL(ge.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), "missing export " + n


def test_header_is_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "%s"\nint main(void) { return 0; }\n' % HEADER)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                   check=True)


def _create(op, **fields):
    d = getattr(experts, "gemm_epi_%s_desc" % op)()
    for k, v in fields.items():
        setattr(d, k, v)
    h = ctypes.c_void_p(99)
    rc = getattr(experts.lib(), "gemm_epi_%s_create" % op)(ctypes.byref(d), ctypes.byref(h))
    if rc == OK:
        getattr(experts.lib(), "gemm_epi_%s_destroy" % op)(h)
    else:
        assert h.value is None and ge.last_error()
    return rc


SORT = dict(tokens=10, cols=64, top_k=2, experts=8, ids_bits=64, x_dtype=T["bf16"])
SORT_BAD = [
    (dict(tokens=0), INVALID), (dict(tokens=-3), INVALID), (dict(top_k=0), INVALID), (dict(top_k=65), INVALID),
    (dict(experts=0), INVALID), (dict(experts=1025), INVALID), (dict(ids_bits=16), INVALID), (dict(cols=-8), INVALID),
    (dict(scale=2), INVALID), (dict(x_dtype=0), INVALID), (dict(x_dtype=99), INVALID),
    (dict(x_dtype=T["u8"]), UNSUPPORTED), (dict(x_dtype=T["i32"]), UNSUPPORTED), (dict(cols=60), ALIGN),
    (dict(cols=0), INVALID), (dict(cols=0, x_dtype=0, scale=1), INVALID), (dict(cols=0, x_dtype=0, ldx=8), INVALID),
    (dict(ldx=56), INVALID), (dict(ldx=68), ALIGN), (dict(ldy=-64), INVALID), (dict(ldy=1 << 62), INVALID),
    (dict(ldy=1 << 60), INVALID), (dict(cols=1 << 40), UNSUPPORTED), (dict(tokens=1 << 25), UNSUPPORTED),
    (dict(tokens=(1 << 63) - 1), UNSUPPORTED), (dict(tokens=1 << 24, cols=8192), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", SORT_BAD, ids=lambda v: str(v))
def test_sort_validation(bad, code):
    assert _create("expert_sort", **(SORT | bad)) == code, ge.last_error()


COMBINE = dict(tokens=10, cols=64, top_k=2, x_dtype=T["bf16"], weights=1)
COMBINE_BAD = [
    (dict(tokens=0), INVALID), (dict(cols=0), INVALID), (dict(top_k=0), INVALID), (dict(top_k=100), INVALID),
    (dict(x_dtype=0), INVALID), (dict(x_dtype=T["e4m3"]), UNSUPPORTED), (dict(cols=4), ALIGN), (dict(ldy=12), INVALID),
    (dict(ldd=68), ALIGN), (dict(tokens=1 << 30), UNSUPPORTED), (dict(tokens=1 << 40), UNSUPPORTED),
    (dict(ldy=1 << 60), INVALID), (dict(tokens=1 << 28, cols=256), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", COMBINE_BAD + [(dict(weights=2), INVALID), (dict(residual=-1), INVALID),
                                                    (dict(ldr=64), INVALID)], ids=lambda v: str(v))
def test_combine_validation(bad, code):
    assert _create("expert_combine", **(COMBINE | bad)) == code, ge.last_error()


@pytest.mark.parametrize("bad,code", COMBINE_BAD + [(dict(ldg=8), INVALID), (dict(tokens=1 << 27, top_k=1), UNSUPPORTED)],
                         ids=lambda v: str(v))
def test_combine_grad_validation(bad, code):
    good = {k: v for k, v in COMBINE.items() if k != "weights"}
    assert _create("expert_combine_grad", **(good | bad)) == code, ge.last_error()


LINEAR = dict(rows=100, experts=8, N=256, K=512, ab_dtype=T["bf16"], d_dtype=T["bf16"])
LINEAR_BAD = [
    (dict(rows=0), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(experts=0), INVALID),
    (dict(experts=1025), INVALID), (dict(ab_dtype=0), INVALID), (dict(ab_dtype=T["f32"]), INVALID),
    (dict(ab_dtype=T["e5m2"]), UNSUPPORTED), (dict(ab_dtype=T["u8"]), UNSUPPORTED), (dict(d_dtype=T["i32"]), INVALID),
    (dict(d_dtype=0), INVALID), (dict(bias_dtype=T["i8"]), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(mul=2), INVALID), (dict(z=-1), INVALID), (dict(scale_a=3), INVALID), (dict(scale_b=-1), INVALID),
    (dict(K=516), ALIGN), (dict(N=252), ALIGN), (dict(ab_dtype=T["e4m3"], K=520), ALIGN), (dict(lda=500), INVALID),
    (dict(lda=516), ALIGN), (dict(ldd=260), ALIGN), (dict(ldu=256), INVALID), (dict(ldz=256), INVALID),
    (dict(N=260, d_dtype=T["f32"], bias_dtype=T["f16"]), ALIGN),
    (dict(lda=1 << 40), UNSUPPORTED), (dict(K=1 << 40), UNSUPPORTED), (dict(N=1 << 40), UNSUPPORTED),
    (dict(rows=1 << 40), UNSUPPORTED), (dict(rows=(1 << 63) - 1), UNSUPPORTED), (dict(ab_dtype=T["i8"], K=1 << 17), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", LINEAR_BAD, ids=lambda v: str(v))
def test_linear_validation(bad, code):
    assert _create("expert_linear", **(LINEAR | bad)) == code, ge.last_error()


GRAD = dict(rows=100, experts=8, N=256, K=512, ab_dtype=T["bf16"], da_dtype=T["bf16"], db_dtype=T["f32"],
            dbias_dtype=T["f32"])
GRAD_BAD = [
    (dict(rows=0), INVALID), (dict(K=-5), INVALID), (dict(experts=2000), INVALID), (dict(ab_dtype=0), INVALID),
    (dict(ab_dtype=T["e4m3"]), UNSUPPORTED), (dict(act=9), INVALID), (dict(mul=-1), INVALID),
    (dict(da_dtype=T["i32"]), INVALID), (dict(dbias_dtype=T["e4m3"]), INVALID),
    (dict(da_dtype=0, db_dtype=0, dbias_dtype=0), INVALID), (dict(N=250), ALIGN), (dict(K=500), ALIGN),
    (dict(tile=32), INVALID), (dict(rows=1 << 62), UNSUPPORTED), (dict(K=1 << 22), UNSUPPORTED),
    (dict(rows=1 << 22), UNSUPPORTED),  # A of 2 GiB or more
]


@pytest.mark.parametrize("bad,code", GRAD_BAD, ids=lambda v: str(v))
def test_linear_grad_validation(bad, code):
    assert _create("expert_linear_grad", **(GRAD | bad)) == code, ge.last_error()


def test_linear_variants():
    names = ge.expert_linear_variant_names()
    assert len(set(names)) == len(names) and names[-1] == "experts_rows16"
    L = experts.lib()
    assert L.gemm_epi_expert_linear_variant_name(-1) is None
    assert L.gemm_epi_expert_linear_variant_name(len(names)) is None
    d, h = experts.gemm_epi_expert_linear_desc(**LINEAR), ctypes.c_void_p()
    create = L.gemm_epi_expert_linear_create_variant
    assert create(ctypes.byref(d), len(names), ctypes.byref(h)) == INVALID
    assert create(ctypes.byref(d), names.index("experts_f16_256x256"), ctypes.byref(h)) == UNSUPPORTED
    d.rows = 1 << 20  # more chunks of four rows than a launch's second dimension has
    assert create(ctypes.byref(d), names.index("experts_rows4"), ctypes.byref(h)) == UNSUPPORTED


def test_valid_problems_stop_at_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for more in ({}, dict(tokens=1, top_k=1, experts=1), dict(cols=0, x_dtype=0), dict(ids_bits=32, ldx=72, ldy=128),
                 dict(x_dtype=T["e4m3"], scale=1), dict(tokens=1 << 20, top_k=8, experts=1024, x_dtype=T["f32"])):
        assert _create("expert_sort", **(SORT | more)) == DEVICE, ge.last_error()
    assert _create("expert_combine", **(COMBINE | dict(residual=1, ldr=128))) == DEVICE
    for more in ({}, dict(rows=1), dict(ab_dtype=T["e4m3"], d_dtype=T["f32"], scale_a=1, scale_b=1),
                 dict(lda=520, ldd=264, mul=1, ldu=264, z=1, act=4, bias_dtype=T["f16"])):
        assert _create("expert_linear", **(LINEAR | more)) == DEVICE, ge.last_error()
    assert _create("expert_linear_grad", **GRAD) == DEVICE
    assert _create("expert_linear_grad", **(GRAD | dict(da_dtype=0, db_dtype=0, dbias_dtype=0, mul=1))) == DEVICE
    assert _create("expert_combine_grad", **{k: v for k, v in COMBINE.items() if k != "weights"}) == DEVICE


def test_null_arguments():
    L = experts.lib()
    h = ctypes.c_void_p()
    for op in experts._DESCS:
        assert getattr(L, "gemm_epi_%s_create" % op)(None, ctypes.byref(h)) == INVALID
        desc = getattr(experts, "gemm_epi_%s_desc" % op)()
        assert getattr(L, "gemm_epi_%s_create" % op)(ctypes.byref(desc), None) == INVALID
        assert getattr(L, "gemm_epi_%s_destroy" % op)(None) == OK
    assert L.gemm_epi_expert_sort_run(None, 16, 16, None, 16, 16, 16, None, None, 0, None) == INVALID
    assert L.gemm_epi_expert_combine_run(None, 16, 16, None, None, 16, None) == INVALID
    assert L.gemm_epi_expert_combine_grad_run(None, 16, 16, 16, 16, 16, 16, None) == INVALID
    assert L.gemm_epi_expert_linear_run(None, 16, 16, 16, None, None, None, None, 16, None, None) == INVALID
    assert L.gemm_epi_expert_linear_grad_run(None, 16, 16, 16, 16, None, None, None, None, None, 16, 16, None, None, 0,
                                             None) == INVALID
    assert L.gemm_epi_expert_linear_get_plan(None, ctypes.byref(ge.gemm_epi_plan())) == INVALID
    assert L.gemm_epi_expert_sort_workspace(None) == -1 and L.gemm_epi_expert_linear_grad_workspace(None) == -1


def test_unknown_names_are_refused():
    with pytest.raises(ValueError):
        ge.ExpertSort(4, 2, 8, ids="i8")
    with pytest.raises(ValueError):
        ge.ExpertSort(4, 2, 8, cols=64, x="f64")
    with pytest.raises(ValueError):
        ge.ExpertCombine(4, 2, 64, x="f64")
