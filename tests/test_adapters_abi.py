"""The adapters' entry points without a GPU: exports, static validation before
any device query, and the host-side refusals."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import beta_epilogue_amd as ge
from beta_epilogue_amd import adapters, layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = "gemm_epi_adapters.h"
OK, INVALID, UNSUPPORTED, ALIGN, DEVICE = (ge.GEMM_EPI_OK, ge.GEMM_EPI_ERR_INVALID_ARG, ge.GEMM_EPI_ERR_UNSUPPORTED,
                                           ge.GEMM_EPI_ERR_ALIGNMENT, ge.GEMM_EPI_ERR_DEVICE)
T = ge.DTYPES


def test_exports():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", HEADER)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_epi_\w+)\s*\(", text)))
    assert len(names) >= 5
    lib = ctypes.CDLL(ge.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), "missing export " + n


def test_header_is_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "%s"\nint main(void) { return 0; }\n' % HEADER)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                   check=True)


def _create(rank=16, count=4, **fields):
    d = adapters.gemm_epi_adapter_linear_desc(rank=rank, adapters=count)
    good = dict(M=100, N=256, K=512, ab_dtype=T["bf16"], d_dtype=T["bf16"])
    for k, v in (good | fields).items():
        setattr(d.linear, k, v)
    h = ctypes.c_void_p(99)
    rc = adapters.lib().gemm_epi_adapter_linear_create(ctypes.byref(d), ctypes.byref(h))
    if rc == OK:
        adapters.lib().gemm_epi_adapter_linear_destroy(h)
    else:
        assert h.value is None and ge.last_error()
    return rc


BAD = [
    (dict(rank=0), INVALID), (dict(rank=-8), INVALID), (dict(rank=12), ALIGN), (dict(rank=136), UNSUPPORTED),
    (dict(count=0), INVALID), (dict(count=1025), UNSUPPORTED), (dict(M=1 << 26), UNSUPPORTED), (dict(count=-1), INVALID), (dict(M=0), INVALID), (dict(N=-8), INVALID), (dict(K=0), INVALID),
    (dict(ab_dtype=T["e4m3"]), UNSUPPORTED), (dict(ab_dtype=T["i8"]), UNSUPPORTED), (dict(ab_dtype=0), INVALID),
    (dict(ab_dtype=99), INVALID), (dict(d_dtype=T["f32"]), UNSUPPORTED), (dict(d_dtype=T["f16"]), UNSUPPORTED),
    (dict(scale_a=1), UNSUPPORTED), (dict(scale_b=1), UNSUPPORTED), (dict(act=7), INVALID), (dict(bias_dtype=T["i8"]), INVALID),
    (dict(residual=2), INVALID), (dict(K=516), ALIGN), (dict(N=252), ALIGN), (dict(lda=500), INVALID), (dict(ldr=256), INVALID),
    (dict(K=1 << 40), UNSUPPORTED), (dict(N=1 << 40), UNSUPPORTED), (dict(N=1 << 23), UNSUPPORTED), (dict(M=1 << 40), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", BAD, ids=lambda v: str(v))
def test_validation(bad, code):
    assert _create(**bad) == code, ge.last_error()


def test_valid_problems_stop_at_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for more in ({}, dict(M=1, rank=8, count=1), dict(rank=128, count=1024), dict(ab_dtype=T["f16"], d_dtype=T["f16"], act=4),
                 dict(residual=1, ldr=264, z=1, lda=520, ldd=256, bias_dtype=T["f32"], splits=2)):
        assert _create(**more) == DEVICE, ge.last_error()


def test_null_arguments():
    L, h = adapters.lib(), ctypes.c_void_p()
    assert L.gemm_epi_adapter_linear_create(None, ctypes.byref(h)) == INVALID
    assert L.gemm_epi_adapter_linear_create(ctypes.byref(adapters.gemm_epi_adapter_linear_desc()), None) == INVALID
    assert L.gemm_epi_adapter_linear_destroy(None) == OK
    assert L.gemm_epi_adapter_linear_run(None, 16, 16, 16, 16, 16, 16, None, None, 16, None, None, 0, None) == INVALID
    assert L.gemm_epi_adapter_linear_get_plan(None, ctypes.byref(ge.gemm_epi_plan())) == INVALID


def test_unknown_names_are_refused():
    with pytest.raises(ValueError):
        ge.AdapterLinear(1, 8, 8, 8, 1, ab="f64")
    with pytest.raises(ValueError):
        ge.AdapterLinear(1, 8, 8, 8, 1, act="swish")
    assert layers.ACTIVATIONS["silu"] == 4
