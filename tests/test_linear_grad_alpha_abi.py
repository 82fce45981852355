"""gemm_epi_linear_grad_run_alpha without a GPU."""
import beta_epilogue_amd as ge
from beta_epilogue_amd import layers


def test_null_handle():
    run = layers.lib().gemm_epi_linear_grad_run_alpha
    assert run(None, 16, 16, 16, None, None, None, 16, 16, None, 0.5, None, 0, None) == ge.GEMM_EPI_ERR_INVALID_ARG
    assert "handle" in ge.last_error()
