// gemm_linear_part.hip -- compiles the linear layer's tile kernels of
// gemm_linear_variants.inc whose `part` equals GEMM_LINEAR_PART (the build
// compiles this file once per part, in parallel).
#include "gemm_linear.hpp"

#ifndef GEMM_LINEAR_PART
#error "GEMM_LINEAR_PART must be defined (0 .. 7)"
#endif

namespace gemm_epi {

namespace {
template <int PART, class CF>
void launch_if(bool wanted, const LinParams& p, int grid, hipStream_t s) {
  if constexpr (PART == GEMM_LINEAR_PART) {
    if (wanted) hipLaunchKernelGGL(gemm_epi_kernel<CF>, dim3(grid), dim3(CF::THREADS), 0, s, p);
  }
}
}  // namespace

template <>
void launch_linear_part<GEMM_LINEAR_PART>(int variant, const LinParams& p, int grid, hipStream_t s) {
  int i = 0;
#define X(PART, AB, BM, BN, S, OCC, BL, NAME) launch_if<PART, LinearCfg<AB, BM, BN, S, OCC, BL>>(variant == i++, p, grid, s);
#include "gemm_linear_variants.inc"
#undef X
}

}  // namespace gemm_epi
