// gemm_grouped_part.hip -- compiles the tile kernels of
// gemm_grouped_variants.inc whose `part` equals GEMM_GROUPED_PART (the build
// compiles this file once per part, in parallel).
#include "gemm_grouped.hpp"

#ifndef GEMM_GROUPED_PART
#error "GEMM_GROUPED_PART must be defined (0 .. 6)"
#endif

namespace gemm_epi {

namespace {
template <class CF>
__global__ __launch_bounds__(CF::THREADS, CF::OCC) void grouped_kernel(GroupParams p) {
  __shared__ __attribute__((aligned(1024))) char lds[CF::LDS_BYTES + kGroupTableBytes];
  gemm_epi_body<CF>(p, lds, blockIdx.x, gridDim.x);
}

template <int PART, class CF>
void launch_if(bool wanted, const GroupParams& p, int grid, hipStream_t s) {
  if constexpr (PART == GEMM_GROUPED_PART) {
    if (wanted) hipLaunchKernelGGL(grouped_kernel<CF>, dim3(grid), dim3(CF::THREADS), 0, s, p);
  }
}
}  // namespace

template <>
void launch_grouped_part<GEMM_GROUPED_PART>(int variant, const GroupParams& p, int grid, hipStream_t s) {
  int i = 0;
#define X(PART, AB, BM, BN, S, OCC, BL, NAME) launch_if<PART, GroupedCfg<AB, BM, BN, S, OCC, BL>>(variant == i++, p, grid, s);
#include "gemm_grouped_variants.inc"
#undef X
}

}  // namespace gemm_epi
