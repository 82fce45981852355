// gemm_adapter_part.hip -- compiles the linear layer's tile kernels with
// adapters (gemm_adapter.hpp); GEMM_ADAPTER_PART 0 .. 3: one shape of tile each.
// 4001 x 4096 x 4096 bf16, rank 64, 7 adapters: 110 us, with the sort (6) and the inner
// products (16) before it 130 (the projection by itself 95 to 101).
#include "gemm_adapter.hpp"

#ifndef GEMM_ADAPTER_PART
#error "GEMM_ADAPTER_PART must be defined (0 .. 3)"
#endif

namespace gemm_epi {

namespace {

// The shapes, stages and workgroups per compute unit of gemm_linear_variants.inc.
constexpr int kBm[] = {256, 192, 128, 64}, kBn[] = {256, 256, 128, 64}, kStages[] = {2, 2, 2, 4}, kOcc[] = {1, 1, 2, 2};
constexpr int P = GEMM_ADAPTER_PART;

template <class CF>
__global__ __launch_bounds__(CF::THREADS, CF::OCC) void adapter_kernel(AdapterParams p) {
  __shared__ __attribute__((aligned(1024))) char lds[CF::LDS_BYTES + AdapterTiles<CF>::LDS_BYTES];
  gemm_epi_body<CF>(p, lds, blockIdx.x, gridDim.x);
}

}  // namespace

template <>
void launch_adapter_part<P>(int ab, int bm, const AdapterParams& p, int grid, hipStream_t s) {
  if (bm != kBm[P]) return;
  using F = AdapterCfg<T_F16, kBm[P], kBn[P], kStages[P], kOcc[P]>;
  using B = AdapterCfg<T_BF16, kBm[P], kBn[P], kStages[P], kOcc[P]>;
  if (ab == T_F16) hipLaunchKernelGGL(adapter_kernel<F>, dim3(grid), dim3(F::THREADS), 0, s, p);
  else hipLaunchKernelGGL(adapter_kernel<B>, dim3(grid), dim3(B::THREADS), 0, s, p);
}

}  // namespace gemm_epi
