// gemm_linear_grad_mm.hip -- the two matrix products of the linear layer's
// backward in one launch, compiled once per type and kernel
// (GEMM_LINEAR_GRAD_PART 0 .. 5).
//
// dA = dZ . B and dB = dB_in + dZ^T . A read what the elementwise pass left
// and do not depend on one another, so their tiles (and K slices) share a
// grid: the second product's workgroups start as soon as compute units are
// free instead of behind the first one's last round, and small problems fill
// the chip together.  The chunks' column sums of dZ are added by further
// workgroups of the same launch.  Both products read the weights and
// activations as they lie: dA has B's columns contiguous (N-major), dB both
// operands' rows (M-major, N-major), through the transposing LDS reads.
#include "gemm_linear.hpp"

#ifndef GEMM_LINEAR_GRAD_PART
#error "GEMM_LINEAR_GRAD_PART must be defined (0 .. 5)"
#endif

namespace gemm_epi {

namespace {

template <int AB, int KIND>
__global__ __launch_bounds__(256, grad_occ(KIND)) void linear_grad_mm_kernel(GradParams p) {
  using CA = GradCfg<AB, true, KIND>;
  using CB = GradCfg<AB, false, KIND>;
  __shared__ __attribute__((aligned(1024))) char lds[CA::LDS_BYTES > CB::LDS_BYTES ? CA::LDS_BYTES : CB::LDS_BYTES];
  const int bid = blockIdx.x;
  if (bid < p.ga) gemm_epi_body<CA>(p.a, lds, bid, p.ga);
  else if (bid < p.ga + p.gb) gemm_epi_body<CB>(p.b, lds, bid - p.ga, p.gb);
  else colsum_block<8>(p.partial, p.P, p.C, p.dbias, p.dbias_dtype, bid - p.ga - p.gb, (float*)lds);
}

}  // namespace

constexpr int kAb = GEMM_LINEAR_GRAD_PART % 2 ? T_BF16 : T_F16, kKind = GEMM_LINEAR_GRAD_PART / 2;

template <>
void launch_linear_grad_mm<kAb, kKind>(const GradParams& p, hipStream_t s) {
  const int64_t sums = p.partial ? (p.C + 31) / 32 : 0;
  hipLaunchKernelGGL((linear_grad_mm_kernel<kAb, kKind>), dim3((unsigned)(p.ga + p.gb + sums)), dim3(256), 0, s, p);
}

}  // namespace gemm_epi
