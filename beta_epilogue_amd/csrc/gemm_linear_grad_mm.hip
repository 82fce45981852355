// gemm_linear_grad_mm.hip -- the two matrix products of the linear layer's
// backward in one launch, compiled once per type and kernel
// (GEMM_LINEAR_GRAD_PART 0 .. 7).
//
// dA = dZ . B and dB = dB_in + dZ^T . A read what the elementwise pass left
// and do not depend on one another, so their tiles (and K slices) share a
// grid: the second product's workgroups start as soon as compute units are
// free instead of behind the first one's last round, and small problems fill
// the chip together; the one with the longer items goes first (1812 x 560 x
// 3824 bf16: 34.7 us with dA's 450 tiles of 9 K tiles first, 27.2 with dB's 150
// of 29).  The column sums of dZ (of the elementwise pass's chunks,
// or without an activation of dD's rows) are made by further workgroups of
// the same launch.  Both products read the weights and
// activations as they lie: dA has B's columns contiguous (N-major), dB both
// operands' rows (M-major, N-major), through the transposing LDS reads.
#include "gemm_linear.hpp"

#ifndef GEMM_LINEAR_GRAD_PART
#error "GEMM_LINEAR_GRAD_PART must be defined (0 .. 7)"
#endif

namespace gemm_epi {

namespace {

// 64 columns per workgroup of 256 threads: 8 lanes of 8 columns by 32 strands
// of rows, joined in a fixed order.  red: 32 x 68 words.
template <int AB>
__device__ __forceinline__ void colsum_rows_block(const uint16_t* x, int64_t P, int64_t C, void* out, int t,
                                                  int64_t block, float* red) {
  const int cl = threadIdx.x & 7, pl = threadIdx.x >> 3;
  const int64_t c = block * 64 + cl * 8;
  float s[8] = {};
  if (c < C) {
#pragma unroll 8
    for (int64_t r = pl; r < P; r += 32) {
      const v4u w = *(const v4u*)(x + r * C + c);
      const v4f lo = epi_dec<AB>(w, 0), hi = epi_dec<AB>(w, 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += lo[k], s[4 + k] += hi[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) red[pl * 68 + cl * 8 + k] = s[k];
  __syncthreads();
  const int64_t n = block * 64 + threadIdx.x;
  if (threadIdx.x >= 64 || n >= C) return;
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; ++k) v += red[k * 68 + threadIdx.x];
  store_as(out, n, t, v);
}

template <int AB, int KIND>
__global__ __launch_bounds__(256, grad_occ(KIND)) void linear_grad_mm_kernel(GradParams p) {
  using CA = GradCfg<AB, true, KIND>;
  using CB = GradCfg<AB, false, KIND>;
  __shared__ __attribute__((aligned(1024))) char lds[CA::LDS_BYTES > CB::LDS_BYTES ? CA::LDS_BYTES : CB::LDS_BYTES];
  const int bid = blockIdx.x, a0 = p.b_first ? p.gb : 0, b0 = p.b_first ? 0 : p.ga;
  if (bid >= a0 && bid < a0 + p.ga) gemm_epi_body<CA>(p.a, lds, bid - a0, p.ga);
  else if (bid < p.ga + p.gb) gemm_epi_body<CB>(p.b, lds, bid - b0, p.gb);
  else if (p.partial) colsum_block<8>(p.partial, p.P, p.C, p.dbias, p.dbias_dtype, bid - p.ga - p.gb, (float*)lds);
  else colsum_rows_block<AB>((const uint16_t*)p.rows, p.P, p.C, p.dbias, p.dbias_dtype, bid - p.ga - p.gb, (float*)lds);
}

}  // namespace

constexpr int kAb = GEMM_LINEAR_GRAD_PART % 2 ? T_BF16 : T_F16, kKind = GEMM_LINEAR_GRAD_PART / 2;

template <>
void launch_linear_grad_mm<kAb, kKind>(const GradParams& p, hipStream_t s) {
  const int64_t sums = p.partial ? (p.C + 31) / 32 : p.rows ? (p.C + 63) / 64 : 0;
  hipLaunchKernelGGL((linear_grad_mm_kernel<kAb, kKind>), dim3((unsigned)(p.ga + p.gb + sums)), dim3(256), 0, s, p);
}

}  // namespace gemm_epi
