// gemm_linear_grad.hip -- the linear layer's backward outside its two matrix
// products (gemm_linear_grad_mm.hip):
//   dZ = dD * act'(Z), rounded to the operands' type (the MFMA reads it), and
//   dbias[n] = sum over m of dZ[m][n], summed in fp32 before that rounding.
// One pass reads dD and Z and writes dZ, with the column sums on the way:
// every workgroup sums the rows of its chunk and leaves one partial sum per
// column, and a second kernel adds the chunks in a fixed order, so the result
// does not depend on the order in which workgroups run.
#include "gemm_linear.hpp"

namespace gemm_epi {

namespace {

template <int T>
__device__ __forceinline__ void decode8(v4u r, float (&v)[8]) {
  const v4f lo = epi_dec<T>(r, 0), hi = epi_dec<T>(r, 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
}

// A workgroup: 256 columns (32 lanes of 8) by `chunk` rows, 8 rows at a time.
// HAS_Z: dZ is computed and stored; else dZ is dD and only summed.
template <int T, bool HAS_Z>
__global__ __launch_bounds__(256) void linear_dact_kernel(const uint16_t* dD, const uint16_t* Z, uint16_t* dZ,
                                                          float* partial, void* dbias, int dbias_dtype, int64_t M,
                                                          int64_t N, int chunk, int act) {
  __shared__ float red[8][256 + 4];
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 256 + cl * 8;
  const int64_t m0 = (int64_t)blockIdx.y * chunk, m1 = min(m0 + chunk, M);
  float sum[8] = {};
  if (c < N) {
    with_act(HAS_Z ? act : ACT_NONE, [&](auto act_c) {
#pragma unroll 4
      for (int64_t m = m0 + rl; m < m1; m += 8) {
        const int64_t i = m * N + c;
        float d[8];
        decode8<T>(__builtin_nontemporal_load((const v4u*)(dD + i)), d);
        if constexpr (HAS_Z) {
          float z[8];
          decode8<T>(__builtin_nontemporal_load((const v4u*)(Z + i)), z);
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k] *= act_slope<decltype(act_c)::value>(z[k]);
          *(v4u*)(dZ + i) = epi_pack<T>(v4f{d[0], d[1], d[2], d[3]}, v4f{d[4], d[5], d[6], d[7]});
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += d[k];
      }
    });
  }
  if (!partial && !dbias) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) red[rl][cl * 8 + k] = sum[k];
  __syncthreads();
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += red[k][threadIdx.x];
  if (partial) partial[(int64_t)blockIdx.y * N + n] = s;
  else store_as(dbias, n, dbias_dtype, s);
}

__global__ __launch_bounds__(1024) void colsum_kernel(const float* partial, int64_t P, int64_t C, void* out, int t) {
  __shared__ float red[32 * 33];
  colsum_block<32>(partial, P, C, out, t, blockIdx.x, red);
}

template <int T>
void dact(int act, const void* dD, const void* Z, void* dZ, float* partial, void* dbias, int dbias_dtype, int64_t M,
          int64_t N, int chunk, hipStream_t s) {
  const dim3 grid((unsigned)((N + 255) / 256), (unsigned)((M + chunk - 1) / chunk));
  if (act != ACT_NONE)
    hipLaunchKernelGGL((linear_dact_kernel<T, true>), grid, dim3(256), 0, s, (const uint16_t*)dD, (const uint16_t*)Z,
                       (uint16_t*)dZ, partial, dbias, dbias_dtype, M, N, chunk, act);
  else
    hipLaunchKernelGGL((linear_dact_kernel<T, false>), grid, dim3(256), 0, s, (const uint16_t*)dD, nullptr, nullptr,
                       partial, dbias, dbias_dtype, M, N, chunk, act);
}

}  // namespace

void launch_linear_dact(int t, int act, const void* dD, const void* Z, void* dZ, float* partial, void* dbias,
                        int dbias_dtype, int64_t M, int64_t N, int chunk, hipStream_t s) {
  if (t == T_F16) dact<T_F16>(act, dD, Z, dZ, partial, dbias, dbias_dtype, M, N, chunk, s);
  else dact<T_BF16>(act, dD, Z, dZ, partial, dbias, dbias_dtype, M, N, chunk, s);
}

void launch_colsum(const float* partial, int64_t P, int64_t C, void* out, int t, hipStream_t s) {
  hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((C + 31) / 32)), dim3(1024), 0, s, partial, P, C, out, t);
}

}  // namespace gemm_epi
