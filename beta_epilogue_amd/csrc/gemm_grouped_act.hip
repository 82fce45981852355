// gemm_grouped_act.hip -- the elementwise pass of the experts' backward:
//   g = dD * U,  dZ = g * act'(Z),  dU = dD * act(Z)
// each rounded once to the operands' type (the matrix cores read dZ), and the
// column sums of dZ before that rounding, one partial sum per chunk of an
// expert's rows.  Bound by memory: every row of the batch is read and written
// once, rows behind the last expert's not at all (16384 x 4096 bf16 with U, 671 MB
// in 126 us, 5.3 TB/s).
#include "gemm_grouped.hpp"

namespace gemm_epi {

namespace {

template <int T>
__device__ __forceinline__ void decode8(v4u r, float (&v)[8]) {
  const v4f lo = epi_dec<T>(r, 0), hi = epi_dec<T>(r, 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
}

template <int T>
__device__ __forceinline__ v4u pack8(const float (&v)[8]) {
  return epi_pack<T>(v4f{v[0], v[1], v[2], v[3]}, v4f{v[4], v[5], v[6], v[7]});
}

// A workgroup: 256 columns (32 lanes of 8) by a chunk's rows, 8 at a time.
template <int T, bool HAS_Z, bool MUL>
__global__ __launch_bounds__(256) void grouped_act_kernel(GroupActParams p) {
  __shared__ float red[8][256 + 4];
  const GroupTile t = group_chunk(p, blockIdx.y, p.chunk);
  if (t.group < 0) return;
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t N = p.N, c = (int64_t)blockIdx.x * 256 + cl * 8;
  float sum[8] = {};
  if (c < N) {
    with_act(HAS_Z ? p.act : ACT_NONE, [&](auto act_c) {
      constexpr int ACT = decltype(act_c)::value;
#pragma unroll 4
      for (int m = t.begin + rl; m < t.end; m += 8) {
        const int64_t i = m * N + c;
        float d[8];
        decode8<T>(__builtin_nontemporal_load((const v4u*)((const uint16_t*)p.dD + i)), d);
        if constexpr (HAS_Z) {
          float z[8], g[8];
          decode8<T>(__builtin_nontemporal_load((const v4u*)((const uint16_t*)p.dZin + i)), z);
          if constexpr (MUL) {
            float u[8];
            decode8<T>(__builtin_nontemporal_load((const v4u*)((const uint16_t*)p.U + i)), u);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              g[k] = d[k] * act_value<ACT>(z[k]);
              d[k] *= u[k];
            }
            __builtin_nontemporal_store(pack8<T>(g), (v4u*)((uint16_t*)p.dU + i));
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k] *= act_slope<ACT>(z[k]);
          *(v4u*)((uint16_t*)p.dZ + i) = pack8<T>(d);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += d[k];
      }
    });
  }
  if (!p.partial) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) red[rl][cl * 8 + k] = sum[k];
  __syncthreads();
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += red[k][threadIdx.x];
  p.partial[(int64_t)blockIdx.y * N + n] = s;
}

template <int T>
void act(const GroupActParams& p, int slots, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 255) / 256), (unsigned)slots);
  if (p.U) hipLaunchKernelGGL((grouped_act_kernel<T, true, true>), grid, dim3(256), 0, s, p);
  else if (p.dZin) hipLaunchKernelGGL((grouped_act_kernel<T, true, false>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((grouped_act_kernel<T, false, false>), grid, dim3(256), 0, s, p);
}

}  // namespace

void launch_grouped_act(int t, const GroupActParams& p, int slots, hipStream_t s) {
  if (t == T_F16) act<T_F16>(p, slots, s);
  else act<T_BF16>(p, slots, s);
}

}  // namespace gemm_epi
