// gemm_adapter.hpp -- device code of the linear layer with low-rank adapters as
// its host code (gemm_adapters.hip) sees it:
//   D = act(A . B^T + bias + scale[g] (A . down[g]^T) . up[g]^T) + R,
// g = ids[m], the adapter of row m (none outside 0 .. adapters - 1).
//
// Two launches.  The first makes U[m] = scale[g] A[m] . down[g]^T (M x rank,
// gemm_adapter_down.hip), rounded once to the operands' type, which the matrix
// cores read next; the second is the linear layer's kernel, whose accumulators
// take U . up[g]^T on top of A . B^T, so D is read and written once and the sum is
// rounded once.
#pragma once

#include "gemm_linear.hpp"

namespace gemm_epi {

struct AdapterParams : LinParams {
  const void* U;       // M x rank
  const void* up;      // adapters x N x rank
  const int32_t* ids;  // M
  int32_t rank, adapters;
};

constexpr int kMaxRank = 128;

// The adapter of row m; -1: none, or no such row.
__device__ __forceinline__ int row_adapter(const AdapterParams& p, int64_t m) {
  const int g = m < p.M ? p.ids[m] : -1;
  return g >= 0 && g < p.adapters ? g : -1;
}

// A fragment's 16 bytes of 16 rows: lane (q, r) has k = k0 + 8 q .. + 7 of its row.
__device__ __forceinline__ v4i adapter_load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t adapter_up(const AdapterParams& p, int g) {
  const int64_t bytes = p.N * p.rank * 2;
  return __builtin_amdgcn_make_buffer_rsrc((void*)((const char*)p.up + g * bytes), (short)0, (int)bytes, 0x00020000);
}

// Adds U . up[g]^T to a wave's accumulators (16x16 blocks, rows mw .., columns
// nw ..), one adapter of its rows after the other; fragments come straight from the
// cache.  A block of 16 rows that are not all g's own is summed apart and only
// g's rows are added: an infinity or a NaN in up[g] times a zero would reach the
// others.
template <class CF, class ACC>
__device__ __forceinline__ void adapter_step(const AdapterParams& p, ACC (&acc)[CF::FM][CF::FN], int mw, int nw) {
  using MM = typename CF::MM;
  static_assert(CF::BLK == 16 && MM::KSB == 64, "16-bit operands, 16x16 blocks");
  const int lane = __lane_id(), r = lane & 15, q = lane >> 4;
  int id[CF::FM];
  uint32_t todo[CF::FM];  // rows (lanes 0 .. 15) whose adapter is still to come
#pragma unroll
  for (int i = 0; i < CF::FM; ++i) {
    id[i] = row_adapter(p, mw + i * 16 + r);
    todo[i] = (uint32_t)__ballot(id[i] >= 0) & 0xffffu;
  }
  const int rows = (int)min(max(p.M - mw, (int64_t)0), (int64_t)CF::WM);
  const __amdgpu_buffer_rsrc_t ru = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((const char*)p.U + (int64_t)mw * p.rank * 2), (short)0, rows * p.rank * 2, 0x00020000);
  const uint32_t row = (uint32_t)p.rank * 2, ub = (uint32_t)r * row + 16 * q, nb = (uint32_t)(nw + r) * row + 16 * q;
  for (;;) {
    int g = -1;
    static_for<0, CF::FM>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      if (g < 0 && todo[i]) g = __builtin_amdgcn_readlane(id[i], __ffs(todo[i]) - 1);
    });
    if (g < 0) break;
    const __amdgpu_buffer_rsrc_t rp = adapter_up(p, g);
    for (int k = 0; k < p.rank; k += 32) {
      const bool in = k + 8 * q < p.rank;
      v4i fb[CF::FN];
      // (columns past the matrix lie outside the resource)
#pragma unroll
      for (int j = 0; j < CF::FN; ++j) fb[j] = adapter_load(rp, in ? nb + j * 16 * row + 2 * k : 0x80000000u);
      static_for<0, CF::FM>([&](auto i_c) {
        constexpr int i = decltype(i_c)::value;
        const uint32_t mine = (uint32_t)__ballot(id[i] == g) & 0xffffu;
        if (mine == 0) return;
        const v4i fa = adapter_load(ru, in && id[i] == g ? ub + i * 16 * row + 2 * k : 0x80000000u);
        if (mine == 0xffffu) {
#pragma unroll
          for (int j = 0; j < CF::FN; ++j) acc[i][j] = MM::mma(fa, fb[j], acc[i][j]);
        } else {
#pragma unroll
          for (int j = 0; j < CF::FN; ++j) {
            const typename MM::acc_t t = MM::mma(fa, fb[j], typename MM::acc_t{});
#pragma unroll
            for (int v = 0; v < MM::ACCN; ++v) acc[i][j][v] += mine >> MM::acc_row(lane, v) & 1 ? t[v] : 0.0f;
          }
        }
      });
    }
    static_for<0, CF::FM>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      todo[i] &= ~((uint32_t)__ballot(id[i] == g) & 0xffffu);
    });
  }
}

// U[m] = scale[g] A[m] . down[g]^T of type ab (T_F16 or T_BF16); rows without an
// adapter are left as they are.
struct AdapterDownParams {
  const void* A;
  const void* down;    // adapters x rank x K
  const float* scale;  // adapters
  const int32_t* ids;
  void* U;
  int64_t M, K, lda;
  int32_t rank, adapters;
};
void launch_adapter_down(int ab, const AdapterDownParams& p, hipStream_t s);

// The linear layer's kernels with the step above.
template <int AB, int BM, int BN, int S, int OCC>
using AdapterCfg = Cfg<AB, true, true, true, BM, BN, 128, 2, 2, S, 0, 16, 6, OCC>;
// Tile kernel bm x bn of the linear layer's plan (one of part PART).
constexpr int kAdapterParts = 4;
template <int PART>
void launch_adapter_part(int ab, int bm, const AdapterParams& p, int grid, hipStream_t s);
void launch_adapter_rows(int ab, int nw, const AdapterParams& p, hipStream_t s);

}  // namespace gemm_epi
