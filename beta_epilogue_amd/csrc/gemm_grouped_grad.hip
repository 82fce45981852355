// gemm_grouped_grad.hip -- the two matrix products of the experts' backward in
// one launch, compiled once per type and kernel (GEMM_GROUPED_GRAD_PART 0 .. 7).
//
// dA = dZ . B[e] has tiles of each expert's rows; dB[e] = dB_in[e] + dZ^T . A sums
// over the expert's rows, one set of tiles per expert, those of the experts with
// the most rows first and each expert's spread over the XCDs (16384 rows of 8
// experts, 825 to 4282 each, N 4096, K 2048: dB 344 us with an expert per XCD).
// Bound by the MFMAs and the transposing LDS reads: both products of those rows take
// 462 us (1190 TFLOP/s).  dbias is made by further workgroups from the elementwise pass's
// column sums, in the order of the chunks, or without such a pass from dD's rows: all of
// an expert's at once, or chunk by chunk, for a second launch of this kernel that has
// nothing but the join to do.
#include "gemm_grouped.hpp"

#ifndef GEMM_GROUPED_GRAD_PART
#error "GEMM_GROUPED_GRAD_PART must be defined (0 .. 7)"
#endif

namespace gemm_epi {

namespace {

// 64 columns of a group's dbias, or of a chunk's sums, straight from the rows of dD: 8
// lanes of 8 columns by 32 strands of rows, joined in a fixed order.  red: 32 x 68 words.
template <int AB>
__device__ __forceinline__ void group_row_sums(const GroupGradParams& p, int block, float* red) {
  const int per = (int)((p.N + 63) / 64), slot = block / per;
  const GroupTile t = p.row_sums ? group_chunk(p.a, slot, p.chunk) : group_rows(p.a, slot);
  if (t.group < 0) return;
  const int cl = threadIdx.x & 7, pl = threadIdx.x >> 3;
  const int64_t c0 = (int64_t)(block - slot * per) * 64, c = c0 + cl * 8;
  float s[8] = {};
  if (c < p.N) {
#pragma unroll 8
    for (int r = t.begin + pl; r < t.end; r += 32) {
      const v4u w = *(const v4u*)((const uint16_t*)p.sum_rows + r * p.N + c);
      const v4f lo = epi_dec<AB>(w, 0), hi = epi_dec<AB>(w, 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += lo[k], s[4 + k] += hi[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) red[pl * 68 + cl * 8 + k] = s[k];
  __syncthreads();
  const int64_t n = c0 + threadIdx.x;
  if (threadIdx.x >= 64 || n >= p.N) return;
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; ++k) v += red[k * 68 + threadIdx.x];
  if (p.row_sums) p.row_sums[slot * p.N + n] = v;
  else store_as(p.dbias, slot * p.N + n, p.dbias_dtype, v);
}

// 256 columns of group g's dbias.
__device__ __forceinline__ void group_sums(const GroupGradParams& p, int block, int* first) {
  const GroupParams& q = p.a;
  group_table_rows(q, first, p.chunk);
  const int per = (int)((p.N + 255) / 256), g = block / per;
  const int64_t n = (int64_t)(block - g * per) * 256 + threadIdx.x;
  if (n >= p.N) return;
  float s = 0.0f;
#pragma unroll 8
  for (int c = first[g]; c < first[g + 1]; ++c) s += p.partial[c * p.N + n];
  store_as(p.dbias, g * p.N + n, p.dbias_dtype, s);
}

// dB[e] of an expert without rows is dB_in[e] or zero: each of the expert's items
// copies its share, straight from and to memory (one token, 6 of 28 experts, 3856 x 896
// bf16, 193 MB: 46 us, as tiles with a K tile of zeros 180).  False: the item's expert has
// rows.
__device__ __forceinline__ bool fill_without_rows(const GroupParams& p, const GroupWork& w) {
  if (w.rows_end > w.row) return false;
  const int item = w.begin, tiles = p.tiles_m * p.tiles_n, e = item / tiles;
  if (p.R == p.D) return true;
  const int64_t n = p.M * p.N << epi_shift(p.d_dtype) >> 4, share = (n + tiles - 1) / tiles;  // 16-byte pieces
  const int64_t begin = (item - e * tiles) * share, end = min(begin + share, n);
  v4u* d = (v4u*)p.D + e * n;
  const v4u* r = p.R ? (const v4u*)p.R + e * n : nullptr;
#pragma unroll 4
  for (int64_t i = begin + threadIdx.x; i < end; i += 256)
    __builtin_nontemporal_store(r ? __builtin_nontemporal_load(r + i) : v4u{}, d + i);
  return true;
}

template <int AB, int KIND>
__global__ __launch_bounds__(256, grad_occ(KIND)) void grouped_grad_kernel(GroupGradParams p) {
  using CA = GroupedGradCfg<AB, true, KIND>;
  using CB = GroupedGradCfg<AB, false, KIND>;
  constexpr int A_BYTES = CA::LDS_BYTES + kGroupTableBytes;
  __shared__ __attribute__((aligned(1024))) char lds[A_BYTES > CB::LDS_BYTES ? A_BYTES : CB::LDS_BYTES];
  const int bid = blockIdx.x, a0 = p.b_first ? p.gb + p.sums : 0, b0 = p.b_first ? 0 : p.ga;
  if (bid >= a0 && bid < a0 + p.ga) {
    int* first = (int*)(lds + CA::LDS_BYTES);
    const int total = group_table_rows(p.a, first, CA::BM) * p.a.tiles_n;
    gemm_epi_body<CA>(p.a, lds, bid - a0, p.ga, GroupWork{first, 0, total, 0});
  } else if (bid >= b0 && bid < b0 + p.gb) {
    const GroupWork w = group_k_item(p.b, bid - b0);
    if (w.begin >= p.b.tiles_total || fill_without_rows(p.b, w)) return;
    gemm_epi_body<CB>(p.b, lds, bid - b0, p.gb, w);
  } else {
    const int block = bid - p.gb - (p.b_first ? 0 : p.ga);
    if (p.sum_rows) group_row_sums<AB>(p, block, (float*)lds);
    else group_sums(p, block, (int*)lds);
  }
}

}  // namespace

constexpr int kAb = GEMM_GROUPED_GRAD_PART % 2 ? T_BF16 : T_F16, kKind = GEMM_GROUPED_GRAD_PART / 2;

template <>
void launch_grouped_grad<kAb, kKind>(const GroupGradParams& p, hipStream_t s) {
  hipLaunchKernelGGL((grouped_grad_kernel<kAb, kKind>), dim3((unsigned)(p.ga + p.gb + p.sums)), dim3(256), 0, s, p);
}

}  // namespace gemm_epi
