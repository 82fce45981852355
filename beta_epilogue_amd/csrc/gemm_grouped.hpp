// gemm_grouped.hpp -- the experts' linear layers' device code as its host code
// (gemm_experts_linear.hip) sees it: the tile kernels over groups of rows
// (gemm_grouped_part.hip), the few-row kernels (gemm_grouped_rows.hip) and the
// backward (gemm_grouped_grad.hip, gemm_grouped_act.hip).
//
// Rows offsets[e] .. offsets[e + 1] - 1 of A, D, ... are group e's, whose B, bias
// and column scales are the e-th.  Only the device knows the offsets, so a
// launch has as many workgroups as the worst distribution needs, or persistent
// ones, and each finds its group from the offsets by itself: nothing is copied to
// the host and no table is made by another launch.
#pragma once

#include "gemm_experts.hpp"
#include "gemm_linear.hpp"

namespace gemm_epi {

// Arguments of the grouped kernels: the linear layer's, with M the batch's rows or
// (LIN 5) a group's output's; R is the factor of the forward (LIN 3) or dB_in (LIN
// 5).  B, bias, scale_b, and the backward's dB and dB_in hold one packed part
// per group.
struct GroupParams : LinParams {
  const int32_t* offsets;  // groups + 1
  int32_t groups;
  int32_t rows;            // the batch's capacity
};

// Offsets that do not ascend within 0 .. rows are moved into that range, so no access
// leaves the tensors whatever they hold.
__device__ __forceinline__ GroupTile group_rows(const GroupParams& p, int group) {
  GroupTile t = {};
  t.group = group;
  t.begin = min(max(p.offsets[group], 0), p.rows);
  t.end = min(max(p.offsets[group + 1], t.begin), p.rows);
  return t;
}

// GROUP_K: the item (tile of a group's output) of workgroup bid of 8 * groups *
// ceil(tiles / 8), tiles_total for none, and the group's rows.  Workgroups go round
// the 8 XCDs, and a group with many rows has long items: every group's tiles are
// spread over all XCDs, and the groups with the most rows go first.  More than 64 go by
// number, and a long one that comes last costs (128 experts, 768 x 2048, 8192 of 32768
// rows on one, both products: the first 401 us, the last 509; evenly spread 340).
// Every workgroup finds that order by itself, in two instructions per group (2048 rows
// of 64 experts, 1536 x 2048, both products: 200 us; with six, and the offsets read again
// for the rows, 297).
__device__ __forceinline__ GroupWork group_k_item(const GroupParams& p, int bid) {
  const int tiles = p.tiles_m * p.tiles_n, per = (tiles + 7) >> 3, lane = __lane_id();
  int e = (int)((unsigned)(bid >> 3) / (unsigned)per);
  const int j = (bid >> 3) - e * per;
  GroupTile t = {};
  if (p.groups <= 64) {
    // (2^25 rows and more count as alike)
    uint32_t key = 0;
    if (lane < p.groups) {
      t = group_rows(p, lane);
      key = (uint32_t)min(t.end - t.begin, (1 << 25) - 1) << 6 | (63u - lane);
    }
    int before = 0;
#pragma unroll
    for (int base = 0; base < 64; base += 8) {
      if (base >= p.groups) break;
#pragma unroll
      for (int l = base; l < base + 8; ++l) before += (uint32_t)__builtin_amdgcn_readlane((int)key, l) > key ? 1 : 0;
    }
    e = __ffsll((unsigned long long)__ballot(lane < p.groups && before == e)) - 1;
    t.begin = __builtin_amdgcn_readlane(t.begin, e);
    t.end = __builtin_amdgcn_readlane(t.end, e);
  } else {
    t = group_rows(p, e);
    t.begin = __builtin_amdgcn_readfirstlane(t.begin);
    t.end = __builtin_amdgcn_readfirstlane(t.end);
  }
  const int tile = (((bid & 7) + e) & 7) * per + j;
  const int item = __builtin_amdgcn_readfirstlane(tile < tiles ? e * tiles + tile : p.tiles_total);
  return GroupWork{nullptr, item, item + 1, 0, t.begin, t.end};
}

// The table of groups in LDS: first[g] = tiles of `rows` rows in the groups
// before g (first[groups]: in all, returned).  All threads of the workgroup.
// Offsets that do not ascend could count rows more than once; there are never more
// tiles than the worst distribution has, which is what the host made sure of.
constexpr int kGroupTableBytes = (kMaxExperts + 1) * 4 + 12;
__device__ __forceinline__ int group_table_rows(const GroupParams& p, int* first, int rows) {
  const int lane = __lane_id();
  if (threadIdx.x < 64) {
    const int n0 = min(p.rows, p.groups), most = n0 + (p.rows - n0) / rows;
    int before = 0;
    for (int base = 0; base < p.groups; base += 64) {
      const int g = base + lane;
      int n = 0;
      if (g < p.groups) {
        const GroupTile t = group_rows(p, g);
        n = (t.end - t.begin + rows - 1) / rows;
      }
      // (unsigned: 64 groups of up to 2^25 tiles)
      const uint32_t sum = (uint32_t)before + (uint32_t)wave_scan(n);
      if (g < p.groups) first[g] = (int)min(sum - (uint32_t)n, (uint32_t)most);
      before = (int)min((uint32_t)__builtin_amdgcn_readlane((int)sum, 63), (uint32_t)most);
    }
    if (lane == 0) first[p.groups] = before;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(first[p.groups]);
}

// The group of row tile number `row_tile` (below first[groups]).
__device__ __forceinline__ GroupTile group_of_tile(const GroupParams& p, const int* first, int row_tile) {
  const int lane = __lane_id();
  int g = 0;
  for (int base = 0; base < p.groups; base += 64) {
    const int n = __popcll(__ballot(base + lane < p.groups && first[base + lane + 1] <= row_tile));
    g += n;
    if (n < 64) break;
  }
  g = __builtin_amdgcn_readfirstlane(g);
  GroupTile t = group_rows(p, g);
  t.begin = __builtin_amdgcn_readfirstlane(t.begin);
  t.end = __builtin_amdgcn_readfirstlane(t.end);
  t.first = __builtin_amdgcn_readfirstlane(first[g]);
  t.tiles = __builtin_amdgcn_readfirstlane(first[g + 1]) - t.first;
  return t;
}

// Chunk number `slot` of `rows` rows, without a table (one chunk per workgroup):
// begin .. end - 1 are the chunk's rows; group -1: there is no such chunk.
__device__ __forceinline__ GroupTile group_chunk(const GroupParams& p, int slot, int rows) {
  const int lane = __lane_id();
  int before = 0;
  for (int base = 0; base < p.groups; base += 64) {
    const int g = base + lane;
    GroupTile t = {};
    if (g < p.groups) t = group_rows(p, g);
    const int n = (t.end - t.begin + rows - 1) / rows;
    const int sum = before + wave_scan(n);  // chunks of this group and those before
    const uint64_t behind = __ballot(sum > slot);
    if (behind) {
      const int l = __ffsll((unsigned long long)behind) - 1;
      GroupTile r = {};
      r.group = base + l;
      const int begin = __builtin_amdgcn_readlane(t.begin, l), end = __builtin_amdgcn_readlane(t.end, l);
      const int c = slot - __builtin_amdgcn_readlane(sum - n, l);
      r.begin = begin + c * rows;
      r.end = min(end, r.begin + rows);
      return r;
    }
    before = __builtin_amdgcn_readlane(sum, 63);
  }
  GroupTile none = {};
  none.group = -1;
  return none;
}

// Tile kernels of the forward.
template <int AB, int BM, int BN, int S, int OCC, int BLK>
using GroupedCfg = Cfg<AB, true, true, true, BM, BN, 128, 2, 2, S, 0, BLK, 3, OCC>;
// The 128x128 kernel that finishes the last round of 256x256 tiles.
template <int AB>
using GroupedQuarter = GroupedCfg<AB, 128, 128, AB == T_E4M3 ? 4 : 2, 1, AB == T_E4M3 ? 32 : 16>;

constexpr int kGroupedParts = 7;
template <int PART>
void launch_grouped_part(int variant, const GroupParams& p, int grid, hipStream_t s);

// Few rows per group: chunks of up to 4 * mb rows (mb 1 or 4), 16 weight
// rows per workgroup; slots: chunks that the worst distribution has.
void launch_grouped_rows(int ab, int mb, const GroupParams& p, int slots, hipStream_t s);

// The backward's products, one launch for both (GRAD_* as for the linear layer):
//   a: dA = dZ . B[e] over groups of rows; ga workgroups, a tile each at most
//   b: dB[e] = dB_in[e] + dZ^T . A over each group's rows; gb workgroups
// sums workgroups make dbias.  In the order a, b, sums, or with b_first b, sums, a.
template <int AB, bool ROWS, int KIND>
using GroupedGradCfg = Cfg<AB, ROWS, false, true, grad_tile(KIND), grad_tile(KIND), 128, 2, 2, grad_stages(KIND),
                           KIND == GRAD_256 ? 2 : 0, 32, ROWS ? 4 : 5, grad_occ(KIND)>;
struct GroupGradParams {
  GroupParams a, b;
  int32_t ga, gb, sums;   // workgroups
  int32_t b_first;
  const void* sum_rows;   // dD, whose rows dbias adds up; NULL: the chunks' sums
  float* row_sums;        // ... chunk by chunk, into this one's [chunk][N]; NULL: an expert's at once
  const float* partial;   // the chunks' sums, [chunk][N]
  int32_t chunk;          // rows of a chunk
  void* dbias;            // groups x N
  int32_t dbias_dtype;
  int64_t N;
};
template <int AB, int KIND>
void launch_grouped_grad(const GroupGradParams& p, hipStream_t s);

// The elementwise pass over the rows of all groups, in chunks of `chunk` rows:
//   g = dD * U,  dZ = g * act'(Z),  dU = dD * act(Z)
// (without Z: dZ is dD and only summed) and the column sums of dZ, unrounded, of
// each chunk into partial[slot][N] (NULL: not wanted).  Packed tensors of type t.
struct GroupActParams : GroupParams {
  const void *dD, *U, *dZin;  // dZin: Z
  void *dZ, *dU;
  float* partial;
  int32_t chunk;
};
void launch_grouped_act(int t, const GroupActParams& p, int slots, hipStream_t s);

}  // namespace gemm_epi
