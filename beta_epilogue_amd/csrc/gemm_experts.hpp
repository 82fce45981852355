// gemm_experts.hpp -- the device code around the experts' products as its host
// code (gemm_experts.hip) sees it: the sort of tokens by expert, the way back
// and its gradient (gemm_experts_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gemm_epi {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
// Choices (of a token and an expert) that one workgroup ranks: all of up to twice a
// chunk, or a chunk each.
constexpr int kSortChunk = 4096;
inline int64_t sort_chunks(int64_t choices) {
  return choices <= 2 * kSortChunk ? 1 : (choices + kSortChunk - 1) / kSortChunk;
}

// The sum of v over this lane and those before it; every lane of the wave calls.
// Shifts inside rows of 16 lanes, then the rows' totals: register to register, for it
// stands at the start of every workgroup that looks for its expert.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 to row 1, 47 to row 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2 and 3
  return v;
}

struct SortParams {
  const void* ids;       // choices x int32 or int64
  const void* X;         // rows to move, or NULL
  const float* scale;    // of the rows of X, or NULL
  int32_t* offsets;      // experts + 1
  int32_t* rows;         // choices (NULL: not wanted)
  void* Y;
  float* scale_out;
  int32_t* order;        // the choice of each row (NULL: not wanted)
  int32_t* counts;       // workspace: chunks x experts (one chunk: NULL)
  int64_t tokens;
  int64_t row_bytes, ldx, ldy;  // bytes; a multiple of 16
  int32_t top_k, experts, chunks, ids64;
};
void launch_expert_sort(const SortParams& p, hipStream_t s);

struct CombineParams {
  const void* Y;
  const int32_t* rows;
  const float* weights;  // NULL: 1
  const void* R;         // NULL: 0
  void* D;
  const void* dD;        // backward
  void* dY;
  float* dweights;
  int64_t tokens, cols, ldy, ldd, ldr, ldg;  // elements
  int32_t top_k;
};
// t: T_F16, T_BF16 or T_F32.
void launch_expert_combine(int t, const CombineParams& p, hipStream_t s);
void launch_expert_combine_grad(int t, const CombineParams& p, hipStream_t s);

}  // namespace gemm_epi
