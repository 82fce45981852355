// gemm_linear.hpp -- the linear layer's device code as its host code
// (gemm_linear.hip) sees it: the tile kernels (gemm_linear_part.hip), the
// split-K join and the few-row kernels (gemm_linear_rows.hip), and the
// backward's elementwise pass and column sums (gemm_linear_grad.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_epi_kernel.hpp"
#include "linear_act.hpp"

namespace gemm_epi {

// Arguments of the linear layer's kernels: A, B, D, the sizes, the schedule,
// alpha and the K split as above (L == 1; C, X, Y, beta and xf unused), and
//   z = alpha * scale_a[m] * scale_b[n] * acc + bias[n],  D = act(z) + R,
//   Z = z.  D, R and Z have type d_dtype.
struct LinParams : Params {
  const float* scale_a;  // M row scales, or NULL (1)
  const float* scale_b;  // N column scales, or NULL (1)
  const void* bias;      // N values of bias_dtype, or NULL (0)
  const void* R;         // residual, or NULL
  void* Z;               // NULL when the pre-activation is not kept
  int64_t lda, ldb, ldd, ldr, ldz;  // elements between rows
  int32_t bias_dtype;    // T_F16, T_BF16 or T_F32
  int32_t act;           // ACT_*
};

// e4m3 operands with an fp32 D: a fragment is widened to fp16 in registers
// (exact; every e4m3 value is an fp16 value) and multiplied by fp16 MFMAs, whose
// sums keep fp32's precision.  Which eight of a lane's sixteen k an MFMA takes
// does not matter as long as both operands agree.
enum : int { T_E4M3_WIDE = 15 };
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
__device__ __forceinline__ v8h widen8(uint32_t a, uint32_t b) {
  const v2h p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
  const v2h p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
  const v2h p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
  const v2h p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  return v8h{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}
template <> struct Mma<T_E4M3_WIDE, 16> : MmaLayout16 {
  typedef v4f acc_t;
  typedef v4i frag_t;
  static constexpr int ESIZE = 1, KSB = 64;
  static __device__ __forceinline__ acc_t mma(frag_t a, frag_t b, acc_t c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(a[0], a[1]), widen8(b[0], b[1]), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(a[2], a[3]), widen8(b[2], b[3]), c, 0, 0, 0);
  }
};

// Tile kernels: K-major A and B, N-major D, 128-byte rows, 2 x 2 waves, S
// stages, LIN arguments and epilogue.
template <int AB, int BM, int BN, int S, int OCC, int BLK>
using LinearCfg = Cfg<AB, true, true, true, BM, BN, 128, 2, 2, S, 0, BLK, 1, OCC>;

constexpr int kLinearParts = 8;
// Launches variant number `variant` of gemm_linear_variants.inc (one of part
// PART) on `grid` workgroups.
template <int PART>
void launch_linear_part(int variant, const LinParams& p, int grid, hipStream_t s);

// The backward's products, one launch for both:
//   a: dA = alpha dZ . B  (M x K over N: A = dZ K-major, B = B N-major)
//   b: dB = dB_in + alpha dZ^T . A  (N x K over M: A = dZ M-major, B = A N-major)
// ga workgroups run a and gb run b (b's come first with b_first), the rest make
// dbias: of the chunks' column sums in partial, or without an activation of
// dZ = dD itself.  A problem that is not wanted has 0.
// Four kernels per type: 256x256 tiles; 128x128 tiles with two workgroups per
// compute unit; 128x128 tiles with a ring of three stages, for grids of at most
// one workgroup per compute unit, whose transposing reads have nobody else's
// MFMAs to hide behind (dA of 64 x 4096 x 4096 37.7 -> 25.5 us; with 512 tiles,
// 2048^3, the pair takes 35 us and the deep ring 39); 64x64 tiles, two per
// compute unit with rings of four stages, for small problems, whose larger tiles
// would leave compute units idle or need K slices and a join (134 x 1272 x 1336
// 19.1 us with 128x128 tiles and 15.3 with these, 449 x 1952 x 1288 23.5 and
// 21.9; 2048^3 44 and 65).
enum : int { GRAD_256 = 0, GRAD_128 = 1, GRAD_128_DEEP = 2, GRAD_64 = 3, kGradKinds = 4 };
constexpr int grad_tile(int kind) { return kind == GRAD_256 ? 256 : kind == GRAD_64 ? 64 : 128; }
// Workgroups per compute unit.
constexpr int grad_occ(int kind) { return kind == GRAD_128 || kind == GRAD_64 ? 2 : 1; }
constexpr int grad_stages(int kind) { return kind == GRAD_128_DEEP ? 3 : kind == GRAD_64 ? 4 : 2; }
template <int AB, bool A_KMAJOR, int KIND>
using GradCfg = Cfg<AB, A_KMAJOR, false, true, grad_tile(KIND), grad_tile(KIND), 128, 2, 2, grad_stages(KIND),
                    KIND == GRAD_256 ? 2 : 0, 32, 2, grad_occ(KIND)>;
struct GradParams {
  LinParams a, b;
  int32_t ga, gb, b_first;
  const float* partial;  // [P][C], or NULL
  const void* rows;      // [P][C] of type AB to be summed (NULL: none)
  int64_t P, C;
  void* dbias;
  int32_t dbias_dtype;
};
// Kernel KIND of type AB (T_F16 or T_BF16).
template <int AB, int KIND>
void launch_linear_grad_mm(const GradParams& p, hipStream_t s);

// Adds the slices of split tiles of both products (tail_tiles 0: none).
void launch_linear_grad_join(const LinParams& a, const LinParams& b, int tile, int64_t most_blocks, hipStream_t s);

// The second kernel of a split-K plan: adds the slices' partial sums in slice
// order and applies the epilogue.  int_path: int32 partial sums.
void launch_linear_splitk(const LinParams& p, int tile_m, int tile_n, bool int_path, int grid, hipStream_t s);

// Few rows: M <= kRowsMax, 16 weight rows per workgroup of nw waves (4 or 8;
// up to 8 rows always 8).  ab: T_F16, T_BF16, T_E4M3 or T_I8.
constexpr int kRowsMax = 64;
void launch_linear_rows(int ab, int nw, const LinParams& p, hipStream_t s);

// dZ = dD * act'(Z) (skipped with act == ACT_NONE) and, if wanted, the column
// sums: of each chunk of `chunk` rows into partial[chunk][N], or with one chunk
// straight into dbias (partial NULL).  Packed M x N tensors of type t (T_F16
// or T_BF16), N a multiple of 8.
void launch_linear_dact(int t, int act, const void* dD, const void* Z, void* dZ, float* partial, void* dbias,
                        int dbias_dtype, int64_t M, int64_t N, int chunk, hipStream_t s);

// out[c] = sum over p < P of partial[p][c], in a fixed order (a tree over
// strands of ascending p), rounded to type t.
void launch_colsum(const float* partial, int64_t P, int64_t C, void* out, int t, hipStream_t s);

__device__ __forceinline__ void store_as(void* out, int64_t i, int t, float v) {
  if (t == T_F32) ((float*)out)[i] = v;
  else if (t == T_F16) ((_Float16*)out)[i] = (_Float16)v;
  else ((__bf16*)out)[i] = (__bf16)v;
}

// 32 columns per workgroup of 32 * STRANDS threads; red: STRANDS x 33 words.
template <int STRANDS>
__device__ __forceinline__ void colsum_block(const float* partial, int64_t P, int64_t C, void* out, int t,
                                             int64_t block, float* red) {
  const int cl = threadIdx.x & 31, pl = threadIdx.x >> 5;
  const int64_t c = block * 32 + cl;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int64_t p = pl; p < P; p += STRANDS) s += partial[p * C + c];
  }
  red[pl * 33 + cl] = s;
  __syncthreads();
#pragma unroll
  for (int d = STRANDS / 2; d >= 1; d >>= 1) {
    if (pl < d) red[pl * 33 + cl] += red[(pl + d) * 33 + cl];
    __syncthreads();
  }
  if (pl == 0 && c < C) store_as(out, c, t, red[cl]);
}

}  // namespace gemm_epi

#include "gemm_linear_epilogue.hpp"
