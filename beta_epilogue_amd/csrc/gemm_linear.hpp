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

// Tile kernels: K-major A and B, N-major D, 128-byte rows, 2 x 2 waves, two
// stages, LIN arguments and epilogue.
template <int AB, int BM, int BN, int BLK>
using LinearCfg = Cfg<AB, true, true, true, BM, BN, 128, 2, 2, 2, 0, BLK, true>;

constexpr int kLinearParts = 8;
// Launches variant number `variant` of gemm_linear_variants.inc (one of part
// PART) on `grid` workgroups.
template <int PART>
void launch_linear_part(int variant, const LinParams& p, int grid, hipStream_t s);

// The second kernel of a split-K plan: adds the slices' partial sums in slice
// order and applies the epilogue.  int_path: int32 partial sums.
void launch_linear_splitk(const LinParams& p, int tile_m, int tile_n, bool int_path, int grid, hipStream_t s);

// Few rows: M <= 16 * nb (nb 1, 2 or 4); rb blocks of 16 weight rows per
// workgroup (1 or 2).  ab: T_F16, T_BF16, T_E4M3 or T_I8.
constexpr int kRowsMax = 64;
void launch_linear_rows(int ab, int nb, int rb, const LinParams& p, hipStream_t s);

// dZ = dD * act'(Z) (skipped with act == ACT_NONE) and, if partial is given,
// the column sums of each chunk of `chunk` rows into partial[chunk][N].
// Packed M x N tensors of type t (T_F16 or T_BF16), N a multiple of 8.
void launch_linear_dact(int t, int act, const void* dD, const void* Z, void* dZ, float* partial, int64_t M, int64_t N,
                        int chunk, hipStream_t s);

// out[c] = sum over p < P of partial[p][c], in a fixed order (a tree over 32
// interleaved strands of ascending p), rounded to type t.
void launch_colsum(const float* partial, int64_t P, int64_t C, void* out, int t, hipStream_t s);

}  // namespace gemm_epi

#include "gemm_linear_epilogue.hpp"
