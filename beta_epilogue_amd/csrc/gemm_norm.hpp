// gemm_norm.hpp -- the root-mean-square norm's device code (gemm_norm_kernels.hip)
// as its host code (gemm_norm.hip) sees it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gemm_epi {

constexpr int64_t kNormMaxCols = 16384;  // a row stays in the registers of one workgroup

struct NormParams {
  const void* x;
  const void* r;  // residual, or NULL
  const void* w;
  void* y;
  void* h;        // x + r rounded to x's type, or NULL
  float* scale;   // row scales of an 8-bit y
  int64_t rows, cols;
  int64_t ldx, ldr, ldh, ldy;  // elements between rows
  int32_t w_f32;  // the weight is fp32 (else x's type)
  float eps;
};

struct NormGradParams {
  const void* dy;
  const void* h;
  const void* w;
  const void* dh_in;  // gradient that reaches h by other ways, or NULL
  void* dh;
  float* partial;     // [grid][cols] sums for dweight (grid 1: dweight), or NULL
  int64_t rows, cols;
  int64_t ldy, ldh, ldi, ldo;
  int32_t w_f32;
  float eps;
};

// x_dtype: T_F16, T_BF16 or T_F32; y_dtype: x_dtype, T_E4M3 or T_I8.
void launch_rmsnorm(int x_dtype, int y_dtype, const NormParams& p, hipStream_t s);

// Workgroups of the backward for these sizes on `cus` compute units.
int rmsnorm_grad_grid(int64_t rows, int64_t cols, int cus);
void launch_rmsnorm_grad(int x_dtype, const NormGradParams& p, int grid, hipStream_t s);

}  // namespace gemm_epi
