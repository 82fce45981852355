/*
 * gemm_epi_norm.h -- C ABI of the root-mean-square norm on MI355X (gfx950),
 * which writes the operands of the GEMM and the linear layer: with the
 * residual's addition in front, into 16 bits, fp32, or 8 bits with a scale per
 * row (the linear layer's A and scale_a), and its backward.
 *
 *     h = x + r          s = 1 / sqrt(mean(h^2) + eps)          y = h s w
 *     8 bits: scale = max(max_row |y| / qmax, 2^-126),  q = round(y / scale)
 *             (qmax 448 for e4m3, 127 for int8; round to nearest-even)
 *     backward, s of the stored h and g = dy w:
 *       dh = dh_in + s g - h s^3 mean(g h)         dw = sum over rows of dy h s
 *
 * dh is the gradient of x and of r alike.  Everything is computed in fp32 and
 * rounded once; h is also rounded into x's type as an output, while y comes
 * from the unrounded h.  The squares are fp32 numbers too: where their sum
 * overflows (a root mean square of 1.8e19 / sqrt(columns)) s is 0.  eps 0 stands
 * for 2^-149, the least positive fp32 number, so an all-zero row gives zeros
 * with any eps.  A row that holds a NaN or an infinity gets a NaN or infinite
 * scale in 8 bits; its values are NaN or 0 (e4m3), or 0 where they would be NaN
 * (int8).
 *
 * Tensors are row-major with a stride between rows; any number of columns up
 * to 16384, any stride, element alignment (16 bytes are faster).  Status
 * codes, handles, streams and workspaces as in gemm_epi_linear.h.
 */
#ifndef GEMM_EPI_NORM_H
#define GEMM_EPI_NORM_H

#include "gemm_epi.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemm_epi_rmsnorm_desc {
  int64_t rows, cols;          /* >= 1; cols <= 16384 */
  int64_t ldx, ldr, ldh, ldy;  /* elements between rows; 0: cols */
  int32_t x_dtype;             /* F16, BF16 or F32: x, r and h */
  int32_t y_dtype;             /* x_dtype, E4M3 or I8 */
  int32_t weight_dtype;        /* x_dtype or F32 */
  int32_t residual;            /* 1: r is added (and h may be written) */
  float eps;                   /* finite, >= 0 (0: 2^-149) */
} gemm_epi_rmsnorm_desc;

typedef struct gemm_epi_rmsnorm_handle gemm_epi_rmsnorm_handle;

/* Validate and plan.  INVALID_ARG: sizes, codes, strides below cols or given
 * for a tensor that is not used, eps.  UNSUPPORTED: more than 16384 columns,
 * other types, 2^31 rows.  DEVICE: no gfx950. */
int gemm_epi_rmsnorm_create(const gemm_epi_rmsnorm_desc* desc, gemm_epi_rmsnorm_handle** out);

/* Enqueue.  x, weight and Y are required; r exactly with desc.residual; H may
 * be NULL, and may be given only with desc.residual; scale (rows fp32 values)
 * exactly for an 8-bit Y.  H may be x or r itself and Y may be x or r itself
 * (the same pointer, stride and type; not both); no other overlap of an output
 * with another tensor is allowed. */
int gemm_epi_rmsnorm_run(const gemm_epi_rmsnorm_handle* h, const void* x, const void* r, const void* weight, void* Y,
                         void* H, float* scale, void* stream);

/* Free a handle (NULL is fine). */
int gemm_epi_rmsnorm_destroy(gemm_epi_rmsnorm_handle* h);

typedef struct gemm_epi_rmsnorm_grad_desc {
  int64_t rows, cols;          /* >= 1; cols <= 16384 */
  int64_t ldy, ldh, ldi, ldo;  /* of dY, H, dH_in and dH; 0: cols */
  int32_t x_dtype;             /* F16, BF16 or F32: dY, H, dH_in and dH */
  int32_t weight_dtype;        /* x_dtype or F32 */
  int32_t dweight_dtype;       /* NONE (not wanted), F16, BF16 or F32 */
  float eps;
} gemm_epi_rmsnorm_grad_desc;

typedef struct gemm_epi_rmsnorm_grad_handle gemm_epi_rmsnorm_grad_handle;

/* As gemm_epi_rmsnorm_create. */
int gemm_epi_rmsnorm_grad_create(const gemm_epi_rmsnorm_grad_desc* desc, gemm_epi_rmsnorm_grad_handle** out);

/* Enqueue.  dY, H, weight and dH are required; dH_in may be NULL (0); dweight
 * exactly when its type is set (summed in fp32 in a fixed order).  dH may be
 * dY, H or dH_in itself (the same pointer and stride); no other overlap of an
 * output with another tensor is allowed. */
int gemm_epi_rmsnorm_grad_run(const gemm_epi_rmsnorm_grad_handle* h, const void* dY, const void* H, const void* weight,
                              const void* dH_in, void* dH, void* dweight, void* workspace, int64_t workspace_bytes,
                              void* stream);

/* Free a handle (NULL is fine). */
int gemm_epi_rmsnorm_grad_destroy(gemm_epi_rmsnorm_grad_handle* h);

/* Bytes of workspace a run needs (-1 for a NULL handle). */
int64_t gemm_epi_rmsnorm_grad_workspace(const gemm_epi_rmsnorm_grad_handle* h);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_EPI_NORM_H */
