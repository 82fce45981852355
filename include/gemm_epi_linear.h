/*
 * gemm_epi_linear.h -- C ABI of the linear layer on MI355X (gfx950): a matrix
 * product with scales, bias, activation and residual in its epilogue, its
 * form for few rows (decoding), and its backward.
 *
 *     z[m][n] = alpha * scale_a[m] * scale_b[n] * sum_k A[m][k] B[n][k] + bias[n]
 *     D = act(z) + R            Z = z (kept for the backward, if asked for)
 *
 *     dZ = dD * act'(Z)         dbias[n] = sum_m dZ[m][n]
 *     dA = alpha dZ . B         dB = dB_in + alpha dZ^T . A
 *
 * A is M x K (M tokens), B is N x K (the weight, one row per output), D, R, Z
 * and dD are M x N; all are row-major.  The gradient of R is dD itself.  The
 * backward is that of a forward without scale_a and scale_b.
 *
 * Activations (fp32): none; relu max(z, 0); gelu z Phi(z); gelu_tanh
 * z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2; silu z / (1 + exp(-z)).  A
 * NaN z gives a NaN D, and so does z = -infinity with gelu, gelu_tanh and silu
 * (-infinity times 0, as in the formulas).  The slopes of infinite z are their
 * limits; relu's is 1 for z > 0, else 0.
 *
 * Types: A and B fp16, bf16, e4m3 or int8 (one type); D, R and Z one type of
 * fp16, bf16, fp32.  Products are summed in fp32 (int8: int32), the epilogue
 * is fp32, and each output is rounded once, to nearest-even.  e4m3 with an
 * fp32 D is widened (exactly) and runs on the fp16 matrix instructions, whose
 * sums keep fp32's precision.  Scales are meant for the 8-bit types but allowed for all.
 *
 * Conventions as in gemm_epi.h: status codes and gemm_epi_last_error();
 * everything that needs no device is checked at create; contiguous extents
 * and row strides are multiples of 16 bytes and base pointers 16-byte aligned;
 * one immutable handle per shape, usable from any host thread and stream of
 * its device; calls enqueue on the caller's stream and return.  A handle owns
 * no device memory: a plan's workspace is the caller's, is written before it
 * is read in every call, and must not be shared by calls that overlap in time.
 * Nothing is allocated in a run, so every run can be captured into a graph.
 */
#ifndef GEMM_EPI_LINEAR_H
#define GEMM_EPI_LINEAR_H

#include "gemm_epi.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations. */
enum {
  GEMM_EPI_ACT_NONE = 0,
  GEMM_EPI_ACT_RELU = 1,
  GEMM_EPI_ACT_GELU = 2,
  GEMM_EPI_ACT_GELU_TANH = 3,
  GEMM_EPI_ACT_SILU = 4
};

typedef struct gemm_epi_linear_desc {
  int64_t M, N, K;      /* all >= 1 */
  int64_t lda, ldb;     /* elements between rows of A and B; 0: K */
  int64_t ldd, ldr, ldz; /* of D, R and Z; 0: N */
  int32_t ab_dtype;     /* F16, BF16, E4M3 or I8 */
  int32_t d_dtype;      /* F16, BF16 or F32: D, R and Z */
  int32_t bias_dtype;   /* NONE, F16, BF16 or F32 */
  int32_t act;          /* GEMM_EPI_ACT_* */
  int32_t residual;     /* 1: R is added */
  int32_t z;            /* 1: Z is written */
  int32_t scale_a;      /* 1: M fp32 row scales */
  int32_t scale_b;      /* 1: N fp32 column scales */
  int32_t splits;       /* 0: the plan's choice; n: a tile kernel with every
                           tile in n K slices (fewer if K has fewer K tiles) */
} gemm_epi_linear_desc;

typedef struct gemm_epi_linear_handle gemm_epi_linear_handle;

/*
 * Validate a problem and plan it: the few-row kernel, which streams B once (M
 * of at most 16, and up to 64 where a cost model prefers it), or a tile kernel
 * whose tile shape and K split the model chooses.  INVALID_ARG: sizes, codes,
 * flags other than 0 and 1, strides below the extent, a stride of a tensor
 * that is not used.  ALIGNMENT: the 16-byte rule.  UNSUPPORTED: e5m2 and uint8;
 * rows or row strides too long for the kernels' 31-bit tile offsets; 2^31 or
 * more rows, columns or work items; int8 with K of 2^17 or more, whose int32
 * sums could overflow.  DEVICE: no gfx950.
 */
int gemm_epi_linear_create(const gemm_epi_linear_desc* desc, gemm_epi_linear_handle** out);

/* As gemm_epi_linear_create with kernel `variant` (-1: its choice); one that
 * cannot run the problem is UNSUPPORTED (the last variant, "linear_rows",
 * takes M of at most 64 and N of at most 2^26, and has no K slices: splits is
 * ignored). */
int gemm_epi_linear_create_variant(const gemm_epi_linear_desc* desc, int variant, gemm_epi_linear_handle** out);

/*
 * Enqueue D (and Z).  A, B, D are required; bias, scale_a, scale_b, R and Z
 * are given exactly when the desc says so.  D may be R itself (the same
 * pointer, with ldd == ldr); no other overlap of an output with another tensor
 * is allowed.  workspace: at least plan.workspace_bytes of device memory at a
 * 256-byte boundary, or NULL if that is 0.
 */
int gemm_epi_linear_run(const gemm_epi_linear_handle* h, const void* A, const void* B, const void* bias,
                        const float* scale_a, const float* scale_b, const void* R, void* D, void* Z, float alpha,
                        void* workspace, int64_t workspace_bytes, void* stream);

/* Free a handle (NULL is fine). */
int gemm_epi_linear_destroy(gemm_epi_linear_handle* h);

/* What a handle launches, in gemm_epi_plan's terms (variant indexes the linear
 * table; few rows: up to tile_m tokens by tile_n weight rows per workgroup,
 * tile_k and lds_bytes 0). */
int gemm_epi_linear_get_plan(const gemm_epi_linear_handle* h, gemm_epi_plan* out);

/* Number of linear kernels and the name of one (NULL out of range). */
int gemm_epi_linear_variant_count(void);
const char* gemm_epi_linear_variant_name(int variant);

typedef struct gemm_epi_linear_grad_desc {
  int64_t M, N, K;     /* the forward's; all tensors packed */
  int32_t ab_dtype;    /* F16 or BF16: dD, Z, dZ, A and B */
  int32_t act;         /* the forward's activation */
  int32_t da_dtype;    /* NONE (no dA), F16, BF16 or F32 */
  int32_t db_dtype;    /* NONE (no dB), F16, BF16 or F32: dB and dB_in */
  int32_t dbias_dtype; /* NONE (no dbias), F16, BF16 or F32 */
  int32_t tile;        /* 0: the plan's choice; 64, 128 or 256: that tile */
  int32_t splits;      /* 0: the plan's choice; n: every tile of both products
                          in n K slices (fewer if K has fewer K tiles) */
} gemm_epi_linear_grad_desc;

typedef struct gemm_epi_linear_grad_handle gemm_epi_linear_grad_handle;

/*
 * Validate and plan a backward: an elementwise pass (dZ, column sums), then
 * one launch for both matrix products (and one that joins K slices, where the
 * plan has them).  dZ is rounded to ab_dtype, the type the matrix cores read;
 * dbias is summed in fp32 before that rounding, in a fixed order.  Errors as
 * above; at least one gradient must be wanted.  UNSUPPORTED as well: an
 * operand that a product reads across its rows (dA: B; dB: A and dZ) of 2 GiB
 * or more; N above 2^26; 2^24 or more work items.
 */
int gemm_epi_linear_grad_create(const gemm_epi_linear_grad_desc* desc, gemm_epi_linear_grad_handle** out);

/*
 * Enqueue the gradients.  dD is required; A exactly for dB, B exactly for dA;
 * Z and dZ exactly when act is not NONE (with NONE dD takes dZ's place); dA,
 * dB, dbias exactly when their types are set; dB_in (or NULL: 0) only with dB.
 * dZ may be dD or Z itself and dB may be dB_in itself; no other overlap of an
 * output with another tensor is allowed.  workspace as in gemm_epi_linear_run,
 * of gemm_epi_linear_grad_workspace(h) bytes.
 */
int gemm_epi_linear_grad_run(const gemm_epi_linear_grad_handle* h, const void* dD, const void* A, const void* B,
                             const void* Z, const void* dB_in, void* dZ, void* dA, void* dB, void* dbias,
                             void* workspace, int64_t workspace_bytes, void* stream);

/* The same for a forward of this alpha (gemm_epi_linear_grad_run: 1). */
int gemm_epi_linear_grad_run_alpha(const gemm_epi_linear_grad_handle* h, const void* dD, const void* A, const void* B,
                                   const void* Z, const void* dB_in, void* dZ, void* dA, void* dB, void* dbias,
                                   float alpha, void* workspace, int64_t workspace_bytes, void* stream);

/* Free a handle (NULL is fine). */
int gemm_epi_linear_grad_destroy(gemm_epi_linear_grad_handle* h);

/* Bytes of workspace a run needs (-1 for a NULL handle). */
int64_t gemm_epi_linear_grad_workspace(const gemm_epi_linear_grad_handle* h);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_EPI_LINEAR_H */
