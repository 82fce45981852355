/*
 * gemm_epi_experts.h -- C ABI of a mixture of experts' operators on MI355X
 * (gfx950): tokens sorted by expert, the experts' linear layers on the sorted
 * rows, and the results brought back with the router's weights; each with its
 * backward.
 *
 * T tokens choose top_k of E experts each.  A choice outside 0 .. E - 1 is none
 * (padding, a dropped token): it has row -1, and takes no part anywhere.  The
 * others get rows 0 .. n - 1 of a sorted batch of up to T * top_k rows: expert e
 * has rows offsets[e] .. offsets[e + 1] - 1, offsets[0] = 0, n = offsets[E], and
 * within an expert the choices keep their order (t, then j).  Rows behind the
 * n-th are neither read nor written by any of the operators.
 *
 *     sort          Y[rows[t][j]] = X[t]
 *     linear        z[r] = scale_a[r] scale_b[e] A[r] . B[e]^T + bias[e]   (r: a row of e)
 *                   D[r] = act(z[r]) * U[r]     Z[r] = z[r]
 *     combine       D[t] = R[t] + sum_j weights[t][j] Y[rows[t][j]]
 *
 *     combine back  dY[rows[t][j]] = weights[t][j] dD[t]
 *                   dweights[t][j] = dD[t] . Y[rows[t][j]]
 *     linear back   g = dD * U    dZ = g * act'(Z)    dU = dD * act(Z)
 *                   dA[r] = dZ[r] . B[e]    dB[e] = dB_in[e] + dZ[e's rows]^T . A[e's rows]
 *                   dbias[e] = sum of dZ over e's rows
 *     sort back     dX[t] = dX_in[t] + sum_j dY[rows[t][j]]: combine without weights
 *
 * Sums are fp32 (int8 products int32) in an order that does not depend on how
 * workgroups run; every output is rounded once, to nearest-even.  One exception: e4m3
 * with 16-bit outputs in the tile kernels.  The fp8 matrix instructions drop bits of a
 * product far below the largest one of its group: sums in which large products cancel
 * have been off by 0.0006 of the sum of |a||b| (tests allow 0.001).
 * The few-row kernels, and fp32 outputs in any, widen e4m3 to fp16 (exactly) and keep
 * fp32's precision.
 *
 * Conventions as in gemm_epi_linear.h: status codes and gemm_epi_last_error();
 * everything that needs no device is checked at create; rows and row strides
 * are multiples of 16 bytes and base pointers 16-byte aligned (index arrays,
 * weights and scales: aligned to their elements); one immutable handle per shape, usable
 * from any host thread and stream of its device; calls enqueue on the caller's
 * stream and return; nothing is allocated in a run, so every run can be
 * captured into a graph; a workspace is the caller's and must not be shared by
 * calls that overlap in time.  What the sort wrote is trusted by the other
 * operators only so far: offsets and rows with other values give other
 * results, but no access outside the tensors.
 */
#ifndef GEMM_EPI_EXPERTS_H
#define GEMM_EPI_EXPERTS_H

#include "gemm_epi_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemm_epi_expert_sort_desc {
  int64_t tokens;      /* >= 1 */
  int64_t cols;        /* columns of X and Y; 0: only offsets and rows are made */
  int64_t ldx, ldy;    /* elements between rows; 0: cols */
  int32_t top_k;       /* choices per token, 1 .. 64 */
  int32_t experts;     /* 1 .. 1024 */
  int32_t ids_bits;    /* 32 or 64: the type of ids */
  int32_t x_dtype;     /* F16, BF16, F32, E4M3 or I8 (NONE with cols 0) */
  int32_t scale;       /* 1: one fp32 scale per row moves with it */
} gemm_epi_expert_sort_desc;

typedef struct gemm_epi_expert_sort_handle gemm_epi_expert_sort_handle;

/* Validate and plan a sort.  INVALID_ARG: sizes, codes, flags, strides.
 * ALIGNMENT: the 16-byte rule.  UNSUPPORTED: 2^26 or more choices, rows of 1 GiB
 * or more, more 16-byte pieces of X than a launch has threads (2^32). */
int gemm_epi_expert_sort_create(const gemm_epi_expert_sort_desc* desc, gemm_epi_expert_sort_handle** out);

/*
 * Enqueue offsets (experts + 1 int32), rows (tokens x top_k int32) and, with
 * cols, Y (tokens * top_k rows, of which the first n are written) from ids
 * (tokens x top_k).  scale (tokens) and scale_out (tokens * top_k) exactly when
 * the desc says so.  No output may be an input or another output.
 */
int gemm_epi_expert_sort_run(const gemm_epi_expert_sort_handle* h, const void* ids, const void* X, const float* scale,
                             int32_t* offsets, int32_t* rows, void* Y, float* scale_out, void* workspace,
                             int64_t workspace_bytes, void* stream);
int gemm_epi_expert_sort_destroy(gemm_epi_expert_sort_handle* h);
/* Bytes of workspace a run needs (-1 for a NULL handle). */
int64_t gemm_epi_expert_sort_workspace(const gemm_epi_expert_sort_handle* h);

typedef struct gemm_epi_expert_combine_desc {
  int64_t tokens, cols;     /* >= 1 */
  int64_t ldy, ldd, ldr;    /* elements between rows of Y, D and R; 0: cols */
  int32_t top_k;            /* 1 .. 64 */
  int32_t x_dtype;          /* F16, BF16 or F32: Y, D and R */
  int32_t weights;          /* 0: every weight is 1 */
  int32_t residual;         /* 1: R is added */
} gemm_epi_expert_combine_desc;

typedef struct gemm_epi_expert_combine_handle gemm_epi_expert_combine_handle;

/* Validate and plan (errors as for the sort; 2^31 or more choices). */
int gemm_epi_expert_combine_create(const gemm_epi_expert_combine_desc* desc, gemm_epi_expert_combine_handle** out);
/* Enqueue D (tokens x cols) from Y (tokens * top_k rows), rows and weights
 * (tokens x top_k, fp32).  D may be R itself (with ldd == ldr), nothing else. */
int gemm_epi_expert_combine_run(const gemm_epi_expert_combine_handle* h, const void* Y, const int32_t* rows,
                                const float* weights, const void* R, void* D, void* stream);
int gemm_epi_expert_combine_destroy(gemm_epi_expert_combine_handle* h);

typedef struct gemm_epi_expert_combine_grad_desc {
  int64_t tokens, cols;     /* >= 1 */
  int64_t ldd, ldy, ldg;    /* elements between rows of dD, Y and dY; 0: cols */
  int32_t top_k;            /* 1 .. 64 */
  int32_t x_dtype;          /* F16, BF16 or F32: dD, Y and dY */
} gemm_epi_expert_combine_grad_desc;

typedef struct gemm_epi_expert_combine_grad_handle gemm_epi_expert_combine_grad_handle;

int gemm_epi_expert_combine_grad_create(const gemm_epi_expert_combine_grad_desc* desc,
                                        gemm_epi_expert_combine_grad_handle** out);
/* Enqueue dY and dweights (0 for a choice without a row).  The residual's
 * gradient is dD.  No output may be an input or another output. */
int gemm_epi_expert_combine_grad_run(const gemm_epi_expert_combine_grad_handle* h, const void* dD, const void* Y,
                                     const int32_t* rows, const float* weights, void* dY, float* dweights,
                                     void* stream);
int gemm_epi_expert_combine_grad_destroy(gemm_epi_expert_combine_grad_handle* h);

typedef struct gemm_epi_expert_linear_desc {
  int64_t rows;         /* the sorted batch's capacity (tokens * top_k), >= 1 */
  int64_t N, K;         /* an expert's outputs and inputs, >= 1 */
  int64_t lda;          /* elements between rows of A; 0: K */
  int64_t ldd, ldu, ldz; /* of D, U and Z; 0: N */
  int32_t experts;      /* 1 .. 1024 */
  int32_t ab_dtype;     /* F16, BF16, E4M3 or I8 */
  int32_t d_dtype;      /* F16, BF16 or F32: D, U and Z */
  int32_t bias_dtype;   /* NONE, F16, BF16 or F32 */
  int32_t act;          /* GEMM_EPI_ACT_* */
  int32_t mul;          /* 1: D = act(z) * U */
  int32_t z;            /* 1: Z is written */
  int32_t scale_a;      /* 1: one fp32 scale per row */
  int32_t scale_b;      /* 1: one fp32 scale per expert and output */
} gemm_epi_expert_linear_desc;

typedef struct gemm_epi_expert_linear_handle gemm_epi_expert_linear_handle;

/* Validate and plan: a kernel for few rows per expert, which streams the weights
 * of the experts that have rows, or a tile kernel, by a cost model that takes the
 * rows as evenly spread: the desc alone decides, not where the rows went.  Kernels
 * differ in the order of their sums (e4m3: and in their precision, see above).
 * Types and errors as for gemm_epi_linear_create; an expert's bias must be a multiple
 * of 16 bytes long. */
int gemm_epi_expert_linear_create(const gemm_epi_expert_linear_desc* desc, gemm_epi_expert_linear_handle** out);

/* The same with kernel `variant` (-1: the plan's choice); one that cannot run the
 * problem is UNSUPPORTED. */
int gemm_epi_expert_linear_create_variant(const gemm_epi_expert_linear_desc* desc, int variant,
                                          gemm_epi_expert_linear_handle** out);

/*
 * Enqueue D (and Z) for rows 0 .. offsets[experts] - 1.  A is rows x K, B experts x
 * N x K (packed), bias experts x N, scale_a rows, scale_b experts x N, U, D and Z
 * rows x N.  D may be U itself (with ldd == ldu); no other overlap of an output
 * with another tensor is allowed.
 */
int gemm_epi_expert_linear_run(const gemm_epi_expert_linear_handle* h, const void* A, const void* B,
                               const int32_t* offsets, const void* bias, const float* scale_a, const float* scale_b,
                               const void* U, void* D, void* Z, void* stream);
int gemm_epi_expert_linear_destroy(gemm_epi_expert_linear_handle* h);

/* What a handle launches (tiles and grid: for the worst distribution of the rows;
 * few rows: chunks of tile_m rows by tile_n weight rows per workgroup). */
int gemm_epi_expert_linear_get_plan(const gemm_epi_expert_linear_handle* h, gemm_epi_plan* out);

/* Number of the experts' kernels and the name of one (NULL out of range). */
int gemm_epi_expert_linear_variant_count(void);
const char* gemm_epi_expert_linear_variant_name(int variant);

typedef struct gemm_epi_expert_linear_grad_desc {
  int64_t rows, N, K;   /* the forward's; all tensors packed */
  int32_t experts;
  int32_t ab_dtype;     /* F16 or BF16: dD, Z, U, dZ, dU, A and B */
  int32_t act;          /* the forward's activation */
  int32_t mul;          /* the forward's */
  int32_t da_dtype;     /* NONE (no dA), F16, BF16 or F32 */
  int32_t db_dtype;     /* NONE (no dB), F16, BF16 or F32: dB and dB_in */
  int32_t dbias_dtype;  /* NONE (no dbias), F16, BF16 or F32 */
  int32_t tile;         /* 0: the plan's choice; 64, 128 or 256: that tile */
} gemm_epi_expert_linear_grad_desc;

typedef struct gemm_epi_expert_linear_grad_handle gemm_epi_expert_linear_grad_handle;

/*
 * Validate and plan a backward (of a forward without scales): an elementwise
 * pass, then one launch for both products and dbias (and one that joins dbias of
 * many rows where there is no pass and no dB).  dZ is rounded to ab_dtype,
 * the type the matrix cores read; dbias is summed before that rounding, in a
 * fixed order.  UNSUPPORTED as well: an expert's B, or with dB the whole of A or dZ,
 * of 2 GiB or more; 2^24 or more work items.  A larger batch is several runs, each on
 * a range of rows with offsets less its first row (offsets outside a run's rows are
 * moved to their ends) and dB_in the dB before.
 */
int gemm_epi_expert_linear_grad_create(const gemm_epi_expert_linear_grad_desc* desc,
                                       gemm_epi_expert_linear_grad_handle** out);

/*
 * Enqueue the gradients.  dD and offsets are required; A exactly for dB, B exactly
 * for dA; Z and dZ exactly with an activation or mul (else dD takes dZ's place), U and dU
 * exactly with mul; dA, dB, dbias exactly when their types are set; dB_in (or NULL:
 * 0) only with dB.  Rows of dZ, dU and dA behind the last expert's are left as they
 * are; an expert without rows gets dB[e] = dB_in[e] and dbias[e] = 0.  dZ may be dD
 * or Z, dU may be U and dB may be dB_in itself; no other overlap of an output with
 * another tensor is allowed.
 */
int gemm_epi_expert_linear_grad_run(const gemm_epi_expert_linear_grad_handle* h, const void* dD, const void* A,
                                    const void* B, const int32_t* offsets, const void* Z, const void* U,
                                    const void* dB_in, void* dZ, void* dU, void* dA, void* dB, void* dbias,
                                    void* workspace, int64_t workspace_bytes, void* stream);
int gemm_epi_expert_linear_grad_destroy(gemm_epi_expert_linear_grad_handle* h);
/* Bytes of workspace a run needs (-1 for a NULL handle). */
int64_t gemm_epi_expert_linear_grad_workspace(const gemm_epi_expert_linear_grad_handle* h);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_EPI_EXPERTS_H */
