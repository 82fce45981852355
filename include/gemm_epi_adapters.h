/*
 * gemm_epi_adapters.h -- C ABI of the linear layer with low-rank adapters on
 * MI355X (gfx950): one shared projection of a batch whose rows belong to
 * different requests, each with an adapter of its own or none.
 *
 *     z[m] = A[m] . B^T + bias + scale[g] (A[m] . down[g]^T) . up[g]^T,  g = ids[m]
 *     D = act(z) + R            Z = z (if asked for)
 *
 * Rows whose id lies outside 0 .. adapters - 1 have no adapter.  Rows of the same
 * adapter need not lie together; they are fastest where they do (packed prompts).
 * An infinity or a NaN in one adapter's weights reaches that adapter's rows only.
 * The inner products scale[g] A[m] . down[g]^T are summed in fp32 and rounded once
 * to the operands' type, which the matrix cores read.  (fp16: one beyond 65504 is
 * infinite, also where its product with up would not be; one below 6.1e-5 is off by
 * up to 3e-8, half of a subnormal step.)  Everything else is as in
 * gemm_epi_linear.h, whose conventions hold.  Adapters of a smaller rank are padded
 * with zeros.
 */
#ifndef GEMM_EPI_ADAPTERS_H
#define GEMM_EPI_ADAPTERS_H

#include "gemm_epi_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemm_epi_adapter_linear_desc {
  gemm_epi_linear_desc linear; /* the projection: ab_dtype F16 or BF16, D of the
                                  same type, no scale_a and scale_b */
  int32_t rank;                /* 8 .. 128, a multiple of 8 */
  int32_t adapters;            /* 1 .. 1024 */
} gemm_epi_adapter_linear_desc;

typedef struct gemm_epi_adapter_linear_handle gemm_epi_adapter_linear_handle;

/* Validate and plan: the projection's plan, chosen with the work that the adapters add
 * where each adapter's rows lie together (errors as for
 * gemm_epi_linear_create; 2^26 or more rows, and A, up or one adapter's down of 2
 * GiB or more, are UNSUPPORTED). */
int gemm_epi_adapter_linear_create(const gemm_epi_adapter_linear_desc* desc, gemm_epi_adapter_linear_handle** out);

/* The same with the linear layer's kernel `variant` (-1: its choice). */
int gemm_epi_adapter_linear_create_variant(const gemm_epi_adapter_linear_desc* desc, int variant,
                                           gemm_epi_adapter_linear_handle** out);

/*
 * Enqueue D (and Z).  ids: M int32; down: adapters x rank x K and up: adapters x N x
 * rank, packed, of A's type; scale: adapters fp32.  A, B, bias, R, D and Z as in
 * gemm_epi_linear_run; no output may be an operand.  workspace: at least
 * plan.workspace_bytes of device memory at a 256-byte boundary.
 */
int gemm_epi_adapter_linear_run(const gemm_epi_adapter_linear_handle* h, const void* A, const void* B,
                                const int32_t* ids, const void* down, const void* up, const float* scale,
                                const void* bias, const void* R, void* D, void* Z, void* workspace,
                                int64_t workspace_bytes, void* stream);

/* Free a handle (NULL is fine). */
int gemm_epi_adapter_linear_destroy(gemm_epi_adapter_linear_handle* h);

/* The projection's plan, with this call's workspace. */
int gemm_epi_adapter_linear_get_plan(const gemm_epi_adapter_linear_handle* h, gemm_epi_plan* out);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_EPI_ADAPTERS_H */
