// gemm_linear_host.hpp -- the linear layer's handle and its runs' parameters
// (gemm_linear.hip), for host code that launches kernels of its own on its plans.
#pragma once

#include "gemm_epi_linear.h"
#include "gemm_linear.hpp"
#include "gemm_linear_cost.hpp"

struct gemm_epi_linear_handle {
  gemm_epi_linear_desc d;  // strides filled in
  int variant, device, cus, grid;
  int nw;                  // few rows: waves per workgroup
  int64_t tiles_m, tiles_n, tiles, tail, kslice, items;
  int splits, group_m;
  int64_t ws_bytes;
};

namespace gemm_epi {

// gemm_epi_linear_create_variant, for rows with adapters (NULL: none).
int linear_create(const gemm_epi_linear_desc* desc, int variant, const LinearAdapters* adapters,
                  gemm_epi_linear_handle** out);

// What a run checks, and its kernels' arguments.
int linear_params(const gemm_epi_linear_handle* h, const void* A, const void* B, const void* bias,
                  const float* scale_a, const float* scale_b, const void* R, void* D, void* Z, float alpha,
                  void* workspace, int64_t workspace_bytes, LinParams* out);

// Enqueues the join of a split-K plan's slices (none: nothing).
int linear_join(const gemm_epi_linear_handle* h, const LinParams& p, hipStream_t s);

}  // namespace gemm_epi
