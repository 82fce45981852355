// gemm_adapters.hip -- C ABI of the linear layer with low-rank adapters (see
// include/gemm_epi_adapters.h): validation on top of the linear layer's, launches.
#include <hip/hip_runtime.h>

#include <new>

#include "gemm_adapter.hpp"
#include "gemm_epi_adapters.h"
#include "gemm_epi_host.hpp"
#include "gemm_linear_host.hpp"

using namespace gemm_epi;

namespace {
typedef void (*part_fn)(int, int, const AdapterParams&, int, hipStream_t);
part_fn part_of(int bm) {
  return bm == 256 ? launch_adapter_part<0> : bm == 192 ? launch_adapter_part<1> : bm == 128 ? launch_adapter_part<2>
                                                                                              : launch_adapter_part<3>;
}
}  // namespace

struct gemm_epi_adapter_linear_handle {
  gemm_epi_linear_handle* linear;
  int32_t rank, adapters, bm;  // bm: rows of the plan's tile, 0: few rows
  // the workspace: U, finite, and with sorted rows order, offsets and the sort's;
  // then the linear layer's
  int64_t at_finite, at_order, at_offsets, at_counts, own_bytes;
  bool sorted;
};

extern "C" int gemm_epi_adapter_linear_create_variant(const gemm_epi_adapter_linear_desc* desc, int variant,
                                                      gemm_epi_adapter_linear_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  const gemm_epi_linear_desc& d = desc->linear;
  if (desc->rank < 1 || desc->adapters < 1)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "rank and adapters must be >= 1 (got %d %d)", desc->rank, desc->adapters);
  if (desc->rank % 8) return fail(GEMM_EPI_ERR_ALIGNMENT, "rank %d must be a multiple of 8", desc->rank);
  if (desc->adapters > kMaxExperts)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "%d adapters: at most %d", desc->adapters, kMaxExperts);
  if (desc->rank > kMaxRank) return fail(GEMM_EPI_ERR_UNSUPPORTED, "rank %d: at most %d", desc->rank, kMaxRank);
  if (is_type(d.ab_dtype) && d.ab_dtype != GEMM_EPI_F16 && d.ab_dtype != GEMM_EPI_BF16)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "adapters take fp16 or bf16 operands");
  if (is_type(d.ab_dtype) && d.d_dtype != d.ab_dtype)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "with adapters D has the operands' type");
  if (d.scale_a || d.scale_b) return fail(GEMM_EPI_ERR_UNSUPPORTED, "adapters and scales of A and B");
  if (d.M >= int64_t(1) << 26) return fail(GEMM_EPI_ERR_UNSUPPORTED, "2^26 or more rows with adapters");
  // A, all up[g] together, and one down[g], are addressed with 31-bit byte offsets
  if (d.N > INT32_MAX / 2 / desc->rank / desc->adapters || d.K > INT32_MAX / 2 / desc->rank)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "up, or one adapter's down, of 2 GiB or more");
  gemm_epi_linear_handle* linear = nullptr;
  const LinearAdapters adapters = {desc->rank, desc->adapters};
  int rc = linear_create(&d, variant, &adapters, &linear);
  if (rc) return rc;
  if (linear->d.M * linear->d.lda > INT32_MAX / 2) {
    gemm_epi_linear_destroy(linear);
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "A of 2 GiB or more with adapters");
  }
  gemm_epi_plan plan;
  gemm_epi_linear_get_plan(linear, &plan);
  gemm_epi_adapter_linear_handle* h = new (std::nothrow) gemm_epi_adapter_linear_handle();
  if (!h) {
    gemm_epi_linear_destroy(linear);
    return fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
  }
  h->linear = linear;
  h->rank = desc->rank;
  h->adapters = desc->adapters;
  h->bm = plan.tile_k ? plan.tile_m : 0;
  h->sorted = adapter_sorted(d.M, desc->rank, desc->adapters);
  const int64_t chunks = sort_chunks(d.M);
  h->at_finite = up256(d.M * desc->rank * 2);
  h->at_order = h->at_finite + (h->bm ? up256((int64_t)desc->adapters * kFiniteParts) : 0);
  h->at_offsets = h->at_order + (h->sorted ? up256(d.M * 4) : 0);
  h->at_counts = h->at_offsets + (h->sorted ? up256(((int64_t)desc->adapters + 1) * 4) : 0);
  h->own_bytes = h->at_counts + (h->sorted && chunks > 1 ? up256(chunks * desc->adapters * 4) : 0);
  *out = h;
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_adapter_linear_create(const gemm_epi_adapter_linear_desc* desc,
                                              gemm_epi_adapter_linear_handle** out) {
  return gemm_epi_adapter_linear_create_variant(desc, -1, out);
}

extern "C" int gemm_epi_adapter_linear_run(const gemm_epi_adapter_linear_handle* h, const void* A, const void* B,
                                           const int32_t* ids, const void* down, const void* up, const float* scale,
                                           const void* bias, const void* R, void* D, void* Z, void* workspace,
                                           int64_t workspace_bytes, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_linear_desc& d = h->linear->d;
  if (!ids || !down || !up || !scale) return fail(GEMM_EPI_ERR_INVALID_ARG, "ids, down, up and scale are required");
  for (const void* p : {down, up})
    if ((uintptr_t)p & 15u) return fail(GEMM_EPI_ERR_ALIGNMENT, "pointer %p is not 16-byte aligned", p);
  for (const void* p : {(const void*)ids, (const void*)scale})
    if ((uintptr_t)p & 3u) return fail(GEMM_EPI_ERR_ALIGNMENT, "pointer %p is not 4-byte aligned", p);
  for (const void* p : {(const void*)ids, down, up, (const void*)scale})
    if (p == D || p == Z) return fail(GEMM_EPI_ERR_INVALID_ARG, "D and Z may not be an operand");
  int rc = check_workspace(workspace, workspace_bytes, h->own_bytes + h->linear->ws_bytes);
  if (rc) return rc;
  AdapterParams p = {};
  char* ws = (char*)workspace;
  rc = linear_params(h->linear, A, B, bias, nullptr, nullptr, R, D, Z, 1.0f, ws + h->own_bytes,
                     workspace_bytes - h->own_bytes, &p);
  if (rc) return rc;
  p.U = ws;
  p.up = up;
  p.ids = ids;
  p.finite = (const uint32_t*)(ws + h->at_finite);
  p.rank = h->rank;
  p.adapters = h->adapters;
  AdapterDownParams q = {};
  q.A = A;
  q.down = down;
  q.up = up;
  q.scale = scale;
  q.ids = ids;
  q.U = ws;
  q.finite = h->bm ? (uint8_t*)(ws + h->at_finite) : nullptr;
  q.order = h->sorted ? (int32_t*)(ws + h->at_order) : nullptr;
  q.offsets = h->sorted ? (int32_t*)(ws + h->at_offsets) : nullptr;
  q.counts = h->sorted ? (int32_t*)(ws + h->at_counts) : nullptr;
  q.M = d.M;
  q.N = d.N;
  q.K = d.K;
  q.lda = d.lda;
  q.rank = h->rank;
  q.adapters = h->adapters;
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();  // clear a stale error so the checks below are ours
  launch_adapter_down(d.ab_dtype, q, s);
  rc = launched();
  if (rc) return rc;
  if (h->bm == 0) launch_adapter_rows(d.ab_dtype, h->linear->nw, p, s);
  else part_of(h->bm)(d.ab_dtype, h->bm, p, h->linear->grid, s);
  rc = launched();
  return rc ? rc : linear_join(h->linear, p, s);
}

extern "C" int gemm_epi_adapter_linear_destroy(gemm_epi_adapter_linear_handle* h) {
  if (h) gemm_epi_linear_destroy(h->linear);
  delete h;
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_adapter_linear_get_plan(const gemm_epi_adapter_linear_handle* h, gemm_epi_plan* out) {
  clear_error();
  if (!h || !out) return fail(GEMM_EPI_ERR_INVALID_ARG, "NULL argument");
  const int rc = gemm_epi_linear_get_plan(h->linear, out);
  out->workspace_bytes += h->own_bytes;
  return rc;
}
