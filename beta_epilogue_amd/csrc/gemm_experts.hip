// gemm_experts.hip -- C ABI of the sort of tokens by expert, the way back and
// its gradient (see include/gemm_epi_experts.h): validation and launches.
#include <hip/hip_runtime.h>

#include <new>

#include "gemm_epi_experts.h"
#include "gemm_epi_host.hpp"
#include "gemm_experts.hpp"

using namespace gemm_epi;

namespace {

int check_choices(int64_t tokens, int32_t top_k, int64_t below) {
  if (tokens < 1) return fail(GEMM_EPI_ERR_INVALID_ARG, "tokens must be >= 1 (got %lld)", (long long)tokens);
  if (top_k < 1 || top_k > kMaxTopK)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "top_k must be 1 .. %d (got %d)", kMaxTopK, top_k);
  if (tokens >= below / top_k)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "%lld tokens of %d choices: too many", (long long)tokens, top_k);
  return GEMM_EPI_OK;
}

// Row stride `ld` (0: packed) of a tensor of `rows` rows.
int check_rows(const char* name, int64_t* ld, int64_t rows, int64_t cols, int type, bool used) {
  if (!used) {
    if (*ld != 0) return fail(GEMM_EPI_ERR_INVALID_ARG, "ld%s is given but the tensor is not used", name);
    return GEMM_EPI_OK;
  }
  const int es = elem_bytes(type);
  if (cols < 1) return fail(GEMM_EPI_ERR_INVALID_ARG, "cols must be >= 1 (got %lld)", (long long)cols);
  if (cols >= (int64_t(1) << 30) / es) return fail(GEMM_EPI_ERR_UNSUPPORTED, "rows of 1 GiB or more");
  if (*ld == 0) *ld = cols;
  int64_t n;
  if (*ld < cols || !mul_ok(*ld, rows, &n) || !mul_ok(n, es, &n))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "ld%s %lld: below the row's %lld elements, or the tensor beyond int64", name,
                (long long)*ld, (long long)cols);
  if (cols * es % 16 || *ld * es % 16)
    return fail(GEMM_EPI_ERR_ALIGNMENT, "rows (%lld elements) and row strides (%lld) must be multiples of 16 bytes",
                (long long)cols, (long long)*ld);
  // a thread for every 16 bytes of the tokens' rows
  if (!mul_ok(cols * es / 16 + 1, rows, &n) || n > (int64_t(1) << 32) - 256)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "%lld rows of %lld elements: more than a launch has threads for",
                (long long)rows, (long long)cols);
  return GEMM_EPI_OK;
}

int check_float(int t) {
  if (!is_type(t)) return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown dtype %d", t);
  if (!is_float_out(t)) return fail(GEMM_EPI_ERR_UNSUPPORTED, "x_dtype must be F16, BF16 or F32");
  return GEMM_EPI_OK;
}

int aligned(const void* p, unsigned bytes) {
  if ((uintptr_t)p % bytes) return fail(GEMM_EPI_ERR_ALIGNMENT, "pointer %p is not %u-byte aligned", p, bytes);
  return GEMM_EPI_OK;
}

template <class H, class D>
int finish(const D& d, H** out) {
  int device = 0, cus = 0;
  const int rc = device_query(&device, &cus);
  if (rc) return rc;
  *out = new (std::nothrow) H{d, device};
  return *out ? GEMM_EPI_OK : fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
}

}  // namespace

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
struct gemm_epi_expert_sort_handle {
  gemm_epi_expert_sort_desc d;  // strides filled in
  int device;
  int64_t chunks() const { return sort_chunks(d.tokens * d.top_k); }
  int64_t ws() const { return chunks() > 1 ? chunks() * d.experts * 4 : 0; }
};

extern "C" int gemm_epi_expert_sort_create(const gemm_epi_expert_sort_desc* desc, gemm_epi_expert_sort_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  gemm_epi_expert_sort_desc d = *desc;
  int rc = check_choices(d.tokens, d.top_k, int64_t(1) << 26);
  if (rc) return rc;
  if (d.experts < 1 || d.experts > kMaxExperts)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "experts must be 1 .. %d (got %d)", kMaxExperts, d.experts);
  if (d.ids_bits != 32 && d.ids_bits != 64) return fail(GEMM_EPI_ERR_INVALID_ARG, "ids_bits must be 32 or 64");
  if (d.scale != 0 && d.scale != 1) return fail(GEMM_EPI_ERR_INVALID_ARG, "scale must be 0 or 1");
  if (d.cols < 0) return fail(GEMM_EPI_ERR_INVALID_ARG, "cols must be >= 0 (got %lld)", (long long)d.cols);
  const bool move = d.cols > 0;
  if (!move && (d.x_dtype != GEMM_EPI_NONE || d.scale))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "x_dtype and scale without columns");
  if (move && !is_type(d.x_dtype)) return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown x_dtype %d", d.x_dtype);
  if (move && !is_float_out(d.x_dtype) && d.x_dtype != GEMM_EPI_E4M3 && d.x_dtype != GEMM_EPI_I8)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "x_dtype must be F16, BF16, F32, E4M3 or I8");
  rc = check_rows("x", &d.ldx, d.tokens, d.cols, d.x_dtype, move);
  if (!rc) rc = check_rows("y", &d.ldy, d.tokens, d.cols, d.x_dtype, move);
  int64_t n;
  if (!rc && move && (!mul_ok(d.ldy, d.tokens * d.top_k, &n) || !mul_ok(n, 4, &n)))
    rc = fail(GEMM_EPI_ERR_INVALID_ARG, "Y is beyond int64");
  return rc ? rc : finish(d, out);
}

extern "C" int gemm_epi_expert_sort_run(const gemm_epi_expert_sort_handle* h, const void* ids, const void* X,
                                        const float* scale, int32_t* offsets, int32_t* rows, void* Y,
                                        float* scale_out, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_expert_sort_desc& d = h->d;
  const bool move = d.cols > 0;
  if (!ids || !offsets || !rows) return fail(GEMM_EPI_ERR_INVALID_ARG, "ids, offsets and rows are required");
  if ((X != nullptr) != move || (Y != nullptr) != move || (scale != nullptr) != (d.scale != 0) ||
      (scale_out != nullptr) != (d.scale != 0))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "X, Y, scale and scale_out must be given exactly as the plan says");
  int rc = aligned(ids, (unsigned)d.ids_bits / 8);
  for (const void* p : {X, (const void*)Y})
    if (!rc) rc = aligned(p, 16);
  for (const void* p : {(const void*)scale, (const void*)offsets, (const void*)rows, (const void*)scale_out})
    if (!rc) rc = aligned(p, 4);
  if (rc) return rc;
  const void* in[] = {ids, X, scale};
  const void* outp[] = {offsets, rows, Y, scale_out};
  for (int i = 0; i < 4; ++i) {
    if (!outp[i]) continue;
    for (const void* p : in)
      if (p == outp[i]) return fail(GEMM_EPI_ERR_INVALID_ARG, "an output may not be an input");
    for (int j = 0; j < i; ++j)
      if (outp[j] == outp[i]) return fail(GEMM_EPI_ERR_INVALID_ARG, "two outputs share a pointer");
  }
  rc = check_workspace(workspace, workspace_bytes, h->ws());
  if (!rc) rc = check_device(h->device);
  if (rc) return rc;
  SortParams p = {};
  p.ids = ids;
  p.X = X;
  p.scale = scale;
  p.offsets = offsets;
  p.rows = rows;
  p.Y = Y;
  p.scale_out = scale_out;
  p.counts = (int32_t*)workspace;
  p.tokens = d.tokens;
  const int es = move ? elem_bytes(d.x_dtype) : 0;
  p.row_bytes = d.cols * es;
  p.ldx = d.ldx * es;
  p.ldy = d.ldy * es;
  p.top_k = d.top_k;
  p.experts = d.experts;
  p.chunks = (int32_t)h->chunks();
  p.ids64 = d.ids_bits == 64;
  (void)hipGetLastError();  // clear a stale error so the check below is ours
  launch_expert_sort(p, (hipStream_t)stream);
  return launched();
}

extern "C" int gemm_epi_expert_sort_destroy(gemm_epi_expert_sort_handle* h) {
  delete h;
  return GEMM_EPI_OK;
}

extern "C" int64_t gemm_epi_expert_sort_workspace(const gemm_epi_expert_sort_handle* h) { return h ? h->ws() : -1; }

// ---------------------------------------------------------------------------
// The way back
// ---------------------------------------------------------------------------
struct gemm_epi_expert_combine_handle {
  gemm_epi_expert_combine_desc d;  // strides filled in
  int device;
};

extern "C" int gemm_epi_expert_combine_create(const gemm_epi_expert_combine_desc* desc,
                                              gemm_epi_expert_combine_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  gemm_epi_expert_combine_desc d = *desc;
  int rc = check_choices(d.tokens, d.top_k, int64_t(1) << 31);
  if (!rc) rc = check_float(d.x_dtype);
  if (rc) return rc;
  if ((d.weights != 0 && d.weights != 1) || (d.residual != 0 && d.residual != 1))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "weights and residual must be 0 or 1");
  rc = check_rows("d", &d.ldd, d.tokens, d.cols, d.x_dtype, true);
  if (!rc) rc = check_rows("r", &d.ldr, d.tokens, d.cols, d.x_dtype, d.residual);
  if (!rc) rc = check_rows("y", &d.ldy, d.tokens, d.cols, d.x_dtype, true);
  int64_t n;
  if (!rc && (!mul_ok(d.ldy, d.tokens * d.top_k, &n) || !mul_ok(n, 4, &n)))
    rc = fail(GEMM_EPI_ERR_INVALID_ARG, "Y is beyond int64");
  return rc ? rc : finish(d, out);
}

extern "C" int gemm_epi_expert_combine_run(const gemm_epi_expert_combine_handle* h, const void* Y, const int32_t* rows,
                                           const float* weights, const void* R, void* D, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_expert_combine_desc& d = h->d;
  if (!Y || !rows || !D) return fail(GEMM_EPI_ERR_INVALID_ARG, "Y, rows and D are required");
  if ((weights != nullptr) != (d.weights != 0) || (R != nullptr) != (d.residual != 0))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "weights and R must be given exactly as the plan says");
  int rc = GEMM_EPI_OK;
  for (const void* p : {Y, R, (const void*)D})
    if (!rc) rc = aligned(p, 16);
  for (const void* p : {(const void*)rows, (const void*)weights})
    if (!rc) rc = aligned(p, 4);
  if (rc) return rc;
  if (D == Y || D == (const void*)rows || D == (const void*)weights || (D == R && d.ldd != d.ldr))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "D may be no input but R, with the same row stride");
  rc = check_device(h->device);
  if (rc) return rc;
  CombineParams p = {};
  p.Y = Y;
  p.rows = rows;
  p.weights = weights;
  p.R = R;
  p.D = D;
  p.tokens = d.tokens;
  p.cols = d.cols;
  p.ldy = d.ldy;
  p.ldd = d.ldd;
  p.ldr = d.ldr;
  p.top_k = d.top_k;
  (void)hipGetLastError();
  launch_expert_combine(d.x_dtype, p, (hipStream_t)stream);
  return launched();
}

extern "C" int gemm_epi_expert_combine_destroy(gemm_epi_expert_combine_handle* h) {
  delete h;
  return GEMM_EPI_OK;
}

struct gemm_epi_expert_combine_grad_handle {
  gemm_epi_expert_combine_grad_desc d;  // strides filled in
  int device;
};

extern "C" int gemm_epi_expert_combine_grad_create(const gemm_epi_expert_combine_grad_desc* desc,
                                                   gemm_epi_expert_combine_grad_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  gemm_epi_expert_combine_grad_desc d = *desc;
  int rc = check_choices(d.tokens, d.top_k, int64_t(1) << 31);
  if (!rc) rc = check_float(d.x_dtype);
  if (!rc) rc = check_rows("d", &d.ldd, d.tokens, d.cols, d.x_dtype, true);
  if (!rc) rc = check_rows("y", &d.ldy, d.tokens, d.cols, d.x_dtype, true);
  if (!rc) rc = check_rows("g", &d.ldg, d.tokens, d.cols, d.x_dtype, true);
  int64_t n;
  for (int64_t ld : {d.ldy, d.ldg})
    if (!rc && (!mul_ok(ld, d.tokens * d.top_k, &n) || !mul_ok(n, 4, &n)))
      rc = fail(GEMM_EPI_ERR_INVALID_ARG, "Y or dY is beyond int64");
  if (!rc && d.tokens >= (int64_t(1) << 32) / 64)
    rc = fail(GEMM_EPI_ERR_UNSUPPORTED, "%lld tokens: more than a launch has waves", (long long)d.tokens);
  return rc ? rc : finish(d, out);
}

extern "C" int gemm_epi_expert_combine_grad_run(const gemm_epi_expert_combine_grad_handle* h, const void* dD,
                                                const void* Y, const int32_t* rows, const float* weights, void* dY,
                                                float* dweights, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_expert_combine_grad_desc& d = h->d;
  if (!dD || !Y || !rows || !weights || !dY || !dweights)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dD, Y, rows, weights, dY and dweights are required");
  int rc = GEMM_EPI_OK;
  for (const void* p : {dD, Y, (const void*)dY})
    if (!rc) rc = aligned(p, 16);
  for (const void* p : {(const void*)rows, (const void*)weights, (const void*)dweights})
    if (!rc) rc = aligned(p, 4);
  if (rc) return rc;
  for (const void* p : {dD, Y, (const void*)rows, (const void*)weights})
    if (p == dY || p == (const void*)dweights) return fail(GEMM_EPI_ERR_INVALID_ARG, "an output may not be an input");
  if (dY == (void*)dweights) return fail(GEMM_EPI_ERR_INVALID_ARG, "two outputs share a pointer");
  rc = check_device(h->device);
  if (rc) return rc;
  CombineParams p = {};
  p.Y = Y;
  p.rows = rows;
  p.weights = weights;
  p.dD = dD;
  p.dY = dY;
  p.dweights = dweights;
  p.tokens = d.tokens;
  p.cols = d.cols;
  p.ldd = d.ldd;
  p.ldy = d.ldy;
  p.ldg = d.ldg;
  p.top_k = d.top_k;
  (void)hipGetLastError();
  launch_expert_combine_grad(d.x_dtype, p, (hipStream_t)stream);
  return launched();
}

extern "C" int gemm_epi_expert_combine_grad_destroy(gemm_epi_expert_combine_grad_handle* h) {
  delete h;
  return GEMM_EPI_OK;
}
