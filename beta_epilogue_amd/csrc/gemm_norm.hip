// gemm_norm.hip -- C ABI of the root-mean-square norm and its backward (see
// include/gemm_epi_norm.h): validation and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <new>

#include "gemm_epi_host.hpp"
#include "gemm_epi_norm.h"
#include "gemm_linear.hpp"
#include "gemm_norm.hpp"

using namespace gemm_epi;

namespace {

int check_sizes(int64_t rows, int64_t cols, float eps) {
  if (rows < 1 || cols < 1)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "rows and cols must be >= 1 (got %lld %lld)", (long long)rows,
                (long long)cols);
  if (!std::isfinite(eps) || eps < 0.0f) return fail(GEMM_EPI_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (cols > kNormMaxCols)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "%lld columns: at most %lld", (long long)cols, (long long)kNormMaxCols);
  if (rows >= (int64_t(1) << 31)) return fail(GEMM_EPI_ERR_UNSUPPORTED, "2^31 or more rows");
  return GEMM_EPI_OK;
}

// What a run adds to a row's mean square: without an eps 2^-149, which changes no
// normal number and keeps 1 / sqrt finite, so that a row of zeros is 0 times a
// number rather than 0 times infinity.
float run_eps(float eps) { return eps > 0x1p-149f ? eps : 0x1p-149f; }

int check_stride(const char* name, int64_t* ld, int64_t rows, int64_t cols, bool used) {
  if (!used) {
    if (*ld != 0) return fail(GEMM_EPI_ERR_INVALID_ARG, "ld%s is given but the tensor is not used", name);
    return GEMM_EPI_OK;
  }
  if (*ld == 0) *ld = cols;
  int64_t n;
  if (*ld < cols || !mul_ok(*ld, rows, &n) || !mul_ok(n, 4, &n))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "ld%s %lld: below the row's %lld elements, or the tensor beyond int64", name,
                (long long)*ld, (long long)cols);
  return GEMM_EPI_OK;
}

int check_x(int x, int w) {
  if (!is_type(x) || !is_type(w)) return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown dtype");
  if (!is_float_out(x)) return fail(GEMM_EPI_ERR_UNSUPPORTED, "x_dtype must be F16, BF16 or F32");
  if (w != x && w != GEMM_EPI_F32) return fail(GEMM_EPI_ERR_UNSUPPORTED, "weight_dtype must be x_dtype or F32");
  return GEMM_EPI_OK;
}

int check_align(const void* p, int type) {
  if ((uintptr_t)p % (unsigned)elem_bytes(type))
    return fail(GEMM_EPI_ERR_ALIGNMENT, "pointer %p is not aligned to its elements", p);
  return GEMM_EPI_OK;
}

}  // namespace

struct gemm_epi_rmsnorm_handle {
  gemm_epi_rmsnorm_desc d;  // strides filled in
  int device;
};

extern "C" int gemm_epi_rmsnorm_create(const gemm_epi_rmsnorm_desc* desc, gemm_epi_rmsnorm_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  gemm_epi_rmsnorm_desc d = *desc;
  int rc = check_sizes(d.rows, d.cols, d.eps);
  if (!rc) rc = check_x(d.x_dtype, d.weight_dtype);
  if (rc) return rc;
  if (!is_type(d.y_dtype)) return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown dtype");
  if (d.y_dtype != d.x_dtype && d.y_dtype != GEMM_EPI_E4M3 && d.y_dtype != GEMM_EPI_I8)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "y_dtype must be x_dtype, E4M3 or I8");
  if (d.residual != 0 && d.residual != 1) return fail(GEMM_EPI_ERR_INVALID_ARG, "residual must be 0 or 1");
  rc = check_stride("x", &d.ldx, d.rows, d.cols, true);
  if (!rc) rc = check_stride("r", &d.ldr, d.rows, d.cols, d.residual);
  if (!rc) rc = check_stride("h", &d.ldh, d.rows, d.cols, d.residual);
  if (!rc) rc = check_stride("y", &d.ldy, d.rows, d.cols, true);
  int device = 0, cus = 0;
  if (!rc) rc = device_query(&device, &cus);
  if (rc) return rc;
  gemm_epi_rmsnorm_handle* h = new (std::nothrow) gemm_epi_rmsnorm_handle{d, device};
  if (!h) return fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
  *out = h;
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_rmsnorm_run(const gemm_epi_rmsnorm_handle* h, const void* x, const void* r, const void* weight,
                                    void* Y, void* H, float* scale, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_rmsnorm_desc& d = h->d;
  const bool q = d.y_dtype == GEMM_EPI_E4M3 || d.y_dtype == GEMM_EPI_I8;
  if (!x || !weight || !Y) return fail(GEMM_EPI_ERR_INVALID_ARG, "x, weight and Y are required");
  if ((r != nullptr) != (d.residual != 0) || (H && !r))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "r must be given exactly with a residual, H only with one");
  if ((scale != nullptr) != q) return fail(GEMM_EPI_ERR_INVALID_ARG, "scale must be given exactly for an 8-bit Y");
  int rc = check_align(x, d.x_dtype);
  if (!rc) rc = check_align(r, d.x_dtype);
  if (!rc) rc = check_align(weight, d.weight_dtype);
  if (!rc) rc = check_align(H, d.x_dtype);
  if (!rc) rc = check_align(Y, d.y_dtype);
  if (!rc) rc = check_align(scale, GEMM_EPI_F32);
  if (rc) return rc;
  if ((H == x && H && d.ldh != d.ldx) || (H == r && H && d.ldh != d.ldr))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "H may be x or r only with the same row stride");
  if ((Y == x && (q || d.ldy != d.ldx)) || (Y == r && (q || d.ldy != d.ldr)))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "Y may be x or r only with the same type and row stride");
  if (Y == H || Y == weight || (H && H == weight) || (scale && (scale == Y || scale == H || scale == x ||
                                                                scale == r || scale == weight)))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "an output may not be the weight or another output");
  rc = check_device(h->device);
  if (rc) return rc;
  NormParams p;
  p.x = x;
  p.r = r;
  p.w = weight;
  p.y = Y;
  p.h = H;
  p.scale = scale;
  p.rows = d.rows;
  p.cols = d.cols;
  p.ldx = d.ldx;
  p.ldr = d.ldr;
  p.ldh = d.ldh;
  p.ldy = d.ldy;
  p.w_f32 = d.weight_dtype == GEMM_EPI_F32 ? 1 : 0;
  p.eps = run_eps(d.eps);
  (void)hipGetLastError();  // clear a stale error so the check below is ours
  launch_rmsnorm(d.x_dtype, d.y_dtype, p, (hipStream_t)stream);
  return launched();
}

extern "C" int gemm_epi_rmsnorm_destroy(gemm_epi_rmsnorm_handle* h) {
  delete h;
  return GEMM_EPI_OK;
}

struct gemm_epi_rmsnorm_grad_handle {
  gemm_epi_rmsnorm_grad_desc d;  // strides filled in
  int device, grid;
  int64_t ws_bytes;
};

extern "C" int gemm_epi_rmsnorm_grad_create(const gemm_epi_rmsnorm_grad_desc* desc,
                                            gemm_epi_rmsnorm_grad_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  gemm_epi_rmsnorm_grad_desc d = *desc;
  int rc = check_sizes(d.rows, d.cols, d.eps);
  if (!rc) rc = check_x(d.x_dtype, d.weight_dtype);
  if (rc) return rc;
  if (d.dweight_dtype != GEMM_EPI_NONE && !is_float_out(d.dweight_dtype))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dweight_dtype must be NONE, F16, BF16 or F32");
  rc = check_stride("y", &d.ldy, d.rows, d.cols, true);
  if (!rc) rc = check_stride("h", &d.ldh, d.rows, d.cols, true);
  if (!rc) rc = check_stride("i", &d.ldi, d.rows, d.cols, true);
  if (!rc) rc = check_stride("o", &d.ldo, d.rows, d.cols, true);
  int device = 0, cus = 0;
  if (!rc) rc = device_query(&device, &cus);
  if (rc) return rc;
  const int grid = rmsnorm_grad_grid(d.rows, d.cols, cus);
  const bool direct = grid == 1 && d.dweight_dtype == GEMM_EPI_F32;  // the only workgroup's sums are dweight
  const int64_t ws = d.dweight_dtype == GEMM_EPI_NONE || direct ? 0 : (int64_t)grid * d.cols * 4;
  gemm_epi_rmsnorm_grad_handle* h = new (std::nothrow) gemm_epi_rmsnorm_grad_handle{d, device, grid, ws};
  if (!h) return fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
  *out = h;
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_rmsnorm_grad_run(const gemm_epi_rmsnorm_grad_handle* h, const void* dY, const void* H,
                                         const void* weight, const void* dH_in, void* dH, void* dweight,
                                         void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_rmsnorm_grad_desc& d = h->d;
  if (!dY || !H || !weight || !dH) return fail(GEMM_EPI_ERR_INVALID_ARG, "dY, H, weight and dH are required");
  if ((dweight != nullptr) != (d.dweight_dtype != GEMM_EPI_NONE))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dweight must be given exactly when dweight_dtype is set");
  int rc = check_align(dY, d.x_dtype);
  if (!rc) rc = check_align(H, d.x_dtype);
  if (!rc) rc = check_align(weight, d.weight_dtype);
  if (!rc) rc = check_align(dH_in, d.x_dtype);
  if (!rc) rc = check_align(dH, d.x_dtype);
  if (!rc && dweight) rc = check_align(dweight, d.dweight_dtype);
  if (rc) return rc;
  if ((dH == dY && d.ldo != d.ldy) || (dH == H && d.ldo != d.ldh) || (dH == dH_in && d.ldo != d.ldi))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dH may be dY, H or dH_in only with the same row stride");
  if (dH == weight || (dweight && (dweight == dY || dweight == H || dweight == weight || dweight == dH_in ||
                                   dweight == dH)))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "an output may not be the weight, and dweight no other tensor");
  rc = check_workspace(workspace, workspace_bytes, h->ws_bytes);
  if (!rc) rc = check_device(h->device);
  if (rc) return rc;
  NormGradParams p;
  p.dy = dY;
  p.h = H;
  p.w = weight;
  p.dh_in = dH_in;
  p.dh = dH;
  const bool direct = dweight && h->ws_bytes == 0;
  p.partial = direct ? (float*)dweight : dweight ? (float*)workspace : nullptr;
  p.rows = d.rows;
  p.cols = d.cols;
  p.ldy = d.ldy;
  p.ldh = d.ldh;
  p.ldi = d.ldi;
  p.ldo = d.ldo;
  p.w_f32 = d.weight_dtype == GEMM_EPI_F32 ? 1 : 0;
  p.eps = run_eps(d.eps);
  (void)hipGetLastError();  // clear a stale error so the checks below are ours
  launch_rmsnorm_grad(d.x_dtype, p, h->grid, (hipStream_t)stream);
  rc = launched();
  if (rc || !dweight || direct) return rc;
  launch_colsum(p.partial, h->grid, d.cols, dweight, d.dweight_dtype, (hipStream_t)stream);
  return launched();
}

extern "C" int gemm_epi_rmsnorm_grad_destroy(gemm_epi_rmsnorm_grad_handle* h) {
  delete h;
  return GEMM_EPI_OK;
}

extern "C" int64_t gemm_epi_rmsnorm_grad_workspace(const gemm_epi_rmsnorm_grad_handle* h) {
  return h ? h->ws_bytes : -1;
}
