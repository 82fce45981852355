// gemm_linear.hip -- C ABI of the linear layer and its backward (see
// include/gemm_epi_linear.h): validation, kernel choice, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <new>

#include "gemm_epi_host.hpp"
#include "gemm_epi_linear.h"
#include "gemm_epi_plan.hpp"
#include "gemm_epi_prep.hpp"
#include "gemm_linear.hpp"

using namespace gemm_epi;

namespace {

struct LinearVariant {
  const char* name;
  int part, ab, bm, bn, bk, lds;
};
#define X(PART, AB, BM, BN, BL, NAME) \
  {NAME, PART, AB, BM, BN, LinearCfg<AB, BM, BN, BL>::BK, LinearCfg<AB, BM, BN, BL>::LDS_BYTES},
const LinearVariant kLinear[] = {
#include "gemm_linear_variants.inc"
};
#undef X
constexpr int kTiles = (int)(sizeof kLinear / sizeof kLinear[0]);
constexpr int kRowsVariant = kTiles;  // the few-row kernels, one entry
constexpr int kThreads = 256, kRowsThreads = 512;

typedef void (*part_fn)(int, const LinParams&, int, hipStream_t);
const part_fn kParts[kLinearParts] = {launch_linear_part<0>, launch_linear_part<1>, launch_linear_part<2>,
                                      launch_linear_part<3>, launch_linear_part<4>, launch_linear_part<5>,
                                      launch_linear_part<6>, launch_linear_part<7>};

// Row stride `ld` (0: packed) of a tensor with `cols` elements of `es` bytes
// per row; a stride of a tensor that is not there must be 0.
int check_stride(const char* name, int64_t* ld, int64_t cols, int es, bool used) {
  if (!used) {
    if (*ld != 0) return fail(GEMM_EPI_ERR_INVALID_ARG, "ld%s is given but the tensor is not used", name);
    return GEMM_EPI_OK;
  }
  if (*ld == 0) *ld = cols;
  if (*ld < cols)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "ld%s %lld is below the row's %lld elements", name, (long long)*ld,
                (long long)cols);
  // checked before any product: 256 rows stay within 31-bit byte offsets
  if (*ld >= (int64_t(1) << 31) / 256 / es)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "rows of %lld elements are too long for 31-bit tile offsets",
                (long long)*ld);
  if (cols * es % 16 || *ld * es % 16)
    return fail(GEMM_EPI_ERR_ALIGNMENT, "rows (%lld elements) and row strides (%lld) must be multiples of 16 bytes",
                (long long)cols, (long long)*ld);
  return GEMM_EPI_OK;
}

bool flag_ok(int f) { return f == 0 || f == 1; }

}  // namespace

struct gemm_epi_linear_handle {
  gemm_epi_linear_desc d;  // strides filled in
  int variant, device, cus, grid;
  int nb, rb;              // few rows: token and weight blocks
  int64_t tiles_m, tiles_n, tiles, tail, kslice, items;
  int splits, group_m;
  bool widen;              // e4m3 runs as fp16 copies
  int64_t prep_off, ws_bytes;
};

static int validate_linear(gemm_epi_linear_desc* d) {
  if (d->M < 1 || d->N < 1 || d->K < 1)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "M, N, K must be >= 1 (got %lld %lld %lld)", (long long)d->M,
                (long long)d->N, (long long)d->K);
  if (!is_type(d->ab_dtype) || d->ab_dtype == GEMM_EPI_F32 || d->ab_dtype == GEMM_EPI_I32)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "ab_dtype must be F16, BF16, E4M3 or I8");
  if (d->ab_dtype == GEMM_EPI_E5M2 || d->ab_dtype == GEMM_EPI_U8)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "the linear layer has no e5m2 or uint8 form");
  if (!is_float_out(d->d_dtype)) return fail(GEMM_EPI_ERR_INVALID_ARG, "d_dtype must be F16, BF16 or F32");
  if (d->bias_dtype != GEMM_EPI_NONE && !is_float_out(d->bias_dtype))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "bias_dtype must be NONE, F16, BF16 or F32");
  if (d->act < GEMM_EPI_ACT_NONE || d->act > GEMM_EPI_ACT_SILU)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown activation %d", d->act);
  if (!flag_ok(d->residual) || !flag_ok(d->z) || !flag_ok(d->scale_a) || !flag_ok(d->scale_b))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "residual, z, scale_a and scale_b must be 0 or 1");
  if (d->splits < 0) return fail(GEMM_EPI_ERR_INVALID_ARG, "splits must be >= 0 (got %d)", d->splits);
  // (e4m3 operands may be widened to two bytes)
  const int es = elem_bytes(d->ab_dtype), ds = elem_bytes(d->d_dtype);
  int rc = check_stride("a", &d->lda, d->K, es, true);
  if (!rc) rc = check_stride("b", &d->ldb, d->K, es, true);
  if (!rc) rc = check_stride("d", &d->ldd, d->N, ds, true);
  if (!rc) rc = check_stride("r", &d->ldr, d->N, ds, d->residual);
  if (!rc) rc = check_stride("z", &d->ldz, d->N, ds, d->z);
  if (rc) return rc;
  if (std::max(d->lda, d->ldb) >= (int64_t(1) << 31) / 256 / 2)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "K too large for 31-bit tile offsets");
  // partial sums are fp32 rows of a tile; row and column numbers are 32-bit
  if (d->M >= (int64_t(1) << 31) - 512 || d->N >= (int64_t(1) << 31) - 512)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "M and N must be below 2^31 - 512");
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_linear_create_variant(const gemm_epi_linear_desc* desc, int variant,
                                              gemm_epi_linear_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  gemm_epi_linear_desc d = *desc;
  int rc = validate_linear(&d);
  if (rc) return rc;
  if (variant < -1 || variant > kRowsVariant)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "variant %d out of range", variant);
  const bool widened = d.ab_dtype == GEMM_EPI_E4M3 && d.d_dtype == GEMM_EPI_F32;
  const int kernel_ab = widened ? (int)GEMM_EPI_F16 : d.ab_dtype;
  if (variant == kRowsVariant ? d.M > kRowsMax : variant >= 0 && kLinear[variant].ab != kernel_ab)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "variant %s cannot run this problem", gemm_epi_linear_variant_name(variant));
  int device = 0, cus = 0;
  rc = device_query(&device, &cus);
  if (rc) return rc;

  const PlanProblem pp{d.M, d.N, d.K, 1, (double)elem_bytes(d.d_dtype) * (1 + d.residual + d.z), true};
  auto find_tile = [&](int bm, int bn) {
    for (int i = 0; i < kTiles; ++i)
      if (kLinear[i].bm == bm && kLinear[i].bn == bn && kLinear[i].ab == kernel_ab) return i;
    return -1;
  };
  auto model = [&](int i) { return split_choice(kLinear[i].bm, kLinear[i].bn, kLinear[i].bk, pp, cus); };
  if (variant == -1) {
    if (d.M <= kRowsMax) {
      variant = kRowsVariant;
    } else {
      // the GEMM plan's rule (gemm_epi_create) on the same tile shapes
      variant = find_tile(256, 256);
      const int64_t big = ((d.M + 255) / 256) * ((d.N + 255) / 256);
      if (d.splits == 0 && big * 4 <= cus) {
        variant = find_tile(128, 128);
      } else if (d.splits == 0 && big % cus != 0) {
        double best = 0.95 * model(variant).us;
        for (const int cand : {find_tile(192, 256), find_tile(128, 256)}) {
          const double t = model(cand).us;
          if (t < best) {
            best = t;
            variant = cand;
          }
        }
      }
    }
  }

  gemm_epi_linear_handle* h = new (std::nothrow) gemm_epi_linear_handle();
  if (!h) return fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
  h->d = d;
  h->variant = variant;
  h->device = device;
  h->cus = cus;
  h->splits = 1;
  if (variant == kRowsVariant) {
    h->nb = d.M <= 16 ? 1 : d.M <= 32 ? 2 : 4;
    // two weight blocks halve the token traffic per weight byte, once there
    // are workgroups for every compute unit
    h->rb = (d.N + 31) / 32 >= cus ? 2 : 1;
    h->tiles_m = 1;
    h->tiles_n = (d.N + 16 * h->rb - 1) / (16 * h->rb);
    h->tiles = h->items = h->tiles_n;
    h->grid = (int)h->tiles_n;
    *out = h;
    return GEMM_EPI_OK;
  }
  const LinearVariant& v = kLinear[variant];
  h->tiles_m = (d.M + v.bm - 1) / v.bm;
  h->tiles_n = (d.N + v.bn - 1) / v.bn;
  h->tiles = h->tiles_m * h->tiles_n;
  h->group_m = h->tiles_n > 32 ? 8 : 4;
  const int64_t ktiles = (d.K + v.bk - 1) / v.bk;
  int64_t splits = 1;
  if (d.splits >= 1) {
    splits = std::min<int64_t>(d.splits, ktiles);
    h->tail = h->tiles;
  } else {
    const SplitChoice c = model(variant);
    splits = c.splits;
    h->tail = c.tail;
  }
  h->kslice = ((ktiles + splits - 1) / splits) * v.bk;
  h->splits = (int)((d.K + h->kslice - 1) / h->kslice);
  if (h->splits == 1) {
    h->kslice = d.K;
    h->tail = 0;
  }
  h->items = h->tiles - h->tail + h->tail * h->splits;
  if (h->tiles >= (int64_t(1) << 31) || h->items >= (int64_t(1) << 31)) {
    delete h;
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "2^31 or more work items (tiles and K slices)");
  }
  h->grid = (int)std::min<int64_t>(h->items, cus);
  h->ws_bytes = h->splits > 1 ? h->splits * h->tail * v.bm * v.bn * 4 : 0;
  h->widen = widened;
  h->prep_off = up256(h->ws_bytes);
  // copies keep the row strides
  if (widened) h->ws_bytes = h->prep_off + up256(d.M * d.lda * 2) + up256(d.N * d.ldb * 2);
  *out = h;
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_linear_create(const gemm_epi_linear_desc* desc, gemm_epi_linear_handle** out) {
  return gemm_epi_linear_create_variant(desc, -1, out);
}

extern "C" int gemm_epi_linear_run(const gemm_epi_linear_handle* h, const void* A, const void* B, const void* bias,
                                   const float* scale_a, const float* scale_b, const void* R, void* D, void* Z,
                                   float alpha, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_linear_desc& d = h->d;
  if (!A || !B || !D) return fail(GEMM_EPI_ERR_INVALID_ARG, "A, B and D are required");
  if ((bias != nullptr) != (d.bias_dtype != GEMM_EPI_NONE) || (scale_a != nullptr) != (d.scale_a != 0) ||
      (scale_b != nullptr) != (d.scale_b != 0) || (R != nullptr) != (d.residual != 0) || (Z != nullptr) != (d.z != 0))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "bias, scale_a, scale_b, R and Z must be given exactly as the plan says");
  for (const void* p : {A, B, bias, (const void*)scale_a, (const void*)scale_b, R, (const void*)D, (const void*)Z})
    if ((uintptr_t)p & 15u) return fail(GEMM_EPI_ERR_ALIGNMENT, "pointer %p is not 16-byte aligned", p);
  if (D == R && d.ldd != d.ldr) return fail(GEMM_EPI_ERR_INVALID_ARG, "D may be R only with the same row stride");
  if (D == Z || (Z && Z == R)) return fail(GEMM_EPI_ERR_INVALID_ARG, "Z may not be D or R");
  for (const void* p : {A, B, bias, (const void*)scale_a, (const void*)scale_b})
    if (p && (p == D || p == Z)) return fail(GEMM_EPI_ERR_INVALID_ARG, "D and Z may not be an operand");
  int rc = check_workspace(workspace, workspace_bytes, h->ws_bytes);
  if (!rc) rc = check_device(h->device);
  if (rc) return rc;

  LinParams p = {};
  p.A = A;
  p.B = B;
  p.D = D;
  p.M = d.M;
  p.N = d.N;
  p.K = d.K;
  p.alpha = alpha;
  p.d_dtype = d.d_dtype;
  p.scale_a = scale_a;
  p.scale_b = scale_b;
  p.bias = bias;
  p.R = R;
  p.Z = Z;
  p.lda = d.lda;
  p.ldb = d.ldb;
  p.ldd = d.ldd;
  p.ldr = d.ldr;
  p.ldz = d.ldz;
  p.bias_dtype = d.bias_dtype;
  p.act = d.act;
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();  // clear a stale error so the checks below are ours
  if (h->variant == kRowsVariant) {
    launch_linear_rows(d.ab_dtype, h->nb, h->rb, p, s);
    return launched();
  }
  const LinearVariant& v = kLinear[h->variant];
  if (h->widen) {
    // fp16 copies (exact) from the first row's first byte to the last row's
    // last one; what lies between the rows is copied along and never used
    uint16_t* wa = (uint16_t*)((char*)workspace + h->prep_off);
    uint16_t* wb = (uint16_t*)((char*)wa + up256(d.M * d.lda * 2));
    launch_f8_widen((const uint8_t*)A, (d.M - 1) * d.lda + d.K, false, wa, s);
    launch_f8_widen((const uint8_t*)B, (d.N - 1) * d.ldb + d.K, false, wb, s);
    p.A = wa;
    p.B = wb;
  }
  p.tiles_total = (int32_t)h->items;
  p.L = 1;
  p.tiles_m = (int32_t)h->tiles_m;
  p.tiles_n = (int32_t)h->tiles_n;
  p.group_m = h->group_m;
  p.xcd_remap = h->grid % 8 == 0 ? 1 : 0;
  p.dp_tiles = (int32_t)(h->tiles - h->tail);
  p.tail_tiles = (int32_t)h->tail;
  p.splits = h->splits;
  p.kslice = h->kslice;
  p.ws = workspace;
  kParts[v.part](h->variant, p, h->grid, s);
  rc = launched();
  if (rc || h->splits == 1) return rc;
  const int64_t blocks = (h->tail * v.bm * v.bn / 4 + 255) / 256;
  launch_linear_splitk(p, v.bm, v.bn, d.ab_dtype == GEMM_EPI_I8, (int)std::min<int64_t>(blocks, (int64_t)h->cus * 8),
                       s);
  return launched();
}

extern "C" int gemm_epi_linear_destroy(gemm_epi_linear_handle* h) {
  delete h;
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_linear_get_plan(const gemm_epi_linear_handle* h, gemm_epi_plan* out) {
  clear_error();
  if (!h || !out) return fail(GEMM_EPI_ERR_INVALID_ARG, "NULL argument");
  std::memset(out, 0, sizeof *out);
  out->variant = h->variant;
  if (h->variant == kRowsVariant) {
    out->tile_m = 16 * h->nb;
    out->tile_n = 16 * h->rb;
    out->threads = kRowsThreads;
    out->lds_bytes = kRowsThreads * h->nb * h->rb * 16;
  } else {
    const LinearVariant& v = kLinear[h->variant];
    out->tile_m = v.bm;
    out->tile_n = v.bn;
    out->tile_k = v.bk;
    out->threads = kThreads;
    out->lds_bytes = v.lds;
  }
  out->grid = h->grid;
  out->tiles = h->tiles;
  out->cus = h->cus;
  out->splits = h->splits;
  out->workspace_bytes = h->ws_bytes;
  out->split_tiles = h->splits > 1 ? h->tail : 0;
  std::snprintf(out->name, sizeof out->name, "%s", gemm_epi_linear_variant_name(h->variant));
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_linear_variant_count(void) { return kTiles + 1; }

extern "C" const char* gemm_epi_linear_variant_name(int variant) {
  if (variant < 0 || variant > kRowsVariant) return nullptr;
  return variant == kRowsVariant ? "linear_rows" : kLinear[variant].name;
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
struct gemm_epi_linear_grad_handle {
  gemm_epi_linear_grad_desc d;
  int device;
  int chunk;                          // rows per partial column sum
  int64_t partial_bytes, ws_bytes;    // the products' workspace follows the partial sums
  gemm_epi_handle *da = nullptr, *db = nullptr;
};

extern "C" int gemm_epi_linear_grad_create(const gemm_epi_linear_grad_desc* desc, gemm_epi_linear_grad_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  const gemm_epi_linear_grad_desc& d = *desc;
  if (d.M < 1 || d.N < 1 || d.K < 1)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "M, N, K must be >= 1 (got %lld %lld %lld)", (long long)d.M, (long long)d.N,
                (long long)d.K);
  if (!is_type(d.ab_dtype)) return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown ab_dtype %d", d.ab_dtype);
  if (d.ab_dtype != GEMM_EPI_F16 && d.ab_dtype != GEMM_EPI_BF16)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "the backward takes fp16 or bf16 tensors");
  if (d.act < GEMM_EPI_ACT_NONE || d.act > GEMM_EPI_ACT_SILU)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown activation %d", d.act);
  for (int t : {d.da_dtype, d.db_dtype, d.dbias_dtype})
    if (t != GEMM_EPI_NONE && !is_float_out(t))
      return fail(GEMM_EPI_ERR_INVALID_ARG, "a gradient's type must be NONE, F16, BF16 or F32");
  if (d.da_dtype == GEMM_EPI_NONE && d.db_dtype == GEMM_EPI_NONE && d.dbias_dtype == GEMM_EPI_NONE)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "no gradient is wanted");
  int64_t mn, t;
  if (!mul_ok(d.M, d.N, &mn) || !mul_ok(mn, 4, &t))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "tensor byte sizes overflow int64");
  if (d.N % 8) return fail(GEMM_EPI_ERR_ALIGNMENT, "rows of dD (%lld elements) must be multiples of 16 bytes",
                           (long long)d.N);
  if (d.N >= (int64_t(1) << 31) - 512)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "N must be below 2^31 - 512");

  gemm_epi_linear_grad_handle* h = new (std::nothrow) gemm_epi_linear_grad_handle();
  if (!h) return fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
  h->d = d;
  // 64 rows per partial sum; more where 2^16 chunks would not do (the grid's
  // second dimension)
  const int64_t chunk = std::max<int64_t>(64, (d.M + 65534) / 65535);
  int rc = GEMM_EPI_OK;
  if (chunk >= (int64_t(1) << 30)) rc = fail(GEMM_EPI_ERR_UNSUPPORTED, "M is too large");
  h->chunk = (int)chunk;
  int64_t products = 0;
  gemm_epi_desc g = {};
  g.L = 1;
  g.ab_dtype = d.ab_dtype;
  g.cd_major = GEMM_EPI_MAJOR_N;
  if (!rc && d.da_dtype != GEMM_EPI_NONE) {  // M x K over N: B holds its columns contiguous
    g.M = d.M, g.N = d.K, g.K = d.N;
    g.a_major = GEMM_EPI_MAJOR_K, g.b_major = GEMM_EPI_MAJOR_N;
    g.c_dtype = GEMM_EPI_NONE, g.d_dtype = d.da_dtype;
    rc = gemm_epi_create(&g, &h->da);
    if (!rc) products = std::max(products, handle_workspace(h->da));
  }
  if (!rc && d.db_dtype != GEMM_EPI_NONE) {  // N x K over M: both operands contiguous along their rows
    g.M = d.N, g.N = d.K, g.K = d.M;
    g.a_major = GEMM_EPI_MAJOR_M, g.b_major = GEMM_EPI_MAJOR_N;
    g.c_dtype = d.db_dtype, g.d_dtype = d.db_dtype;
    rc = gemm_epi_create(&g, &h->db);
    if (!rc) products = std::max(products, handle_workspace(h->db));
  }
  int cus = 0;
  if (!rc) rc = device_query(&h->device, &cus);
  if (rc) {
    gemm_epi_linear_grad_destroy(h);
    return rc;
  }
  if (d.dbias_dtype != GEMM_EPI_NONE) h->partial_bytes = up256((d.M + chunk - 1) / chunk * d.N * 4);
  h->ws_bytes = h->partial_bytes + products;
  *out = h;
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_linear_grad_run(const gemm_epi_linear_grad_handle* h, const void* dD, const void* A,
                                        const void* B, const void* Z, const void* dB_in, void* dZ, void* dA, void* dB,
                                        void* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_linear_grad_desc& d = h->d;
  const bool act = d.act != GEMM_EPI_ACT_NONE;
  if (!dD) return fail(GEMM_EPI_ERR_INVALID_ARG, "dD is required");
  if ((Z != nullptr) != act || (dZ != nullptr) != act)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "Z and dZ must be given exactly with an activation");
  if ((dA != nullptr) != (h->da != nullptr) || (B != nullptr) != (h->da != nullptr))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dA and B must be given exactly when da_dtype is set");
  if ((dB != nullptr) != (h->db != nullptr) || (A != nullptr) != (h->db != nullptr) || (dB_in && !dB))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dB and A (and dB_in) must be given exactly when db_dtype is set");
  if ((dbias != nullptr) != (d.dbias_dtype != GEMM_EPI_NONE))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dbias must be given exactly when dbias_dtype is set");
  const void* in[] = {dD, Z, A, B, dB_in};
  const void* outp[] = {dZ, dA, dB, dbias};
  for (const void* p : in)
    if ((uintptr_t)p & 15u) return fail(GEMM_EPI_ERR_ALIGNMENT, "pointer %p is not 16-byte aligned", p);
  for (int i = 0; i < 4; ++i) {
    const void* o = outp[i];
    if (!o) continue;
    if ((uintptr_t)o & 15u) return fail(GEMM_EPI_ERR_ALIGNMENT, "pointer %p is not 16-byte aligned", o);
    for (const void* p : in)
      if (p == o && !(i == 0 && (p == dD || p == Z)) && !(i == 2 && p == dB_in))
        return fail(GEMM_EPI_ERR_INVALID_ARG, "a gradient may not be an input (dZ may be dD or Z, dB may be dB_in)");
    for (int j = 0; j < i; ++j)
      if (outp[j] == o) return fail(GEMM_EPI_ERR_INVALID_ARG, "two gradients share a pointer");
  }
  int rc = check_workspace(workspace, workspace_bytes, h->ws_bytes);
  if (!rc) rc = check_device(h->device);
  if (rc) return rc;

  hipStream_t s = (hipStream_t)stream;
  float* partial = dbias ? (float*)workspace : nullptr;
  void* products = (char*)workspace + h->partial_bytes;
  (void)hipGetLastError();  // clear a stale error so the checks below are ours
  if (act || partial) {
    launch_linear_dact(d.ab_dtype, d.act, dD, Z, dZ, partial, d.M, d.N, h->chunk, s);
    rc = launched();
    if (!rc && partial) {
      launch_colsum(partial, (d.M + h->chunk - 1) / h->chunk, d.N, dbias, d.dbias_dtype, s);
      rc = launched();
    }
  }
  const void* g = act ? dZ : dD;
  if (!rc && dA) rc = run_with_workspace(h->da, g, B, nullptr, dA, 0.0f, products, stream);
  if (!rc && dB) rc = run_with_workspace(h->db, g, A, dB_in, dB, dB_in ? 1.0f : 0.0f, products, stream);
  return rc;
}

extern "C" int gemm_epi_linear_grad_destroy(gemm_epi_linear_grad_handle* h) {
  if (h) {
    gemm_epi_destroy(h->da);
    gemm_epi_destroy(h->db);
  }
  delete h;
  return GEMM_EPI_OK;
}

extern "C" int64_t gemm_epi_linear_grad_workspace(const gemm_epi_linear_grad_handle* h) {
  return h ? h->ws_bytes : -1;
}
