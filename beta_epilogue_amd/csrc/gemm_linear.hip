// gemm_linear.hip -- C ABI of the linear layer and its backward (see
// include/gemm_epi_linear.h): validation, kernel choice, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <new>

#include "gemm_epi_host.hpp"
#include "gemm_epi_linear.h"
#include "gemm_linear.hpp"

using namespace gemm_epi;

namespace {

struct LinearVariant {
  const char* name;
  int part, ab, bm, bn, bk, lds, occ;
};
#define X(PART, AB, BM, BN, S, OCC, BL, NAME) \
  {NAME, PART, AB, BM, BN, LinearCfg<AB, BM, BN, S, OCC, BL>::BK, LinearCfg<AB, BM, BN, S, OCC, BL>::LDS_BYTES, OCC},
const LinearVariant kLinear[] = {
#include "gemm_linear_variants.inc"
};
#undef X
constexpr int kTiles = (int)(sizeof kLinear / sizeof kLinear[0]);
constexpr int kRowsVariant = kTiles;  // the few-row kernels, one entry
constexpr int kThreads = 256;
// A launch has less than 2^32 threads: 16 columns for a workgroup of up to 512 ...
constexpr int64_t kRowsMaxN = int64_t(1) << 26;
// ... and 32 for one of 1024 in the column sums; 256 threads for an item.
constexpr int64_t kGradMaxN = int64_t(1) << 26, kGradMaxBlocks = int64_t(1) << 24;

// The plan's cost model (us), fitted per type to 1054 forced plans (24 shapes, M
// 90 to 8192, N 704 to 8192, K 512 to 8192; every tile, 1 to 6 slices), weighted
// towards each shape's best ones: 3 to 6 % rms from the measured times there, and
// the plans that it chooses of them take under 1 % longer on the mean, 17 % at worst,
// than the best measured ones.  An item (a tile or a K slice of one) takes its
// K tiles times tk plus an epilogue of e0 + e1 * area (in 256x256 tiles); rounds
// of items fill the compute units.  Smaller tiles of which two or three share a
// compute unit take pair or three together.  Slices add a second launch, `join`
// us and their partial sums at bw TB/s.
struct LinearCost {
  double start, join, bw, e0, e1;
  double tk256, tk192, tk128x256, tk128, tk64, pair128, pair64, three64;
};
constexpr LinearCost kCost16 = {0.98, 3.65, 21.9, 3.11, 10.4, 1.296, 1.032, 0.0, 0.592, 0.231, 0.821, 0.344, 0.0};
constexpr LinearCost kCostE4m3 = {1.89, 4.93, 32.2, 2.6, 11.4, 1.373, 1.007, 0.685, 0.407, 0.218, 0.0, 0.329, 0.0};
constexpr LinearCost kCostI8 = {1.1, 4.2, 21.8, 3.36, 10.8, 1.287, 1.027, 0.0, 0.61, 0.259, 0.856, 0.361, 0.509};
constexpr LinearCost kCostWide = {2.41, 3.49, 14.5, 2.14, 14.3, 0.0, 0.0, 0.0, 0.796, 0.349, 1.43, 0.53, 0.0};

// Tiles of variant v: the first whole, the last `tail` in K slices of `kslice`.
struct LinearCut {
  int64_t tiles_m, tiles_n, tiles, tail, kslice;
  int splits;
  int64_t items() const { return tiles - tail + tail * splits; }
};

// all: every tile in slices; else those that whole rounds leave over.
LinearCut cut_linear(const LinearVariant& v, const gemm_epi_linear_desc& d, int64_t splits, bool all, int64_t cus) {
  LinearCut c;
  const int64_t ktiles = (d.K + v.bk - 1) / v.bk;
  c.tiles_m = (d.M + v.bm - 1) / v.bm;
  c.tiles_n = (d.N + v.bn - 1) / v.bn;
  c.tiles = c.tiles_m * c.tiles_n;
  splits = std::max<int64_t>(1, std::min(splits, ktiles));
  c.kslice = (ktiles + splits - 1) / splits * v.bk;
  c.splits = (int)((d.K + c.kslice - 1) / c.kslice);
  c.tail = c.splits == 1 ? 0 : all ? c.tiles : c.tiles % (cus * v.occ);
  if (c.tail == 0) c.splits = 1, c.kslice = d.K;
  return c;
}

// The few-row kernel's time (us): its waves stream runs of 256 bytes of K, and a
// run costs its latency (first figure) or, with all compute units at work, its
// share of the bandwidth and of the products (second); fitted at N and K of 512
// to 8192, 16 and 8 bits, within 15 %.
double rows_time(const gemm_epi_linear_desc& d, int64_t cus) {
  const int64_t runs = (d.K * elem_bytes(d.ab_dtype) + 8 * 256 - 1) / (8 * 256), blocks = (d.N + 15) / 16;
  const double per_cu = blocks < cus ? (double)blocks / (double)cus : (double)((blocks + cus - 1) / cus);
  const double latency = d.M <= 32 ? 1.2 : 1.9, busy = d.M <= 32 ? 1.9 : d.M <= 48 ? 2.3 : 2.55;
  return std::max(4.5 + (double)runs * latency, 3.0 + (double)runs * per_cu * busy);
}

double linear_time(const LinearVariant& v, const LinearCut& c, const gemm_epi_linear_desc& d, int64_t cus) {
  const LinearCost& w = v.ab == T_E4M3 ? kCostE4m3 : v.ab == T_I8 ? kCostI8 : v.ab == T_E4M3_WIDE ? kCostWide : kCost16;
  const double area = (double)v.bm * v.bn / 65536.0, epi = w.e0 + w.e1 * area;
  auto rounds = [&](int64_t items, int64_t k) {
    if (items == 0) return 0.0;
    double tk = v.bm == 256 ? w.tk256 : v.bm == 192 ? w.tk192 : v.bn == 256 ? w.tk128x256 : v.bm == 128 ? w.tk128 : w.tk64;
    int64_t slots = cus;
    if (v.occ >= 2 && items > cus) tk = v.bm == 128 ? w.pair128 : w.pair64, slots = 2 * cus;
    if (v.occ >= 3 && items > 2 * cus) tk = w.three64, slots = 3 * cus;
    return (double)((items + slots - 1) / slots) * (tk * (double)((k + v.bk - 1) / v.bk) + epi);
  };
  const double products = rounds(c.tiles - c.tail, d.K) + rounds(c.tail * c.splits, std::min(c.kslice, d.K));
  // A and B once from memory, at the 4.5 TB/s that tiles of few rows reach (24
  // bf16 rows, N = K = 8192: 39 us, 20 by the items alone)
  const double stream = (double)(d.M + d.N) * (double)(d.K * elem_bytes(d.ab_dtype)) / 4.5e6 + epi;
  double t = w.start + std::max(products, stream);
  if (c.tail) t += w.join + (double)c.tail * v.bm * v.bn * 4.0 * (2 * c.splits + 1) / (w.bw * 1e6);
  return t;
}

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
  int nw;                  // few rows: waves per workgroup
  int64_t tiles_m, tiles_n, tiles, tail, kslice, items;
  int splits, group_m;
  int64_t ws_bytes;
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
  const int es = elem_bytes(d->ab_dtype), ds = elem_bytes(d->d_dtype);
  int rc = check_stride("a", &d->lda, d->K, es, true);
  if (!rc) rc = check_stride("b", &d->ldb, d->K, es, true);
  if (!rc) rc = check_stride("d", &d->ldd, d->N, ds, true);
  if (!rc) rc = check_stride("r", &d->ldr, d->N, ds, d->residual);
  if (!rc) rc = check_stride("z", &d->ldz, d->N, ds, d->z);
  if (rc) return rc;
  // partial sums are fp32 rows of a tile; row and column numbers are 32-bit
  if (d->M >= (int64_t(1) << 31) - 512 || d->N >= (int64_t(1) << 31) - 512)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "M and N must be below 2^31 - 512");
  // 2^17 products of -128 by -128 reach 2^31
  if (d->ab_dtype == GEMM_EPI_I8 && d->K >= int64_t(1) << 17)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "int8 with K of 2^17 or more: the int32 sums could overflow");
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
  // (the fp8 MFMA sums a group of products with fewer bits than fp32 keeps)
  const bool widened = d.ab_dtype == GEMM_EPI_E4M3 && d.d_dtype == GEMM_EPI_F32;
  const int kernel_ab = widened ? (int)T_E4M3_WIDE : d.ab_dtype;
  const bool rows_fit = d.M <= kRowsMax && d.N <= kRowsMaxN;
  if (variant == kRowsVariant ? !rows_fit : variant >= 0 && kLinear[variant].ab != kernel_ab)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "variant %s cannot run this problem", gemm_epi_linear_variant_name(variant));
  int device = 0, cus = 0;
  rc = device_query(&device, &cus);
  if (rc) return rc;

  LinearCut best = {};
  if (variant != kRowsVariant) {
    // the tile shape and K split of the lowest modelled time
    const int forced = variant;
    double best_us = 0.0;
    for (int i = 0; i < kTiles; ++i) {
      if (kLinear[i].ab != kernel_ab || (forced != -1 && i != forced)) continue;
      for (int64_t s = d.splits ? d.splits : 1; s <= (d.splits ? d.splits : 16); ++s) {
        const LinearCut c = cut_linear(kLinear[i], d, s, d.splits != 0, cus);
        const double us = linear_time(kLinear[i], c, d, cus);
        if (best.tiles == 0 || us < best_us) best_us = us, best = c, variant = i;
      }
    }
    // few rows: up to 16 always (the tiles would be mostly empty), up to 64
    // where the model says so (32 bf16 rows: N = K = 4096 10.8 us against
    // 12.7 as tiles, N = 512 and K = 8192 14.2 against 11.6)
    if (forced == -1 && d.splits == 0 && rows_fit && (d.M <= 16 || rows_time(d, cus) < best_us))
      variant = kRowsVariant;
  }

  gemm_epi_linear_handle* h = new (std::nothrow) gemm_epi_linear_handle();
  if (!h) return fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
  h->d = d;
  h->variant = variant;
  h->device = device;
  h->cus = cus;
  h->splits = 1;
  if (variant == kRowsVariant) {
    // with more than 8 rows a workgroup of 8 waves takes a compute unit's LDS:
    // 4 waves once there is more than one workgroup for each (16 e4m3 rows,
    // K = N: 4096 7.7 us with 4 waves, 7.0 with 8; 8192 15.5 and 16.3)
    h->nw = d.M <= 8 || (d.N + 15) / 16 <= cus ? 8 : 4;
    h->tiles_m = 1;
    h->tiles_n = (d.N + 15) / 16;
    h->tiles = h->items = h->tiles_n;
    h->grid = (int)h->tiles_n;
    *out = h;
    return GEMM_EPI_OK;
  }
  const LinearVariant& v = kLinear[variant];
  h->tiles_m = best.tiles_m;
  h->tiles_n = best.tiles_n;
  h->tiles = best.tiles;
  h->group_m = h->tiles_n > 32 ? 8 : 4;
  h->splits = best.splits;
  h->kslice = best.kslice;
  h->tail = best.tail;
  h->items = best.items();
  if (h->tiles >= (int64_t(1) << 31) || h->items >= (int64_t(1) << 31)) {
    delete h;
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "2^31 or more work items (tiles and K slices)");
  }
  h->grid = (int)std::min<int64_t>(h->items, (int64_t)cus * v.occ);
  h->ws_bytes = h->splits > 1 ? h->splits * h->tail * v.bm * v.bn * 4 : 0;
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
    launch_linear_rows(d.ab_dtype, h->nw, p, s);
    return launched();
  }
  const LinearVariant& v = kLinear[h->variant];
  p.tiles_total = (int32_t)h->items;
  p.L = 1;
  p.tiles_m = (int32_t)h->tiles_m;
  p.tiles_n = (int32_t)h->tiles_n;
  p.group_m = h->group_m;
  p.xcd_remap = 1;
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
    out->tile_m = kRowsMax;
    out->tile_n = 16;
    out->threads = h->nw * 64;
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
namespace {

// One product of the backward: M x N over K in tile x tile tiles.
struct GradProduct {
  bool on = false;
  int64_t M = 0, N = 0, K = 0;
  int64_t tiles_m = 0, tiles_n = 0, tiles = 0, kslice = 0;
  int splits = 1;
  int64_t items() const { return on ? tiles * splits : 0; }
  int64_t slots(int tile) const { return on && splits > 1 ? tiles * splits * tile * tile * 4 : 0; }
};

constexpr int kGradKTile = 64;

void cut(GradProduct* p, int tile, int64_t splits) {
  if (!p->on) return;
  const int64_t ktiles = (p->K + kGradKTile - 1) / kGradKTile;
  p->tiles_m = (p->M + tile - 1) / tile;
  p->tiles_n = (p->N + tile - 1) / tile;
  p->tiles = p->tiles_m * p->tiles_n;
  splits = std::max<int64_t>(1, std::min(splits, ktiles));
  p->kslice = (ktiles + splits - 1) / splits * kGradKTile;
  p->splits = (int)((p->K + p->kslice - 1) / p->kslice);
}

// Modelled time (us) of the launch and the join, from forced runs of 40 shapes
// (M 1 to 6385, N and K 256 to 4096): an item takes 1.1 us per K tile with 256x256
// tiles, 0.45 with 128x128 and 0.16 with 64x64 ones, or 0.85 and 0.38 for two
// that share a compute unit, and 8, 4 or 2.2 us besides.  A grid of several
// rounds ends unevenly by half an item: with few large tiles one of the shorter
// product, which starts last (7157 x 2152 x 1576: 137 us without the K slices
// that half a long item made it choose, 158 with them).  The plans that it
// chooses take up to 8 % longer than the best forced ones, 12 % at worst.
double grad_time(const GradProduct& a, const GradProduct& b, int tile, int cus) {
  const double items = (double)(a.items() + b.items());
  const bool pairs = tile != 256 && items > cus;
  const double slots = pairs ? 2.0 * cus : cus;
  const double tk = tile == 256 ? 1.1 : tile == 128 ? (pairs ? 0.85 : 0.45) : (pairs ? 0.38 : 0.16);
  const double fixed = tile == 256 ? 8.0 : tile == 128 ? 4.0 : 2.2;
  double longest = 0.0, last = 0.0, total = 0.0, join = 0.0;
  for (const GradProduct* p : {&a, &b}) {
    if (!p->on) continue;
    const double item = fixed + tk * (double)((std::min(p->kslice, p->K) + kGradKTile - 1) / kGradKTile);
    last = last == 0.0 ? item : std::min(last, item);  // the longer items go first
    longest = std::max(longest, item);
    total += item * (double)p->items();
    if (p->splits > 1) join = std::max(join, 5.0) + 2.0 * (double)p->slots(tile) / 5.0e6;
  }
  const double tail = 0.5 * (tile == 64 ? longest : last);
  return (items <= slots ? longest : std::max(longest, total / slots + tail)) + join;
}

}  // namespace

struct gemm_epi_linear_grad_handle {
  gemm_epi_linear_grad_desc d;
  int device, cus;
  int chunk;       // rows per partial column sum
  int tile;
  GradProduct a, b;  // dA, dB
  int64_t ws_a, ws_b, ws_bytes;  // workspace: partial sums, then a's and b's slices
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
  if (d.tile != 0 && d.tile != 64 && d.tile != 128 && d.tile != 256)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "tile must be 0, 64, 128 or 256 (got %d)", d.tile);
  if (d.splits < 0) return fail(GEMM_EPI_ERR_INVALID_ARG, "splits must be >= 0 (got %d)", d.splits);
  const bool da = d.da_dtype != GEMM_EPI_NONE, db = d.db_dtype != GEMM_EPI_NONE;
  // every extent below 2^31 - 512 first, so that no product below overflows
  const int64_t most = (int64_t(1) << 31) - 512;
  if (d.M >= most || d.N >= most || d.K >= most)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "M, N and K must be below 2^31 - 512");
  if (d.N > kGradMaxN) return fail(GEMM_EPI_ERR_UNSUPPORTED, "more than 2^26 columns");
  if (d.N % 8 || ((da || db) && d.K % 8))
    return fail(GEMM_EPI_ERR_ALIGNMENT, "rows of dD (%lld elements) and of A and B (%lld) must be multiples of 16 bytes",
                (long long)d.N, (long long)d.K);
  // 256 rows of an output or a K-major operand, and a whole operand that is
  // read across its rows, are addressed with 31-bit byte offsets
  if ((da || db) && (d.K * 4 * 256 > INT32_MAX || d.N * 4 * 256 > INT32_MAX))
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "rows too long for 31-bit tile offsets");
  const int64_t pad = 2 * kGradKTile;
  if ((da && (d.N + pad) * d.K * 2 > INT32_MAX) ||
      (db && ((d.M + pad) * d.N * 2 > INT32_MAX || (d.M + pad) * d.K * 2 > INT32_MAX)))
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "an operand read across its rows is 2 GiB or larger");
  int device = 0, cus = 0;
  const int rc = device_query(&device, &cus);
  if (rc) return rc;

  gemm_epi_linear_grad_handle* h = new (std::nothrow) gemm_epi_linear_grad_handle();
  if (!h) return fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
  h->d = d;
  h->device = device;
  h->cus = cus;
  // rows per workgroup of the elementwise pass (and per partial sum): 64, fewer
  // as long as there are under four workgroups for a compute unit (596 x 2592:
  // 14.5 us with 64 rows), more where 2^16 chunks would not do (the grid's
  // second dimension)
  int64_t chunk = 64;
  while (chunk > 8 && (d.N + 255) / 256 * ((d.M + chunk - 1) / chunk) < 4 * cus) chunk /= 2;
  h->chunk = (int)std::max<int64_t>(chunk, (d.M + 65534) / 65535);
  h->a.on = da;
  h->a.M = d.M, h->a.N = d.K, h->a.K = d.N;
  h->b.on = db;
  h->b.M = d.N, h->b.N = d.K, h->b.K = d.M;
  double best = 0.0;
  for (const int tile : {256, 128, 64}) {
    if (d.tile != 0 && d.tile != tile) continue;
    for (int64_t sa = 1; sa <= (da && !d.splits ? 16 : 1); ++sa)
      for (int64_t sb = 1; sb <= (db && !d.splits ? 16 : 1); ++sb) {
        GradProduct a = h->a, b = h->b;
        cut(&a, tile, d.splits ? d.splits : sa);
        cut(&b, tile, d.splits ? d.splits : sb);
        const double t = grad_time(a, b, tile, cus);
        if (h->tile == 0 || t < best) best = t, h->tile = tile, h->a = a, h->b = b;
      }
  }
  if (h->a.items() + h->b.items() + (d.N + 31) / 32 >= kGradMaxBlocks) {
    delete h;
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "2^24 or more work items (tiles and K slices)");
  }
  const int64_t chunks = (d.M + h->chunk - 1) / h->chunk;
  const bool sum_rows = d.act == GEMM_EPI_ACT_NONE && (da || db);
  h->ws_a = d.dbias_dtype != GEMM_EPI_NONE && !sum_rows && chunks > 1 ? up256(chunks * d.N * 4) : 0;
  h->ws_b = h->ws_a + h->a.slots(h->tile);
  h->ws_bytes = h->ws_b + h->b.slots(h->tile);
  *out = h;
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_linear_grad_run(const gemm_epi_linear_grad_handle* h, const void* dD, const void* A,
                                        const void* B, const void* Z, const void* dB_in, void* dZ, void* dA, void* dB,
                                        void* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
  return gemm_epi_linear_grad_run_alpha(h, dD, A, B, Z, dB_in, dZ, dA, dB, dbias, 1.0f, workspace, workspace_bytes,
                                        stream);
}

extern "C" int gemm_epi_linear_grad_run_alpha(const gemm_epi_linear_grad_handle* h, const void* dD, const void* A,
                                              const void* B, const void* Z, const void* dB_in, void* dZ, void* dA,
                                              void* dB, void* dbias, float alpha, void* workspace,
                                              int64_t workspace_bytes, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_linear_grad_desc& d = h->d;
  const bool act = d.act != GEMM_EPI_ACT_NONE;
  if (!dD) return fail(GEMM_EPI_ERR_INVALID_ARG, "dD is required");
  if ((Z != nullptr) != act || (dZ != nullptr) != act)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "Z and dZ must be given exactly with an activation");
  if ((dA != nullptr) != h->a.on || (B != nullptr) != h->a.on)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dA and B must be given exactly when da_dtype is set");
  if ((dB != nullptr) != h->b.on || (A != nullptr) != h->b.on || (dB_in && !dB))
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
  const int64_t chunks = (d.M + h->chunk - 1) / h->chunk;
  const bool products = dA || dB;
  const bool sum_rows = dbias && !act && products;  // the products' launch sums dD itself
  float* partial = dbias && !sum_rows && chunks > 1 ? (float*)workspace : nullptr;
  (void)hipGetLastError();  // clear a stale error so the checks below are ours
  if (act || (dbias && !sum_rows)) {
    launch_linear_dact(d.ab_dtype, d.act, dD, Z, dZ, partial, dbias, d.dbias_dtype, d.M, d.N, h->chunk, s);
    rc = launched();
    if (rc) return rc;
  }
  if (!products) {
    if (partial) launch_colsum(partial, chunks, d.N, dbias, d.dbias_dtype, s);
    return launched();
  }
  const void* g = act ? dZ : dD;
  GradParams p = {};
  auto product = [&](LinParams* q, const GradProduct& w, const void* qa, const void* qb, const void* add, void* qd,
                     int type, int64_t ws) {
    q->A = qa;
    q->B = qb;
    q->D = qd;
    q->R = add;
    q->M = w.M;
    q->N = w.N;
    q->K = w.K;
    q->lda = w.K;  // (of a K-major A; the other operands are packed)
    q->ldd = q->ldr = q->ldz = w.N;
    q->alpha = alpha;
    q->d_dtype = type;
    q->tiles_total = (int32_t)w.items();
    q->L = 1;
    q->tiles_m = (int32_t)w.tiles_m;
    q->tiles_n = (int32_t)w.tiles_n;
    q->group_m = w.tiles_n > 32 ? 8 : 4;
    q->xcd_remap = 1;
    q->splits = w.splits;
    q->kslice = w.kslice;
    q->tail_tiles = w.splits > 1 ? (int32_t)w.tiles : 0;
    q->dp_tiles = (int32_t)w.tiles - q->tail_tiles;
    q->ws = (char*)workspace + ws;
  };
  if (dA) product(&p.a, h->a, g, B, nullptr, dA, d.da_dtype, h->ws_a);
  if (dB) product(&p.b, h->b, g, A, dB_in, dB, d.db_dtype, h->ws_b);
  p.ga = p.a.tiles_total;
  p.gb = p.b.tiles_total;
  p.b_first = dB && (!dA || std::min(h->b.kslice, h->b.K) > std::min(h->a.kslice, h->a.K)) ? 1 : 0;
  p.partial = partial;
  p.rows = sum_rows ? dD : nullptr;
  p.P = sum_rows ? d.M : chunks;
  p.C = d.N;
  p.dbias = dbias;
  p.dbias_dtype = d.dbias_dtype;
  const int kind = h->tile == 256 ? GRAD_256 : h->tile == 64 ? GRAD_64 : p.ga + p.gb > h->cus ? GRAD_128 : GRAD_128_DEEP;
  static void (*const kLaunch[2][kGradKinds])(const GradParams&, hipStream_t) = {
      {launch_linear_grad_mm<T_F16, 0>, launch_linear_grad_mm<T_F16, 1>, launch_linear_grad_mm<T_F16, 2>,
       launch_linear_grad_mm<T_F16, 3>},
      {launch_linear_grad_mm<T_BF16, 0>, launch_linear_grad_mm<T_BF16, 1>, launch_linear_grad_mm<T_BF16, 2>,
       launch_linear_grad_mm<T_BF16, 3>}};
  kLaunch[d.ab_dtype == GEMM_EPI_BF16][kind](p, s);
  rc = launched();
  if (rc || (p.a.tail_tiles == 0 && p.b.tail_tiles == 0)) return rc;
  launch_linear_grad_join(p.a, p.b, h->tile, (int64_t)h->cus * 8, s);
  return launched();
}

extern "C" int gemm_epi_linear_grad_destroy(gemm_epi_linear_grad_handle* h) {
  delete h;
  return GEMM_EPI_OK;
}

extern "C" int64_t gemm_epi_linear_grad_workspace(const gemm_epi_linear_grad_handle* h) {
  return h ? h->ws_bytes : -1;
}
