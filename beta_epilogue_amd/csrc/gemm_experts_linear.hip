// gemm_experts_linear.hip -- C ABI of the experts' linear layer and its
// backward (see include/gemm_epi_experts.h): validation, kernel choice, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <new>

#include "gemm_epi_experts.h"
#include "gemm_epi_host.hpp"
#include "gemm_grouped.hpp"
#include "gemm_linear_cost.hpp"

using namespace gemm_epi;

namespace {

struct GroupedVariant {
  const char* name;
  int part, ab, bm, bn, bk, lds, occ;
};
#define X(PART, AB, BM, BN, S, OCC, BL, NAME)                        \
  {NAME, PART, AB, BM, BN, GroupedCfg<AB, BM, BN, S, OCC, BL>::BK,   \
   GroupedCfg<AB, BM, BN, S, OCC, BL>::LDS_BYTES + kGroupTableBytes, OCC},
const GroupedVariant kGrouped[] = {
#include "gemm_grouped_variants.inc"
};
#undef X
constexpr int kTiles = (int)(sizeof kGrouped / sizeof kGrouped[0]);
// The few-row kernels: chunks of 4 and 16 rows.  (8 and 32 were never ahead of
// both and the 64x64 tiles by more than 3 %.)
constexpr int kRowsBlocks[] = {1, 4};
const char* const kRowsNames[] = {"experts_rows4", "experts_rows16"};
constexpr int kVariants = kTiles + 2;

typedef void (*part_fn)(int, const GroupParams&, int, hipStream_t);
const part_fn kParts[kGroupedParts] = {launch_grouped_part<0>, launch_grouped_part<1>, launch_grouped_part<2>,
                                       launch_grouped_part<3>, launch_grouped_part<4>, launch_grouped_part<5>,
                                       launch_grouped_part<6>};

// Chunks of `chunk` rows (or tiles of as many) that the worst distribution of
// `rows` rows over the experts has.
int64_t worst_chunks(int64_t rows, int64_t experts, int64_t chunk) {
  const int64_t n = std::min(rows, experts);
  return n + (rows - n) / chunk;
}

// ... and that are to be expected of a router: an expert's last chunk is half full
// on the mean, and there is one at least.
double likely_chunks(int64_t rows, int64_t experts, int64_t chunk) {
  const double n = (double)std::min(rows, experts), per = (double)rows / n;
  return n * std::max(1.0, per / (double)chunk + (per > 1.0 ? 0.5 : 0.0));
}

// Modelled time (us) of a tile kernel: the linear layer's model over the tiles
// that are to be expected (half a round on the mean for the last one; 256x256 tiles
// may finish it as quarters), and the weights of the experts that have rows once
// from memory, at the 5.2 TB/s that the 64x64 tiles reach and the larger ones do not
// (512 rows, 64 experts, bf16 1536 x 2048: 78, 102 and 141 us).
double tiles_time(const GroupedVariant& v, const gemm_epi_expert_linear_desc& d, int64_t cus) {
  const LinearCost& w = linear_cost(v.ab);
  const double items = likely_chunks(d.rows, d.experts, v.bm) * (double)((d.N + v.bn - 1) / v.bn);
  const double epi = linear_epilogue_time(w, v.bm, v.bn);
  double tk = v.bm == 256 ? w.tk256 : v.bm == 128 ? w.tk128 : w.tk64, slots = (double)cus;
  if (v.occ >= 2 && items > (double)cus) tk = v.bm == 128 ? w.pair128 : w.pair64, slots *= 2;
  if (v.occ >= 3 && items > 2.0 * (double)cus) tk = w.three64, slots *= 1.5;
  const double item = tk * (double)((d.K + v.bk - 1) / v.bk) + epi;
  const double full = items / slots, last = full <= 0.8 ? 0.2 : v.bm == 256 ? 0.35 : 0.5;
  const double rounds = std::max(1.0, full + last);
  const double es = elem_bytes(d.ab_dtype), n = (double)std::min<int64_t>(d.rows, d.experts);
  const double stream = (n * (double)d.N + (double)d.rows) * (double)d.K * es / 5.2e6;
  return w.start + std::max(rounds * item, stream * (v.bm == 64 ? 1.0 : v.bm == 128 ? 1.15 : 1.5));
}

// The few-row kernels: a workgroup's waves stream runs of 256 bytes of K each; a
// run costs its latency or, with every compute unit at work, its share of the
// bandwidth.  Within a fifth of 14 shapes of 1 to 128 rows, N 256 to 4096, K 768 to
// 8192, bf16 and e4m3.
double rows_time(int mb, const gemm_epi_expert_linear_desc& d, int64_t cus) {
  const int bytes = mb == 1 ? 8 * 256 : 4 * 256;  // of K, all waves' runs
  const double runs = (double)((d.K * elem_bytes(d.ab_dtype) + bytes - 1) / bytes);
  const double blocks = likely_chunks(d.rows, d.experts, 4 * mb) * (double)((d.N + 15) / 16) / (double)cus;
  const double latency = mb == 1 ? 0.55 : 0.37;
  return std::max(4.2 + runs * latency, 3.0 + blocks * (mb == 1 ? runs * 1.3 + 1.0 : runs * 0.67 + 1.3));
}

// As the linear layer's: row stride `ld` (0: packed) of a tensor with `cols`
// elements of `es` bytes per row.
int check_stride(const char* name, int64_t* ld, int64_t cols, int es, bool used) {
  if (!used) {
    if (*ld != 0) return fail(GEMM_EPI_ERR_INVALID_ARG, "ld%s is given but the tensor is not used", name);
    return GEMM_EPI_OK;
  }
  if (*ld == 0) *ld = cols;
  if (*ld < cols)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "ld%s %lld is below the row's %lld elements", name, (long long)*ld,
                (long long)cols);
  if (*ld >= (int64_t(1) << 31) / 256 / es)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "rows of %lld elements are too long for 31-bit tile offsets",
                (long long)*ld);
  if (cols * es % 16 || *ld * es % 16)
    return fail(GEMM_EPI_ERR_ALIGNMENT, "rows (%lld elements) and row strides (%lld) must be multiples of 16 bytes",
                (long long)cols, (long long)*ld);
  return GEMM_EPI_OK;
}

int check_sizes(int64_t rows, int64_t N, int64_t K, int experts) {
  if (rows < 1 || N < 1 || K < 1)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "rows, N, K must be >= 1 (got %lld %lld %lld)", (long long)rows,
                (long long)N, (long long)K);
  if (experts < 1 || experts > kMaxExperts)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "experts must be 1 .. %d (got %d)", kMaxExperts, experts);
  const int64_t most = (int64_t(1) << 31) - 512;
  if (rows >= most || N >= most || K >= most)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "rows, N and K must be below 2^31 - 512");
  return GEMM_EPI_OK;
}

bool flag_ok(int f) { return f == 0 || f == 1; }

int aligned16(const void* p) {
  if ((uintptr_t)p & 15u) return fail(GEMM_EPI_ERR_ALIGNMENT, "pointer %p is not 16-byte aligned", p);
  return GEMM_EPI_OK;
}

int aligned4(const void* p) {
  if ((uintptr_t)p & 3u) return fail(GEMM_EPI_ERR_ALIGNMENT, "pointer %p is not 4-byte aligned", p);
  return GEMM_EPI_OK;
}

}  // namespace

struct gemm_epi_expert_linear_handle {
  gemm_epi_expert_linear_desc d;  // strides filled in
  int variant, device, cus;
  int64_t tiles_n, grid;          // few rows: grid is the number of chunks
};

extern "C" int gemm_epi_expert_linear_create_variant(const gemm_epi_expert_linear_desc* desc, int variant,
                                                     gemm_epi_expert_linear_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  gemm_epi_expert_linear_desc d = *desc;
  int rc = check_sizes(d.rows, d.N, d.K, d.experts);
  if (rc) return rc;
  if (!is_type(d.ab_dtype) || d.ab_dtype == GEMM_EPI_F32 || d.ab_dtype == GEMM_EPI_I32)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "ab_dtype must be F16, BF16, E4M3 or I8");
  if (d.ab_dtype == GEMM_EPI_E5M2 || d.ab_dtype == GEMM_EPI_U8)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "the experts' linear layer has no e5m2 or uint8 form");
  if (!is_float_out(d.d_dtype)) return fail(GEMM_EPI_ERR_INVALID_ARG, "d_dtype must be F16, BF16 or F32");
  if (d.bias_dtype != GEMM_EPI_NONE && !is_float_out(d.bias_dtype))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "bias_dtype must be NONE, F16, BF16 or F32");
  if (d.act < GEMM_EPI_ACT_NONE || d.act > GEMM_EPI_ACT_SILU)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown activation %d", d.act);
  if (!flag_ok(d.mul) || !flag_ok(d.z) || !flag_ok(d.scale_a) || !flag_ok(d.scale_b))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "mul, z, scale_a and scale_b must be 0 or 1");
  const int es = elem_bytes(d.ab_dtype), ds = elem_bytes(d.d_dtype);
  int64_t ldb = 0;
  rc = check_stride("a", &d.lda, d.K, es, true);
  if (!rc) rc = check_stride("b", &ldb, d.K, es, true);
  if (!rc) rc = check_stride("d", &d.ldd, d.N, ds, true);
  if (!rc) rc = check_stride("u", &d.ldu, d.N, ds, d.mul);
  if (!rc) rc = check_stride("z", &d.ldz, d.N, ds, d.z);
  if (rc) return rc;
  if (d.bias_dtype != GEMM_EPI_NONE && d.N * elem_bytes(d.bias_dtype) % 16)
    return fail(GEMM_EPI_ERR_ALIGNMENT, "an expert's bias (%lld elements) must be a multiple of 16 bytes", (long long)d.N);
  if (d.scale_b && d.N % 4)
    return fail(GEMM_EPI_ERR_ALIGNMENT, "an expert's scale_b (%lld elements) must be a multiple of 16 bytes", (long long)d.N);
  // 2^17 products of -128 by -128 reach 2^31
  if (d.ab_dtype == GEMM_EPI_I8 && d.K >= int64_t(1) << 17)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "int8 with K of 2^17 or more: the int32 sums could overflow");
  if (variant < -1 || variant >= kVariants) return fail(GEMM_EPI_ERR_INVALID_ARG, "variant %d out of range", variant);
  // The fp8 MFMA sums a group of products with fewer bits than fp32 keeps (+-8192 among
  // products near 1: 5.6e-4 of sum |a||b|), which 16-bit outputs allow for the sake
  // of its rate: 98760 rows of 128 experts, 1536 x 4096, 637 us, widened to fp16 1105.
  const int kernel_ab = d.ab_dtype == GEMM_EPI_E4M3 && d.d_dtype == GEMM_EPI_F32 ? (int)T_E4M3_WIDE : d.ab_dtype;
  auto rows_fit = [&](int v) {  // a launch's second dimension, and less than 2^32 threads
    const int64_t chunks = worst_chunks(d.rows, d.experts, 4 * kRowsBlocks[v - kTiles]);
    return chunks <= 65535 && (d.N + 15) / 16 < (int64_t(1) << 32) / 512 / chunks;
  };
  if (variant >= 0 && (variant < kTiles ? kGrouped[variant].ab != kernel_ab : !rows_fit(variant)))
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "variant %s cannot run this problem",
                gemm_epi_expert_linear_variant_name(variant));
  int device = 0, cus = 0;
  rc = device_query(&device, &cus);
  if (rc) return rc;
  if (variant == -1) {
    double best = 0.0;
    for (int i = 0; i < kVariants; ++i) {
      if (i < kTiles ? kGrouped[i].ab != kernel_ab : !rows_fit(i)) continue;
      const double us = i < kTiles ? tiles_time(kGrouped[i], d, cus) : rows_time(kRowsBlocks[i - kTiles], d, cus);
      if (variant == -1 || us < best) best = us, variant = i;
    }
  }
  gemm_epi_expert_linear_handle h = {d, variant, device, cus, 0, 0};
  if (variant < kTiles) {
    const GroupedVariant& v = kGrouped[variant];
    h.tiles_n = (d.N + v.bn - 1) / v.bn;
    const int64_t tiles_m = worst_chunks(d.rows, d.experts, v.bm);
    if (tiles_m >= (int64_t(1) << 29) / h.tiles_n)  // their quarters are counted in 32 bits
      return fail(GEMM_EPI_ERR_UNSUPPORTED, "2^29 or more tiles");
    h.grid = std::min<int64_t>(tiles_m * h.tiles_n, (int64_t)cus * v.occ);
  } else {
    h.tiles_n = (d.N + 15) / 16;
    h.grid = worst_chunks(d.rows, d.experts, 4 * kRowsBlocks[variant - kTiles]);
  }
  *out = new (std::nothrow) gemm_epi_expert_linear_handle(h);
  return *out ? GEMM_EPI_OK : fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
}

extern "C" int gemm_epi_expert_linear_create(const gemm_epi_expert_linear_desc* desc,
                                             gemm_epi_expert_linear_handle** out) {
  return gemm_epi_expert_linear_create_variant(desc, -1, out);
}

extern "C" int gemm_epi_expert_linear_run(const gemm_epi_expert_linear_handle* h, const void* A, const void* B,
                                          const int32_t* offsets, const void* bias, const float* scale_a,
                                          const float* scale_b, const void* U, void* D, void* Z, void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_expert_linear_desc& d = h->d;
  if (!A || !B || !offsets || !D) return fail(GEMM_EPI_ERR_INVALID_ARG, "A, B, offsets and D are required");
  if ((bias != nullptr) != (d.bias_dtype != GEMM_EPI_NONE) || (scale_a != nullptr) != (d.scale_a != 0) ||
      (scale_b != nullptr) != (d.scale_b != 0) || (U != nullptr) != (d.mul != 0) || (Z != nullptr) != (d.z != 0))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "bias, scale_a, scale_b, U and Z must be given exactly as the plan says");
  int rc = aligned4(offsets);
  if (!rc) rc = aligned4(scale_a);
  for (const void* p : {A, B, bias, (const void*)scale_b, U, (const void*)D, (const void*)Z})
    if (!rc) rc = aligned16(p);
  if (rc) return rc;
  if (D == U && d.ldd != d.ldu) return fail(GEMM_EPI_ERR_INVALID_ARG, "D may be U only with the same row stride");
  if (D == Z || (Z && Z == U)) return fail(GEMM_EPI_ERR_INVALID_ARG, "Z may not be D or U");
  for (const void* p : {A, B, bias, (const void*)scale_a, (const void*)scale_b, (const void*)offsets})
    if (p && (p == D || p == Z)) return fail(GEMM_EPI_ERR_INVALID_ARG, "D and Z may not be an operand");
  rc = check_device(h->device);
  if (rc) return rc;
  GroupParams p = {};
  p.A = A;
  p.B = B;
  p.D = D;
  p.M = d.rows;
  p.N = d.N;
  p.K = d.K;
  p.alpha = 1.0f;
  p.d_dtype = d.d_dtype;
  p.scale_a = scale_a;
  p.scale_b = scale_b;
  p.bias = bias;
  p.R = U;
  p.Z = Z;
  p.lda = d.lda;
  p.ldb = d.K;
  p.ldd = d.ldd;
  p.ldr = d.ldu;
  p.ldz = d.ldz;
  p.bias_dtype = d.bias_dtype;
  p.act = d.act;
  p.offsets = offsets;
  p.groups = d.experts;
  p.rows = (int32_t)d.rows;
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();  // clear a stale error so the check below is ours
  if (h->variant >= kTiles) {
    launch_grouped_rows(d.ab_dtype, kRowsBlocks[h->variant - kTiles], p, (int)h->grid, s);
    return launched();
  }
  p.L = 1;
  p.tiles_n = (int32_t)h->tiles_n;
  p.group_m = h->tiles_n > 32 ? 8 : 4;
  p.xcd_remap = 1;
  kParts[kGrouped[h->variant].part](h->variant, p, (int)h->grid, s);
  return launched();
}

extern "C" int gemm_epi_expert_linear_destroy(gemm_epi_expert_linear_handle* h) {
  delete h;
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_expert_linear_get_plan(const gemm_epi_expert_linear_handle* h, gemm_epi_plan* out) {
  clear_error();
  if (!h || !out) return fail(GEMM_EPI_ERR_INVALID_ARG, "NULL argument");
  std::memset(out, 0, sizeof *out);
  out->variant = h->variant;
  const gemm_epi_expert_linear_desc& d = h->d;
  if (h->variant >= kTiles) {
    const int mb = kRowsBlocks[h->variant - kTiles];
    out->tile_m = 4 * mb;
    out->tile_n = 16;
    out->threads = (mb == 1 ? 8 : 4) * 64;
    out->tiles = h->grid * h->tiles_n;
    out->grid = (int)std::min<int64_t>(out->tiles, INT32_MAX);
  } else {
    const GroupedVariant& v = kGrouped[h->variant];
    out->tile_m = v.bm;
    out->tile_n = v.bn;
    out->tile_k = v.bk;
    out->threads = 256;
    out->lds_bytes = v.lds;
    out->tiles = worst_chunks(d.rows, d.experts, v.bm) * h->tiles_n;
    out->grid = (int)h->grid;
  }
  out->cus = h->cus;
  out->splits = 1;
  std::snprintf(out->name, sizeof out->name, "%s", gemm_epi_expert_linear_variant_name(h->variant));
  return GEMM_EPI_OK;
}

extern "C" int gemm_epi_expert_linear_variant_count(void) { return kVariants; }

extern "C" const char* gemm_epi_expert_linear_variant_name(int variant) {
  if (variant < 0 || variant >= kVariants) return nullptr;
  return variant < kTiles ? kGrouped[variant].name : kRowsNames[variant - kTiles];
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
namespace {

constexpr int kGradKTile = 64;
// dbias straight from dD's rows (no activation and mul): a workgroup adds up 64 columns
// of an expert's rows, 2 us for 1024 of them.  The rows may all be one expert's.  With dB
// its tiles take longer over the same rows; without, of more than kSumRows, workgroups add
// up kSumChunk each and a second launch (4 us) joins them.  65536 rows of 8 experts,
// 512 x 512, dA and dbias: even 59 us, 40960 of one expert 73; each expert's at once 64 and
// 138.  16384 rows: 17 and 29, in chunks 18.5 and 22.
constexpr int64_t kSumRows = 16384, kSumChunk = 1024;

// Modelled time (us) of the products with the rows spread evenly, with the linear
// backward's figures: an item takes 1.1 us per K tile with 256x256 tiles, 0.45 (a
// pair on a compute unit 0.85) with 128x128 and 0.16 (0.38) with 64x64 ones, and 8,
// 4 or 2.2 us besides; in more than one round dB's, which mostly store, 5, 2 and 2
// more, and those of an expert without rows half of that.  Over 24 shapes of 1 to 8192
// tokens and 4 to 128 experts the choice is within 2 % of the best tile.
double grad_time(const gemm_epi_expert_linear_grad_desc& d, int tile, int cus) {
  const int64_t n = std::min<int64_t>(d.rows, d.experts), per = (d.rows + n - 1) / n;
  const bool da = d.da_dtype != GEMM_EPI_NONE, db = d.db_dtype != GEMM_EPI_NONE;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const double ia = da ? (double)(n * up(per, tile) * up(d.K, tile)) : 0.0;
  const double tiles = db ? (double)(up(d.N, tile) * up(d.K, tile)) : 0.0;
  const double ib = (double)n * tiles, empty = (double)(d.experts - n) * tiles, items = ia + ib + empty;
  const bool pairs = tile != 256 && items > cus;
  const double slots = pairs ? 2.0 * cus : cus;
  const double tk = tile == 256 ? 1.1 : tile == 128 ? (pairs ? 0.85 : 0.45) : (pairs ? 0.38 : 0.16);
  const double fixed = tile == 256 ? 8.0 : tile == 128 ? 4.0 : 2.2;
  const double store = fixed + (items <= slots ? 0.0 : tile == 256 ? 5.0 : 2.0);
  const double la = fixed + tk * (double)up(d.N, kGradKTile), lb = store + tk * (double)up(per, kGradKTile);
  const double total = ia * la + ib * lb + empty * 0.5 * store;
  const double last = da ? la : lb, longest = std::max(da ? la : 0.0, db ? lb : 0.0);
  return items <= slots ? longest : std::max(longest, total / slots + 0.5 * last);
}

}  // namespace

struct gemm_epi_expert_linear_grad_handle {
  gemm_epi_expert_linear_grad_desc d;
  int device, cus;
  int tile;
  int64_t chunk, slots;   // rows of a chunk of the elementwise pass, and chunks at most
  int64_t ga, gb, sums;   // workgroups of the products and of the column sums
  int64_t ws_bytes;
  bool sum_rows;  // dbias from dD's rows, beside the products
  bool sum_chunks() const { return sum_rows && d.rows > kSumRows && d.db_dtype == GEMM_EPI_NONE; }
  bool pass() const { return has_z() || (d.dbias_dtype != GEMM_EPI_NONE && !sum_rows); }
  bool has_z() const { return d.act != GEMM_EPI_ACT_NONE || d.mul; }
};

extern "C" int gemm_epi_expert_linear_grad_create(const gemm_epi_expert_linear_grad_desc* desc,
                                                  gemm_epi_expert_linear_grad_handle** out) {
  clear_error();
  if (!out) return fail(GEMM_EPI_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!desc) return fail(GEMM_EPI_ERR_INVALID_ARG, "desc is NULL");
  const gemm_epi_expert_linear_grad_desc& d = *desc;
  int rc = check_sizes(d.rows, d.N, d.K, d.experts);
  if (rc) return rc;
  if (!is_type(d.ab_dtype)) return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown ab_dtype %d", d.ab_dtype);
  if (d.ab_dtype != GEMM_EPI_F16 && d.ab_dtype != GEMM_EPI_BF16)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "the backward takes fp16 or bf16 tensors");
  if (d.act < GEMM_EPI_ACT_NONE || d.act > GEMM_EPI_ACT_SILU)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "unknown activation %d", d.act);
  if (!flag_ok(d.mul)) return fail(GEMM_EPI_ERR_INVALID_ARG, "mul must be 0 or 1");
  for (int t : {d.da_dtype, d.db_dtype, d.dbias_dtype})
    if (t != GEMM_EPI_NONE && !is_float_out(t))
      return fail(GEMM_EPI_ERR_INVALID_ARG, "a gradient's type must be NONE, F16, BF16 or F32");
  if (d.da_dtype == GEMM_EPI_NONE && d.db_dtype == GEMM_EPI_NONE && d.dbias_dtype == GEMM_EPI_NONE && !d.mul)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "no gradient is wanted");
  if (d.tile != 0 && d.tile != 64 && d.tile != 128 && d.tile != 256)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "tile must be 0, 64, 128 or 256 (got %d)", d.tile);
  if (d.N % 8 || d.K % 8)
    return fail(GEMM_EPI_ERR_ALIGNMENT, "rows of dD (%lld elements) and of A and B (%lld) must be multiples of 16 bytes",
                (long long)d.N, (long long)d.K);
  // 256 rows of an output or a K-major operand, and what a product reads across
  // its rows (dA: an expert's B, dB: all rows of A and dZ), are addressed with
  // 31-bit byte offsets
  const int64_t pad = 2 * kGradKTile;
  if (d.K * 4 * 256 > INT32_MAX || d.N * 4 * 256 > INT32_MAX)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "rows too long for 31-bit tile offsets");
  if ((d.da_dtype != GEMM_EPI_NONE && (d.N + pad) * d.K * 2 > INT32_MAX) ||
      (d.db_dtype != GEMM_EPI_NONE && (d.rows + pad) * std::max(d.N, d.K) * 2 > INT32_MAX))
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "an operand read across its rows is 2 GiB or larger");
  int device = 0, cus = 0;
  rc = device_query(&device, &cus);
  if (rc) return rc;
  gemm_epi_expert_linear_grad_handle h = {};
  h.d = d;
  h.device = device;
  h.cus = cus;
  double best = 0.0;
  for (const int tile : {256, 128, 64}) {
    if (d.tile != 0 && d.tile != tile) continue;
    const double us = grad_time(d, tile, cus);
    if (h.tile == 0 || us < best) best = us, h.tile = tile;
  }
  const int64_t tn = (d.N + h.tile - 1) / h.tile, tk = (d.K + h.tile - 1) / h.tile;
  h.ga = d.da_dtype != GEMM_EPI_NONE ? worst_chunks(d.rows, d.experts, h.tile) * tk : 0;
  h.gb = d.db_dtype != GEMM_EPI_NONE ? 8 * d.experts * ((tn * tk + 7) / 8) : 0;
  const bool dbias = d.dbias_dtype != GEMM_EPI_NONE;
  h.sum_rows = dbias && !h.has_z() && h.ga + h.gb > 0;
  const int64_t columns = h.sum_rows ? 64 : 256;
  const int64_t parts = h.sum_chunks() ? worst_chunks(d.rows, d.experts, kSumChunk) : d.experts;
  h.sums = dbias ? parts * ((d.N + columns - 1) / columns) : 0;
  // 256 threads for each, fewer than 2^32 in all
  if (h.ga + h.gb + h.sums >= int64_t(1) << 24) return fail(GEMM_EPI_ERR_UNSUPPORTED, "2^24 or more work items");
  // rows per workgroup of the elementwise pass: 64, fewer as long as there are under
  // four workgroups for a compute unit, more where 2^16 chunks would not do
  h.chunk = 64;
  while (h.chunk > 8 && (d.N + 255) / 256 * worst_chunks(d.rows, d.experts, h.chunk) < 4 * cus) h.chunk /= 2;
  while (worst_chunks(d.rows, d.experts, h.chunk) > 65535) h.chunk *= 2;
  if (h.sum_chunks()) h.chunk = kSumChunk;
  h.slots = worst_chunks(d.rows, d.experts, h.chunk);
  h.ws_bytes = dbias && (!h.sum_rows || h.sum_chunks()) ? up256(h.slots * d.N * 4) : 0;
  *out = new (std::nothrow) gemm_epi_expert_linear_grad_handle(h);
  return *out ? GEMM_EPI_OK : fail(GEMM_EPI_ERR_HOST_ALLOC, "out of host memory");
}

extern "C" int gemm_epi_expert_linear_grad_run(const gemm_epi_expert_linear_grad_handle* h, const void* dD,
                                               const void* A, const void* B, const int32_t* offsets, const void* Z,
                                               const void* U, const void* dB_in, void* dZ, void* dU, void* dA,
                                               void* dB, void* dbias, void* workspace, int64_t workspace_bytes,
                                               void* stream) {
  clear_error();
  if (!h) return fail(GEMM_EPI_ERR_INVALID_ARG, "handle is NULL");
  const gemm_epi_expert_linear_grad_desc& d = h->d;
  const bool has_z = h->has_z(), da = d.da_dtype != GEMM_EPI_NONE, db = d.db_dtype != GEMM_EPI_NONE;
  if (!dD || !offsets) return fail(GEMM_EPI_ERR_INVALID_ARG, "dD and offsets are required");
  if ((Z != nullptr) != has_z || (dZ != nullptr) != has_z)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "Z and dZ must be given exactly with an activation or mul");
  if ((U != nullptr) != (d.mul != 0) || (dU != nullptr) != (d.mul != 0))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "U and dU must be given exactly with mul");
  if ((dA != nullptr) != da || (B != nullptr) != da)
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dA and B must be given exactly when da_dtype is set");
  if ((dB != nullptr) != db || (A != nullptr) != db || (dB_in && !dB))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dB and A (and dB_in) must be given exactly when db_dtype is set");
  if ((dbias != nullptr) != (d.dbias_dtype != GEMM_EPI_NONE))
    return fail(GEMM_EPI_ERR_INVALID_ARG, "dbias must be given exactly when dbias_dtype is set");
  int rc = aligned4(offsets);
  const void* in[] = {dD, Z, U, A, B, dB_in, offsets};
  const void* outp[] = {dZ, dU, dA, dB, dbias};
  for (int i = 0; i < 6; ++i)
    if (!rc) rc = aligned16(in[i]);
  for (int i = 0; i < 5; ++i) {
    const void* o = outp[i];
    if (!o) continue;
    if (!rc) rc = aligned16(o);
    if (rc) return rc;
    for (const void* p : in)
      if (p == o && !(i == 0 && (p == dD || p == Z)) && !(i == 1 && p == U) && !(i == 3 && p == dB_in))
        return fail(GEMM_EPI_ERR_INVALID_ARG,
                    "a gradient may not be an input (dZ may be dD or Z, dU may be U, dB may be dB_in)");
    for (int j = 0; j < i; ++j)
      if (outp[j] == o) return fail(GEMM_EPI_ERR_INVALID_ARG, "two gradients share a pointer");
  }
  if (!rc) rc = check_workspace(workspace, workspace_bytes, h->ws_bytes);
  if (!rc) rc = check_device(h->device);
  if (rc) return rc;

  hipStream_t s = (hipStream_t)stream;
  GroupParams g = {};
  g.M = d.rows;
  g.offsets = offsets;
  g.groups = d.experts;
  g.rows = (int32_t)d.rows;
  g.alpha = 1.0f;
  g.L = 1;
  g.xcd_remap = 1;
  g.act = d.act;
  (void)hipGetLastError();  // clear a stale error so the checks below are ours
  if (h->pass()) {
    GroupActParams p = {};
    (GroupParams&)p = g;
    p.N = d.N;
    p.dD = dD;
    p.U = U;
    p.dZin = Z;
    p.dZ = dZ;
    p.dU = dU;
    p.partial = dbias ? (float*)workspace : nullptr;
    p.chunk = (int32_t)h->chunk;
    launch_grouped_act(d.ab_dtype, p, (int)h->slots, s);
    rc = launched();
    if (rc) return rc;
  }
  if (h->ga + h->gb + h->sums == 0) return GEMM_EPI_OK;
  GroupGradParams p = {};
  const void* dz = has_z ? dZ : dD;
  p.a = g;
  p.a.A = dz;
  p.a.B = B;
  p.a.D = dA;
  p.a.N = d.K;
  p.a.K = d.N;
  p.a.lda = d.N;
  p.a.ldd = p.a.ldr = p.a.ldz = d.K;
  p.a.d_dtype = d.da_dtype;
  p.a.tiles_n = (int32_t)((d.K + h->tile - 1) / h->tile);
  p.a.group_m = p.a.tiles_n > 32 ? 8 : 4;
  p.b = p.a;
  p.b.A = dz;
  p.b.B = A;
  p.b.D = dB;
  p.b.R = dB_in;
  p.b.M = d.N;
  p.b.N = d.K;
  p.b.K = d.rows;
  p.b.d_dtype = d.db_dtype;
  p.b.tiles_m = (int32_t)((d.N + h->tile - 1) / h->tile);
  p.b.tiles_total = d.experts * p.b.tiles_m * p.b.tiles_n;
  // the last items should be short ones: dA's are N long, dB's (the longest first) and
  // the column sums the experts' rows.  (Sums behind dA: 65536 rows of 8 experts, 40960
  // of one, 256 x 512, both products: 188 us for 155.)
  p.b_first = d.rows > d.experts * d.N;
  p.ga = (int32_t)h->ga;
  p.gb = (int32_t)h->gb;
  p.sums = (int32_t)h->sums;
  p.sum_rows = h->sum_rows ? dD : nullptr;
  p.row_sums = h->sum_chunks() ? (float*)workspace : nullptr;
  p.partial = (const float*)workspace;
  p.chunk = (int32_t)h->chunk;
  p.dbias = dbias;
  p.dbias_dtype = d.dbias_dtype;
  p.N = d.N;
  const int kind = h->tile == 256 ? GRAD_256 : h->tile == 64 ? GRAD_64 : h->ga + h->gb > h->cus ? GRAD_128 : GRAD_128_DEEP;
  static void (*const kLaunch[2][kGradKinds])(const GroupGradParams&, hipStream_t) = {
      {launch_grouped_grad<T_F16, 0>, launch_grouped_grad<T_F16, 1>, launch_grouped_grad<T_F16, 2>,
       launch_grouped_grad<T_F16, 3>},
      {launch_grouped_grad<T_BF16, 0>, launch_grouped_grad<T_BF16, 1>, launch_grouped_grad<T_BF16, 2>,
       launch_grouped_grad<T_BF16, 3>}};
  const auto launch = kLaunch[d.ab_dtype == GEMM_EPI_BF16][kind];
  launch(p, s);
  rc = launched();
  if (rc || !h->sum_chunks()) return rc;
  p.ga = p.gb = 0;
  p.sums = (int32_t)(d.experts * ((d.N + 255) / 256));
  p.sum_rows = nullptr;
  launch(p, s);
  return launched();
}

extern "C" int gemm_epi_expert_linear_grad_destroy(gemm_epi_expert_linear_grad_handle* h) {
  delete h;
  return GEMM_EPI_OK;
}

extern "C" int64_t gemm_epi_expert_linear_grad_workspace(const gemm_epi_expert_linear_grad_handle* h) {
  return h ? h->ws_bytes : -1;
}
