// gemm_linear_rows.hip -- the linear layer with few rows (tokens), and the
// join of a split-K plan's slices.
//
// Few rows: D is M x N with M <= 64, so the time is the weight's: every byte
// of B is read once and meets at most 64 tokens.  The MFMA's roles are turned
// round: 16 (RB times) weight rows are the matrix core's rows, the tokens
// (NB blocks of 16) its columns, so one weight fragment loaded from memory
// feeds NB instructions.  Fragments go from global memory straight into
// registers (a lane's 16 bytes are 16 / ES consecutive k of one row, the four
// lane groups cover 64 consecutive bytes of each row): nothing of B is used
// twice by a workgroup, so LDS would only add a copy.  The eight waves of a
// workgroup split K in interleaved segments (each reads U * 64 bytes of a row
// at a time, eight waves together a contiguous run) and join through LDS in
// wave order; the token fragments come from L2, where all workgroups read the
// same M x K.  e4m3 is widened to fp16 in registers (exact), so every type
// has exact products and fp32 (int32) sums.
#include "gemm_linear.hpp"

namespace gemm_epi {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// Eight e4m3 values (two words) as fp16.
__device__ __forceinline__ v8h widen8(uint32_t a, uint32_t b) {
  const v2h p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
  const v2h p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
  const v2h p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
  const v2h p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  return v8h{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// 16x16 blocks; a fragment is 16 bytes per lane (64 bytes of K per row).
template <int AB> struct RowsMma {
  typedef v4f acc_t;
  typedef v4u frag_t;
  static __device__ __forceinline__ frag_t prep(v4u r) { return r; }
  static __device__ __forceinline__ acc_t mma(frag_t a, frag_t b, acc_t c) {
    if constexpr (AB == T_F16)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0,
                                                     0);
  }
};
template <> struct RowsMma<T_I8> {
  typedef v4i acc_t;
  typedef v4u frag_t;
  static __device__ __forceinline__ frag_t prep(v4u r) { return r; }
  static __device__ __forceinline__ acc_t mma(frag_t a, frag_t b, acc_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), c, 0, 0, 0);
  }
};
// Any assignment of k to lanes serves as long as both operands share it: the
// first MFMA takes the first eight of each lane's sixteen k, the second the rest.
template <> struct RowsMma<T_E4M3> {
  typedef v4f acc_t;
  struct frag_t {
    v8h lo, hi;
  };
  static __device__ __forceinline__ frag_t prep(v4u r) { return frag_t{widen8(r.x, r.y), widen8(r.z, r.w)}; }
  static __device__ __forceinline__ acc_t mma(frag_t a, frag_t b, acc_t c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.lo, b.lo, c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a.hi, b.hi, c, 0, 0, 0);
  }
};

// Four consecutive values of type dt at element i, as fp32.
__device__ __forceinline__ v4f ld4(const void* base, int dt, int64_t i) {
  if (dt == T_F32) return *(const v4f*)((const float*)base + i);
  const v2u u = *(const v2u*)((const uint16_t*)base + i);
  return epi_decode4(v4u{u.x, u.y, 0u, 0u}, dt);
}

__device__ __forceinline__ void st4(void* base, int dt, int64_t i, v4f v) {
  if (dt == T_F32) {
    *(v4f*)((float*)base + i) = v;
  } else if (dt == T_F16) {
    const v4h h = {(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
    *(v4h*)((_Float16*)base + i) = h;
  } else {
    const v4bf b = {(__bf16)v.x, (__bf16)v.y, (__bf16)v.z, (__bf16)v.w};
    *(v4bf*)((__bf16*)base + i) = b;
  }
}

// The epilogue of four consecutive columns n .. n+3 of row m.
struct Epi4 {
  v4f bias, cs, res;
  float sa;
  __device__ __forceinline__ void load(const LinParams& p, int64_t m, int64_t n) {
    sa = p.scale_a ? p.scale_a[m] : 1.0f;
    cs = v4f{p.alpha, p.alpha, p.alpha, p.alpha};
    if (p.scale_b) cs *= *(const v4f*)(p.scale_b + n);
    bias = p.bias ? ld4(p.bias, p.bias_dtype, n) : v4f{};
    res = p.R ? ld4(p.R, p.d_dtype, m * p.ldr + n) : v4f{};
  }
  __device__ __forceinline__ void finish(const LinParams& p, int64_t m, int64_t n, v4f acc) const {
    v4f z;
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = __builtin_fmaf(acc[i], sa * cs[i], bias[i]);
    if (p.Z) st4(p.Z, p.d_dtype, m * p.ldz + n, z);
    with_act(p.act, [&](auto act_c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = act_value<decltype(act_c)::value>(z[i]);
    });
    if (p.R) z += res;
    st4(p.D, p.d_dtype, m * p.ldd + n, z);
  }
};

constexpr int kRowsWaves = 8;

template <int AB, int NB, int RB, int U>
__global__ __launch_bounds__(kRowsWaves * 64) void linear_rows_kernel(LinParams p) {
  using MM = RowsMma<AB>;
  constexpr int ES = AB == T_F16 || AB == T_BF16 ? 2 : 1;
  __shared__ v4u part[kRowsWaves][RB * NB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RB);

  // Buffer resources: the workgroup's weight rows, and all tokens.  Rows past
  // the matrix and bytes past K get an offset outside the extent and read 0.
  const int64_t lda = p.lda * ES, ldb = p.ldb * ES;
  const uint32_t kbytes = (uint32_t)(p.K * ES);
  const int brows = (int)min((int64_t)(16 * RB), p.N - n0);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((const char*)p.B + n0 * ldb), (short)0, (int)((brows - 1) * ldb + kbytes), 0x00020000);
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      (void*)p.A, (short)0, (int)((p.M - 1) * lda + kbytes), 0x00020000);
  uint32_t ob[RB], oa[NB];
#pragma unroll
  for (int i = 0; i < RB; ++i) ob[i] = i * 16 + r < brows ? (uint32_t)((i * 16 + r) * ldb) : 0x80000000u;
#pragma unroll
  for (int j = 0; j < NB; ++j) oa[j] = j * 16 + r < p.M ? (uint32_t)((j * 16 + r) * lda) : 0x80000000u;

  // The outputs this wave finishes: block `wave` of the RB * NB (weight
  // block, token block) pairs; its bias, scales and residual are read ahead.
  constexpr int PAIRS = RB * NB;
  static_assert(PAIRS <= kRowsWaves, "a wave finishes at most one block");
  const int64_t fm = (wave % NB) * 16 + r, fn = n0 + (wave / NB) * 16 + 4 * q;
  const bool fin = wave < PAIRS && fm < p.M && fn < p.N;
  Epi4 epi;
  if (fin) epi.load(p, fm, fn);

  typename MM::acc_t acc[RB][NB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = typename MM::acc_t{};

  for (uint32_t k0 = (uint32_t)wave * (U * 64); k0 < kbytes; k0 += kRowsWaves * U * 64) {
    v4u fb[U][RB], fa[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t k = k0 + u * 64 + q * 16;
      const bool in = k < kbytes;
#pragma unroll
      for (int i = 0; i < RB; ++i)
        fb[u][i] = __builtin_bit_cast(
            v4u, __builtin_amdgcn_raw_buffer_load_b128(rb, (int)(in ? ob[i] + k : 0x80000000u), 0, EPI_NT));
#pragma unroll
      for (int j = 0; j < NB; ++j)
        fa[u][j] = __builtin_bit_cast(
            v4u, __builtin_amdgcn_raw_buffer_load_b128(ra, (int)(in ? oa[j] + k : 0x80000000u), 0, 0));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      typename MM::frag_t a[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) a[j] = MM::prep(fa[u][j]);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const typename MM::frag_t b = MM::prep(fb[u][i]);
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = MM::mma(b, a[j], acc[i][j]);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) part[wave][i * NB + j][lane] = __builtin_bit_cast(v4u, acc[i][j]);
  __syncthreads();
  if (!fin) return;
  // lane (q, r) holds weight rows 4q .. 4q+3 of token r
  typename MM::acc_t sum = __builtin_bit_cast(typename MM::acc_t, part[0][wave][lane]);
#pragma unroll
  for (int w = 1; w < kRowsWaves; ++w) sum += __builtin_bit_cast(typename MM::acc_t, part[w][wave][lane]);
  epi.finish(p, fm, fn, v4f{(float)sum[0], (float)sum[1], (float)sum[2], (float)sum[3]});
}

// ---------------------------------------------------------------------------
// Split K: slice s of split tile dp_tiles + j left its partial sums in slot
// s * tail_tiles + j, packed rows x cols.  A thread takes four consecutive
// columns.
// ---------------------------------------------------------------------------
template <bool INT>
__global__ __launch_bounds__(256) void linear_splitk_kernel(LinParams p, int tile_m, int tile_n) {
  const int64_t slot = (int64_t)tile_m * tile_n, per_tile = slot / 4;
  const int64_t groups = (int64_t)p.tail_tiles * per_tile;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; g < groups; g += stride) {
    const int j = (int)(g / per_tile);
    const int w = (int)(g - (int64_t)j * per_tile);
    const TileRC tc = raster_tile(p.dp_tiles + j, p.tiles_m, p.tiles_n, p.group_m);
    const int64_t m0 = (int64_t)tc.tm * tile_m, n0 = (int64_t)tc.tn * tile_n;
    const int rows = (int)min(p.M - m0, (int64_t)tile_m), cols = (int)min(p.N - n0, (int64_t)tile_n);
    const int row = w / (tile_n / 4), col = (w - row * (tile_n / 4)) * 4;
    if (row >= rows || col >= cols) continue;
    Epi4 epi;
    epi.load(p, m0 + row, n0 + col);
    const uint32_t* src = (const uint32_t*)p.ws + (int64_t)j * slot + (int64_t)row * cols + col;
    v4f acc;
    if constexpr (INT) {
      v4u a = *(const v4u*)src;
      for (int s = 1; s < p.splits; ++s) a += *(const v4u*)(src + (int64_t)s * p.tail_tiles * slot);
      const v4i i = __builtin_bit_cast(v4i, a);
      acc = v4f{(float)i.x, (float)i.y, (float)i.z, (float)i.w};
    } else {
      acc = *(const v4f*)src;
      for (int s = 1; s < p.splits; ++s) acc += *(const v4f*)(src + (int64_t)s * p.tail_tiles * slot);
    }
    epi.finish(p, m0 + row, n0 + col, acc);
  }
}

template <int AB, int NB, int RB>
void rows(const LinParams& p, hipStream_t s) {
  constexpr int U = NB * RB >= 4 ? 2 : 4;
  const int64_t blocks = (p.N + 16 * RB - 1) / (16 * RB);
  hipLaunchKernelGGL((linear_rows_kernel<AB, NB, RB, U>), dim3((unsigned)blocks), dim3(kRowsWaves * 64), 0, s, p);
}

template <int AB>
void rows_ab(int nb, int rb, const LinParams& p, hipStream_t s) {
  if (rb == 1) {
    if (nb == 1) rows<AB, 1, 1>(p, s);
    else if (nb == 2) rows<AB, 2, 1>(p, s);
    else rows<AB, 4, 1>(p, s);
  } else {
    if (nb == 1) rows<AB, 1, 2>(p, s);
    else if (nb == 2) rows<AB, 2, 2>(p, s);
    else rows<AB, 4, 2>(p, s);
  }
}

}  // namespace

void launch_linear_rows(int ab, int nb, int rb, const LinParams& p, hipStream_t s) {
  if (ab == T_F16) rows_ab<T_F16>(nb, rb, p, s);
  else if (ab == T_BF16) rows_ab<T_BF16>(nb, rb, p, s);
  else if (ab == T_E4M3) rows_ab<T_E4M3>(nb, rb, p, s);
  else rows_ab<T_I8>(nb, rb, p, s);
}

void launch_linear_splitk(const LinParams& p, int tile_m, int tile_n, bool int_path, int grid, hipStream_t s) {
  if (int_path) hipLaunchKernelGGL(linear_splitk_kernel<true>, dim3(grid), dim3(256), 0, s, p, tile_m, tile_n);
  else hipLaunchKernelGGL(linear_splitk_kernel<false>, dim3(grid), dim3(256), 0, s, p, tile_m, tile_n);
}

}  // namespace gemm_epi
