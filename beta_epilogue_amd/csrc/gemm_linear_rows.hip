// gemm_linear_rows.hip -- the linear layer with few rows (tokens), and the
// join of a split-K plan's slices.
//
// Few rows: D is M x N with M <= 64, so the time is the weight's: every byte
// of B is read once and meets at most 64 tokens.  The MFMA's roles are turned
// round: 16 weight rows are the matrix core's rows and the tokens (NB blocks of
// 16) its columns, so a weight fragment feeds NB instructions.
//
// What bounds it is how the weights arrive.  Read straight into fragments (16
// rows, 64 bytes each, per load) they come at 4.4 TB/s; the kernel has them
// arrive in LDS by DMA in runs of 256 bytes per row, into a ring that belongs
// to one wave, so waves never wait for one another: 5.1 TB/s for bf16 with one
// token and K = N = 8192 (26.1 us; 30.8 before; runs of 512 and 1024 bytes are
// 5 to 15 % slower, for each wave then has fewer rows in flight).  The tokens
// take the same way.  The waves of a workgroup split K in interleaved runs and
// join their sums through LDS in wave order.  Sixteen e4m3 tokens at 8192^2
// take 15.5 us (4.3 TB/s), 32 bf16 ones at 4096^2 10.7 us (tiles: 12.7 us).
// e4m3 is widened to fp16 in registers (exact), so every type has exact
// products and fp32 (int32) sums.
#include "gemm_linear.hpp"

namespace gemm_epi {

namespace {

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

// The DMA of the weights: as dma16s, with the streaming cache policy.
template <uint32_t IMM>
__device__ __forceinline__ void dma16s_nt(v4i rsrc, uint32_t sbase, uint32_t voff, uint32_t soff) {
  asm volatile(
      "s_add_u32 m0, %0, %4\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen nt lds"
      :
      : "s"(sbase), "v"(voff), "s"(rsrc), "s"(soff), "i"(IMM)
      : "memory", "m0", "scc");
}

// One stage of a wave's ring: 256 bytes of K of 16 weight rows, then of 4 * MB
// token rows; 1 KiB (four rows) per DMA instruction.  The 16-byte chunk c of
// row r lies at c ^ (r & 15), so a fragment read (16 rows, one chunk each) hits
// 16 distinct bank groups.  NW waves, NS stages.
constexpr int kSeg = 256;

template <int AB, int MB, int NW, int NS>
__global__ __launch_bounds__(NW * 64) void linear_rows_kernel(LinParams p) {
  using MM = RowsMma<AB>;
  constexpr int ES = AB == T_F16 || AB == T_BF16 ? 2 : 1;
  constexpr int NB = (MB + 3) / 4;               // token blocks of 16
  constexpr int PER = 4 + MB;                    // DMA instructions (KiB) per stage
  constexpr int RING = NW * NS * PER * 1024, JOIN = NW * NB * 1024;
  static_assert(NS * PER < 64, "counted waits");
  __shared__ __attribute__((aligned(1024))) char lds[RING > JOIN ? RING : JOIN];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;

  // Rows past the matrix and chunks past K get an offset outside the
  // resource's extent and arrive as zeros.
  const int64_t lda = p.lda * ES, ldb = p.ldb * ES;
  const uint32_t kbytes = (uint32_t)(p.K * ES);
  const int brows = (int)min((int64_t)16, p.N - n0);
  const v4i rb = make_rsrc((const char*)p.B + n0 * ldb, (uint32_t)((brows - 1) * ldb + kbytes));
  const v4i ra = make_rsrc(p.A, (uint32_t)((p.M - 1) * lda + kbytes));
  // DMA lane: row 4 * instruction + q, chunk position r
  uint32_t ob[4], oa[MB], cb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cb[i] = (uint32_t)((r ^ (4 * i + q)) * 16);  // logical chunk of row 4 i + q (mod 16)
    ob[i] = 4 * i + q < brows ? (uint32_t)((4 * i + q) * ldb) + cb[i] : 0x80000000u;
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) oa[i] = 4 * i + q < p.M ? (uint32_t)((4 * i + q) * lda) + cb[i & 3] : 0x80000000u;
  const uint32_t ring = (uint32_t)(uintptr_t)(lds_void_t*)lds + (uint32_t)wave * (NS * PER * 1024);

  // The outputs this wave finishes: token block `wave`, whose bias, scales and
  // residual are read ahead.
  static_assert(NB <= NW, "a wave finishes at most one block");
  const int64_t fm = wave * 16 + r, fn = n0 + 4 * q;
  const bool fin = wave < NB && fm < p.M && fn < p.N;
  Epi4 epi;
  if (fin) epi.load(p, fm, fn);

  typename MM::acc_t acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = typename MM::acc_t{};

  // Segment k (bytes) of every row into stage st.
  auto issue = [&](int st, uint32_t k) {
    const uint32_t base = ring + (uint32_t)(st * (PER * 1024));
    static_for<0, 4>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      dma16s_nt<i * 1024u>(rb, base, k + cb[i] < kbytes ? ob[i] + k : 0x80000000u, 0);
    });
    static_for<0, MB>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      dma16s<(4 + i) * 1024u>(ra, base, k + cb[i & 3] < kbytes ? oa[i] + k : 0x80000000u, 0);
    });
  };
  const uint32_t step = NW * kSeg;
  uint32_t k = (uint32_t)wave * kSeg;
#pragma unroll
  for (int st = 0; st < NS; ++st) issue(st, k + (uint32_t)st * step);
  // (segments past K are issued too, without traffic, so the counts hold)
  int st = 0;
  for (; k < kbytes; k += step) {
    wait_vmcnt<(NS - 1) * PER>();
    asm volatile("" ::: "memory");
    const char* sb = lds + wave * (NS * PER * 1024) + st * (PER * 1024);
    v4u fb[4], fa[4][NB];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      fb[s] = *(const v4u*)(sb + r * kSeg + (((s * 4 + q) ^ r) << 4));
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        // (a block with fewer rows: lanes beyond them read a row again, into columns nobody reads)
        const int row = (j * 16 + r) % (4 * MB);
        fa[s][j] = *(const v4u*)(sb + 4096 + row * kSeg + (((s * 4 + q) ^ (row & 15)) << 4));
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read out before it is filled again
    issue(st, k + NS * step);
    st = st + 1 == NS ? 0 : st + 1;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const typename MM::frag_t b = MM::prep(fb[s]);
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[j] = MM::mma(b, MM::prep(fa[s][j]), acc[j]);
    }
  }
  wait_vmcnt<0>();  // no DMA may land in what follows
  __syncthreads();
  v4u(*part)[NB][64] = (v4u(*)[NB][64])lds;
#pragma unroll
  for (int j = 0; j < NB; ++j) part[wave][j][lane] = __builtin_bit_cast(v4u, acc[j]);
  __syncthreads();
  if (!fin) return;
  // lane (q, r) holds weight rows 4q .. 4q+3 of token r
  typename MM::acc_t sum = __builtin_bit_cast(typename MM::acc_t, part[0][wave][lane]);
#pragma unroll
  for (int w = 1; w < NW; ++w) sum += __builtin_bit_cast(typename MM::acc_t, part[w][wave][lane]);
  epi.finish(p, fm, fn, v4f{(float)sum[0], (float)sum[1], (float)sum[2], (float)sum[3]});
}

// ---------------------------------------------------------------------------
// Split K: slice s of split tile dp_tiles + j left its partial sums in slot
// s * tail_tiles + j, packed rows x cols.  A thread takes four consecutive
// columns.
// ---------------------------------------------------------------------------
template <bool INT>
__device__ __forceinline__ void join_slices(const LinParams& p, int tile_m, int tile_n, int64_t block, int64_t blocks) {
  const int64_t slot = (int64_t)tile_m * tile_n, per_tile = slot / 4;
  const int64_t groups = (int64_t)p.tail_tiles * per_tile;
  const int64_t stride = blocks * 256;
  for (int64_t g = block * 256 + threadIdx.x; g < groups; g += stride) {
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
    const int64_t step = (int64_t)p.tail_tiles * slot;
    // slices are added in order, four loads in flight at a time
    typedef typename std::conditional<INT, v4i, v4f>::type acc_t;
    acc_t sum = {};
    int s = 0;
    for (; s + 4 <= p.splits; s += 4) {
      acc_t v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = *(const acc_t*)(src + (s + u) * step);
#pragma unroll
      for (int u = 0; u < 4; ++u) sum += v[u];
    }
    acc_t v[3];
#pragma unroll
    for (int u = 0; u < 3; ++u)
      if (s + u < p.splits) v[u] = *(const acc_t*)(src + (s + u) * step);
#pragma unroll
    for (int u = 0; u < 3; ++u)
      if (s + u < p.splits) sum += v[u];
    const v4f acc = {(float)sum[0], (float)sum[1], (float)sum[2], (float)sum[3]};
    epi.finish(p, m0 + row, n0 + col, acc);
  }
}

template <bool INT>
__global__ __launch_bounds__(256) void linear_splitk_kernel(LinParams p, int tile_m, int tile_n) {
  join_slices<INT>(p, tile_m, tile_n, blockIdx.x, gridDim.x);
}

// Both products of a backward: the first `ja` workgroups join a's tiles.
__global__ __launch_bounds__(256) void linear_grad_join_kernel(LinParams a, LinParams b, int ja, int tile) {
  if ((int)blockIdx.x < ja) join_slices<false>(a, tile, tile, blockIdx.x, ja);
  else join_slices<false>(b, tile, tile, blockIdx.x - ja, gridDim.x - ja);
}

template <int AB, int MB, int NW, int NS>
void rows(const LinParams& p, hipStream_t s) {
  hipLaunchKernelGGL((linear_rows_kernel<AB, MB, NW, NS>), dim3((unsigned)((p.N + 15) / 16)), dim3(NW * 64), 0, s, p);
}

template <int AB>
void rows_ab(int nw, const LinParams& p, hipStream_t s) {
  if (p.M <= 4) rows<AB, 1, 8, 2>(p, s);
  else if (p.M <= 8) rows<AB, 2, 8, 2>(p, s);
  else if (p.M <= 16) nw == 8 ? rows<AB, 4, 8, 2>(p, s) : rows<AB, 4, 4, 2>(p, s);
  else if (p.M <= 32) nw == 8 ? rows<AB, 8, 8, 1>(p, s) : rows<AB, 8, 4, 1>(p, s);
  else nw == 8 ? rows<AB, 16, 8, 1>(p, s) : rows<AB, 16, 4, 1>(p, s);
}

}  // namespace

void launch_linear_rows(int ab, int nw, const LinParams& p, hipStream_t s) {
  if (ab == T_F16) rows_ab<T_F16>(nw, p, s);
  else if (ab == T_BF16) rows_ab<T_BF16>(nw, p, s);
  else if (ab == T_E4M3) rows_ab<T_E4M3>(nw, p, s);
  else rows_ab<T_I8>(nw, p, s);
}

void launch_linear_splitk(const LinParams& p, int tile_m, int tile_n, bool int_path, int grid, hipStream_t s) {
  if (int_path) hipLaunchKernelGGL(linear_splitk_kernel<true>, dim3(grid), dim3(256), 0, s, p, tile_m, tile_n);
  else hipLaunchKernelGGL(linear_splitk_kernel<false>, dim3(grid), dim3(256), 0, s, p, tile_m, tile_n);
}

void launch_linear_grad_join(const LinParams& a, const LinParams& b, int tile, int64_t most_blocks, hipStream_t s) {
  auto blocks = [&](const LinParams& p) {
    const int64_t n = ((int64_t)p.tail_tiles * tile * tile / 4 + 255) / 256;
    return (int)(n < most_blocks ? n : most_blocks);
  };
  const int ja = blocks(a), jb = blocks(b);
  hipLaunchKernelGGL(linear_grad_join_kernel, dim3(ja + jb), dim3(256), 0, s, a, b, ja, tile);
}

}  // namespace gemm_epi
