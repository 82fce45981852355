// gemm_linear_rows.hpp -- the body of the few-row kernels (gemm_linear_rows.hip,
// which says how they work) and their epilogue of four columns, also for other
// kernels whose rows are few.
#pragma once

#include "gemm_linear.hpp"

namespace gemm_epi {

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

// The epilogue of four consecutive columns n .. n+3 of row m.  MUL: R multiplies.
template <bool MUL = false>
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
    if (p.R) z = MUL ? z * res : z + res;
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
struct RowsLds {
  static constexpr int PER = 4 + MB;  // DMA instructions (KiB) per stage
  static constexpr int RING = NW * NS * PER * 1024, JOIN = NW * ((MB + 3) / 4) * 1024;
  static constexpr int BYTES = RING > JOIN ? RING : JOIN;
};

// The products of up to 16 weight rows with p.M <= 4 * MB tokens (the rows of p.A),
// with the LDS array `lds` (1 KiB aligned).  weights: a buffer resource; place(i): the
// byte in it at which weight row i begins (0x80000000: there is none).  begin(m, n)
// is called before the products by the lane that finishes weight rows n .. n + 3 of
// token m, where there are such, and finish(m, n, sums) after them; more(acc): what a
// wave adds to its part of the sums.
template <int AB, int MB, int NW, int NS, class PLACE, class BEGIN, class MORE, class FINISH>
__device__ __forceinline__ void rows_products(const LinParams& p, v4i weights, PLACE&& place, char* lds, BEGIN&& begin,
                                              MORE&& more, FINISH&& finish) {
  using MM = RowsMma<AB>;
  constexpr int ES = AB == T_F16 || AB == T_BF16 ? 2 : 1;
  constexpr int NB = (MB + 3) / 4;               // token blocks of 16
  constexpr int PER = RowsLds<AB, MB, NW, NS>::PER;
  static_assert(NS * PER < 64, "counted waits");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;

  // Rows past the matrix and chunks past K get an offset outside the
  // resource's extent and arrive as zeros.
  const int64_t lda = p.lda * ES;
  const uint32_t kbytes = (uint32_t)(p.K * ES);
  const v4i rb = weights;
  const v4i ra = make_rsrc(p.A, (uint32_t)((p.M - 1) * lda + kbytes));
  // DMA lane: row 4 * instruction + q, chunk position r
  uint32_t ob[4], oa[MB], cb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cb[i] = (uint32_t)((r ^ (4 * i + q)) * 16);  // logical chunk of row 4 i + q (mod 16)
    const uint32_t at = place(4 * i + q);
    ob[i] = at != 0x80000000u ? at + cb[i] : 0x80000000u;
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) oa[i] = 4 * i + q < p.M ? (uint32_t)((4 * i + q) * lda) + cb[i & 3] : 0x80000000u;
  const uint32_t ring = (uint32_t)(uintptr_t)(lds_void_t*)lds + (uint32_t)wave * (NS * PER * 1024);

  // The outputs this wave finishes: token block `wave`, whose bias, scales and
  // residual are read ahead.
  static_assert(NB <= NW, "a wave finishes at most one block");
  const int fm = wave * 16 + r, fn = 4 * q;
  const bool fin = wave < NB && fm < p.M;
  if (fin) begin(fm, fn);

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
  more(acc);
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
  finish(fm, fn, v4f{(float)sum[0], (float)sum[1], (float)sum[2], (float)sum[3]});
}

// Columns n0 .. n0 + 15 of D for p.M <= 4 * MB tokens.
template <int AB, int MB, int NW, int NS, bool MUL, class MORE>
__device__ __forceinline__ void linear_rows_body(const LinParams& p, int64_t n0, char* lds, MORE&& more) {
  constexpr int ES = AB == T_F16 || AB == T_BF16 ? 2 : 1;
  const int64_t ldb = p.ldb * ES;
  const int brows = (int)min((int64_t)16, p.N - n0);
  const v4i rb = make_rsrc((const char*)p.B + n0 * ldb, (uint32_t)((brows - 1) * ldb + p.K * ES));
  Epi4<MUL> epi;
  rows_products<AB, MB, NW, NS>(
      p, rb, [&](int i) { return i < brows ? (uint32_t)(i * ldb) : 0x80000000u; }, lds,
      [&](int m, int n) {
        if (n0 + n < p.N) epi.load(p, m, n0 + n);
      },
      more,
      [&](int m, int n, v4f sum) {
        if (n0 + n < p.N) epi.finish(p, m, n0 + n, sum);
      });
}

}  // namespace gemm_epi
