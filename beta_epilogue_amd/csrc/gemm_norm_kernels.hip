// gemm_norm_kernels.hip -- the root-mean-square norm with the residual's
// addition, into 16 bits, fp32, or 8 bits with a scale per row, and its
// backward.
//
//   h = x + r (fp32),  s = 1 / sqrt(mean(h^2) + eps),  y = h s w
//   8 bits: scale = max(max|y| / qmax, 2^-126), q = round(y / scale)
//   backward, with s of the stored h and g = dy w:
//     dh = dh_in + s g - h s^3 mean(g h),   dw = sum over rows of dy h s
//
// Both are bound by memory: a row is read once into registers (TPR threads
// with NV groups of 8 elements each), its sums are joined by shuffles and one
// LDS exchange, and the results are written from the registers, so no byte
// moves twice.  All sums and the norm itself are fp32; the only roundings are
// those of the outputs (y and h are both rounded from the fp32 values).
// Groups of 8 are loaded and stored as 16-byte (8-bit: 8-byte) accesses at
// element alignment (gfx950 takes unaligned global accesses), so odd row
// lengths and strides run the same path.
#include "gemm_norm.hpp"

#include "gemm_epi_kernel.hpp"

namespace gemm_epi {

namespace {

template <int T> struct Elem;
template <> struct Elem<T_F16> { typedef _Float16 type; };
template <> struct Elem<T_BF16> { typedef __bf16 type; };
template <> struct Elem<T_F32> { typedef float type; };

typedef v2u v2u_any __attribute__((aligned(1)));

typedef float v8f __attribute__((ext_vector_type(8)));

// Eight elements as stored (16 bytes of a 2-byte type), and their values.
template <int T> struct Group {
  typedef typename Elem<T>::type type __attribute__((ext_vector_type(8)));
  typedef type any __attribute__((aligned(sizeof(typename Elem<T>::type))));
};
template <class G>
__device__ __forceinline__ v8f value8(G g) {
  return __builtin_convertvector(g, v8f);
}

// A thread's group of a row.  The group that the row's end cuts, and those past
// it, lie on the row's last 8 elements, of which the first `dead` belong to other
// threads: they are loaded with the rest, count as 0 and are not stored.  So a
// load is one access without a branch, and the loads of all tensors are in
// flight together (backward of 14545 rows of 2461 fp16: 134 us with the cut groups
// loaded element by element, 66 so).  Rows of less than 8 elements are one group
// with `live` of them.
struct Span {
  int64_t at;
  int dead, live;  // elements [dead, live) are the thread's
};
__device__ __forceinline__ Span span_of(int64_t c, int64_t cols) {
  if (cols < 8) return {0, c == 0 ? 0 : 8, (int)cols};
  const int64_t at = c + 8 <= cols ? c : cols - 8;
  return {at, (int)(c - at < 8 ? c - at : 8), 8};
}
__device__ __forceinline__ bool whole(const Span& g) { return g.dead == 0 && g.live == 8; }

// The group's elements, the dead ones among them.
template <int T>
__device__ __forceinline__ typename Group<T>::type load8(const void* row, const Span& g) {
  const typename Elem<T>::type* p = (const typename Elem<T>::type*)row + g.at;
  typename Group<T>::type v = {};
  if (g.live == 8) {  // (the same for all threads)
    v = *(const typename Group<T>::any*)p;
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < g.live) v[k] = p[k];
  }
  return v;
}

// 0 in the dead places.
template <class V>
__device__ __forceinline__ void bury(const Span& g, V& v) {
  if (g.dead) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < g.dead ? 0 : v[k];
  }
}

template <int T>
__device__ __forceinline__ void store8(void* row, const Span& g, v8f v) {
  typename Elem<T>::type* p = (typename Elem<T>::type*)row + g.at;
  if (whole(g)) {
    *(typename Group<T>::any*)p = __builtin_convertvector(v, typename Group<T>::type);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k >= g.dead && k < g.live) p[k] = (typename Elem<T>::type)v[k];
  }
}

template <int T>
__device__ __forceinline__ v8f load_weight8(const void* w, bool f32, const Span& g) {
  return f32 ? load8<T_F32>(w, g) : value8(load8<T>(w, g));
}

// Rounds to nearest-even into 8 bits and stores: values of at most QMAX (1 + 2^-21),
// which round to QMAX, or in e4m3 NaN, which stays.  int8: adding 1.5 * 2^23 leaves
// the rounded integer in the low byte of the sum.
template <int T>
__device__ __forceinline__ void store8_q(void* row, const Span& g, v8f v) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (T == T_E4M3) {
      int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j], v[4 * j + 1], 0, false);
      w[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j + 2], v[4 * j + 3], b, true);
    } else {
      uint32_t b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) b[k] = __float_as_uint(v[4 * j + k] + 12582912.0f);
      // byte 0 of each sum
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
      w[j] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    }
  }
  uint8_t* p = (uint8_t*)row + g.at;
  if (whole(g)) {
    *(v2u_any*)p = v2u{w[0], w[1]};
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k >= g.dead && k < g.live) p[k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
  }
}

// Joins N values over the TPR threads of a row, in a fixed order; every thread
// gets the results.  red: N words per wave, not written again before the next
// barrier of the row.
struct Sum {
  typedef float type;
  static __device__ __forceinline__ float join(float a, float b) { return a + b; }
};
struct Max {
  typedef uint32_t type;
  static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return a > b ? a : b; }
};
template <class OP, int TPR, int N>
__device__ __forceinline__ void row_join(typename OP::type (&v)[N], typename OP::type* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = OP::join(v[i], __shfl_xor(v[i], d, 64));
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = red[i];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = OP::join(v[i], red[w * N + i]);
  }
}

template <int TPR> constexpr int block_threads() { return TPR > 256 ? TPR : 256; }

template <int TX, int TY, int TPR, int NV>
__global__ __launch_bounds__(block_threads<TPR>()) void rmsnorm_kernel(NormParams p) {
  constexpr int RPB = block_threads<TPR>() / TPR;
  constexpr bool Q = TY == T_E4M3 || TY == T_I8;
  __shared__ float red[TPR / 64];
  __shared__ uint32_t redm[TPR / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TPR;
  if (row >= p.rows) return;  // whole waves, and whole workgroups where rows share barriers
  constexpr int XS = sizeof(typename Elem<TX>::type);
  const char* x = (const char*)p.x + row * p.ldx * XS;
  const char* r = p.r ? (const char*)p.r + row * p.ldr * XS : nullptr;
  Span at[NV];
  typename Group<TX>::type xg[NV], rg[NV];
  v8f h[NV], w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    at[i] = span_of((int64_t)(i * TPR + t) * 8, p.cols);
    xg[i] = load8<TX>(x, at[i]);
    rg[i] = typename Group<TX>::type{};
    if (r) rg[i] = load8<TX>(r, at[i]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) w[i] = load_weight8<TX>(p.w, p.w_f32, at[i]);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    h[i] = value8(xg[i]);
    if (r) h[i] += value8(rg[i]);
    bury(at[i], h[i]);
    bury(at[i], w[i]);
  }
  float ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) ss[0] = __builtin_fmaf(h[i][k], h[i][k], ss[0]);
  }
  if (p.h) {
    char* ho = (char*)p.h + row * p.ldh * XS;
#pragma unroll
    for (int i = 0; i < NV; ++i) store8<TX>(ho, at[i], h[i]);
  }
  row_join<Sum, TPR>(ss, red);
  const float s = 1.0f / __builtin_sqrtf(ss[0] / (float)p.cols + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) h[i] *= w[i];
  if constexpr (Q) {
    // the largest |h w| as an integer: the order of non-negative floats, NaN on top
    uint32_t m[1] = {0u};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) m[0] = Max::join(m[0], __float_as_uint(h[i][k]) & 0x7fffffffu);
    row_join<Max, TPR>(m, redm);
    constexpr float QMAX = TY == T_E4M3 ? 448.0f : 127.0f;
    float scale = __uint_as_float(m[0]) * s / QMAX;
    scale = scale < 0x1p-126f ? 0x1p-126f : scale;  // (a NaN stays)
    const float inv = 1.0f / scale;
    float f = s * inv;
    if (f > 0x1.fffffep127f) {  // the smallest scales: in two steps (all-zero rows give 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) h[i] *= s;
      f = inv;
    }
    uint8_t* y = (uint8_t*)p.y + row * p.ldy;
    if (TY == T_I8 && !(scale <= 0x1.fffffep127f)) {
      // finite values over an infinite scale are 0, and what is NaN becomes 0 (the
      // low byte of a NaN may be anything)
#pragma unroll
      for (int i = 0; i < NV; ++i) store8_q<TY>(y, at[i], v8f{});
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) store8_q<TY>(y, at[i], h[i] * f);
    }
    if (t == 0) p.scale[row] = scale;
  } else {
    char* y = (char*)p.y + row * p.ldy * XS;
#pragma unroll
    for (int i = 0; i < NV; ++i) store8<TX>(y, at[i], h[i] * s);
  }
}

// The backward: a workgroup walks rows blockIdx, blockIdx + grid, ... (RPB at
// a time), keeps its weights and its part of dweight in registers, and leaves
// one partial sum per column; colsum adds the workgroups in a fixed order.  The
// next row is loaded before the sums of this one are joined (loaded at the row's
// start, 8192 x 4096 bf16 takes 44.2 us instead of 42.5, with dh_in 56.9 instead of
// 54.8, 4096 x 8448 54.1 instead of 48.6).  1024 threads have 128 registers each:
// their weights stay in LDS, and an fp32 dh_in is loaded with its own row; fp32 still
// spills 10 registers there (4096 x 9001 fp32: 109 us).
template <int T, int TPR, int NV>
__global__ __launch_bounds__(block_threads<TPR>()) void rmsnorm_grad_kernel(NormGradParams p) {
  constexpr int RPB = block_threads<TPR>() / TPR;
  constexpr int XS = sizeof(typename Elem<T>::type);
  constexpr bool W_LDS = TPR == 1024;
  constexpr bool D_AHEAD = !(W_LDS && T == T_F32);
  __shared__ float red[2][2 * (TPR / 64)];
  __shared__ float joined[RPB > 1 ? RPB * TPR * NV * 8 : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  __shared__ v8f wl[W_LDS ? NV * TPR : 1];
  v8f wr[W_LDS ? 1 : NV], dw[NV];
  Span at[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    at[i] = span_of((int64_t)(i * TPR + t) * 8, p.cols);
    v8f v = load_weight8<T>(p.w, p.w_f32, at[i]);
    bury(at[i], v);
    if constexpr (W_LDS) wl[i * TPR + t] = v;  // read by this thread alone
    else wr[i] = v;
    dw[i] = v8f{};
  }
  auto weight = [&](int i) {
    if constexpr (W_LDS) return wl[i * TPR + t];
    else return wr[i];
  };
  const float inv_cols = 1.0f / (float)p.cols;
  typedef typename Group<T>::type group;
  group h1[NV], g1[NV], d1[NV];
  auto fetch_in = [&](int64_t row, group (&d)[NV]) {
    const char* ip = p.dh_in ? (const char*)p.dh_in + row * p.ldi * XS : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      d[i] = group{};
      if (ip) d[i] = load8<T>(ip, at[i]);
    }
  };
  auto fetch = [&](int64_t row) {
    const char* hp = (const char*)p.h + row * p.ldh * XS;
    const char* gp = (const char*)p.dy + row * p.ldy * XS;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      h1[i] = load8<T>(hp, at[i]);
      g1[i] = load8<T>(gp, at[i]);
    }
    if constexpr (D_AHEAD) fetch_in(row, d1);
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + sub;
  if (row < p.rows) fetch(row);
  int flip = 0;
  for (; row < p.rows; row += step) {
    group hr[NV], gr[NV], dr[NV];
    float sums[2] = {0.0f, 0.0f};  // h^2, g w h
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      hr[i] = h1[i], gr[i] = g1[i];
      if constexpr (D_AHEAD) dr[i] = d1[i];
      bury(at[i], hr[i]);
      bury(at[i], gr[i]);
    }
    // (dH may be an input itself: only rows not yet written are read)
    if constexpr (!D_AHEAD) fetch_in(row, dr);
    if (row + step < p.rows) fetch(row + step);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const v8f h = value8(hr[i]), g = value8(gr[i]), w = weight(i);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sums[0] = __builtin_fmaf(h[k], h[k], sums[0]);
        sums[1] = __builtin_fmaf(g[k] * w[k], h[k], sums[1]);
      }
    }
    row_join<Sum, TPR>(sums, red[flip]);
    flip ^= 1;  // the next row's words are others: one barrier separates reuse
    // dh = dh_in + s (g w - h f), f = s^2 mean(g w h).  (s^3 itself leaves fp32's
    // range for rows of 1e13 or 1e-13, whose dh is of ordinary size.)
    const float s = 1.0f / __builtin_sqrtf(sums[0] * inv_cols + p.eps);
    const float f = s * (s * (sums[1] * inv_cols));
    char* op = (char*)p.dh + row * p.ldo * XS;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const v8f h = value8(hr[i]), g = value8(gr[i]), w = weight(i);
      v8f d = value8(dr[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dw[i][k] = __builtin_fmaf(g[k] * s, h[k], dw[i][k]);
        d[k] = __builtin_fmaf(s, __builtin_fmaf(-h[k], f, g[k] * w[k]), d[k]);
      }
      store8<T>(op, at[i], d);
    }
  }
  if (!p.partial) return;
  float* out = p.partial + (int64_t)blockIdx.x * p.cols;
  if constexpr (RPB > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k >= at[i].dead && k < at[i].live) joined[sub * NV * TPR * 8 + (int)at[i].at + k] = dw[i][k];
    __syncthreads();
    for (int c = threadIdx.x; c < p.cols; c += block_threads<TPR>()) {
      float v = joined[c];
#pragma unroll
      for (int u = 1; u < RPB; ++u) v += joined[u * NV * TPR * 8 + c];
      out[c] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) store8<T_F32>(out, at[i], dw[i]);
  }
}

template <int TX, int TY, int TPR, int NV>
void norm(const NormParams& p, hipStream_t s) {
  constexpr int RPB = block_threads<TPR>() / TPR;
  // (a launch has less than 2^32 threads in each direction)
  const int64_t blocks = (p.rows + RPB - 1) / RPB, x = blocks < 1 << 20 ? blocks : 1 << 20;
  hipLaunchKernelGGL((rmsnorm_kernel<TX, TY, TPR, NV>), dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)),
                     dim3(block_threads<TPR>()), 0, s, p);
}

template <int TX, int TY>
void norm_cols(const NormParams& p, hipStream_t s) {
  if (p.cols <= 512) norm<TX, TY, 64, 1>(p, s);
  else if (p.cols <= 1024) norm<TX, TY, 64, 2>(p, s);
  else if (p.cols <= 2048) norm<TX, TY, 256, 1>(p, s);
  else if (p.cols <= 4096) norm<TX, TY, 256, 2>(p, s);
  else if (p.cols <= 8192) norm<TX, TY, 256, 4>(p, s);
  else norm<TX, TY, 1024, 2>(p, s);
}

template <int TX>
void norm_y(int y_dtype, const NormParams& p, hipStream_t s) {
  if (y_dtype == T_E4M3) norm_cols<TX, T_E4M3>(p, s);
  else if (y_dtype == T_I8) norm_cols<TX, T_I8>(p, s);
  else norm_cols<TX, TX>(p, s);
}

template <int T, int TPR, int NV>
void grad(const NormGradParams& p, int grid, hipStream_t s) {
  hipLaunchKernelGGL((rmsnorm_grad_kernel<T, TPR, NV>), dim3(grid), dim3(block_threads<TPR>()), 0, s, p);
}

// As few idle threads as the row allows (4096 x 6144 bf16: 38.9 us with 384
// threads, 41.6 with 512; 4096 x 8448: 51.6 with 768, 57.0 with 1024).  fp32 does
// not fit the registers of 768 threads with its weights (193 us, 135 with 1024
// and the weights in LDS).
template <int T>
void grad_cols(const NormGradParams& p, int grid, hipStream_t s) {
  if (p.cols <= 512) grad<T, 64, 1>(p, grid, s);
  else if (p.cols <= 1024) grad<T, 64, 2>(p, grid, s);
  else if (p.cols <= 2048) grad<T, 256, 1>(p, grid, s);
  else if (p.cols <= 4096) grad<T, 256, 2>(p, grid, s);
  else if (p.cols <= 6144) grad<T, 384, 2>(p, grid, s);
  else if (p.cols <= 8192) grad<T, 512, 2>(p, grid, s);
  else if (T == T_F32 || p.cols > 12288) grad<T, 1024, 2>(p, grid, s);
  else if constexpr (T != T_F32) grad<T, 768, 2>(p, grid, s);
}

}  // namespace

void launch_rmsnorm(int x_dtype, int y_dtype, const NormParams& p, hipStream_t s) {
  if (x_dtype == T_F16) norm_y<T_F16>(y_dtype, p, s);
  else if (x_dtype == T_BF16) norm_y<T_BF16>(y_dtype, p, s);
  else norm_y<T_F32>(y_dtype, p, s);
}

int rmsnorm_grad_grid(int64_t rows, int64_t cols, int cus) {
  const int64_t groups = cols <= 1024 ? (rows + 3) / 4 : rows;
  // a few rows: one workgroup walks them, and its sums are the result (2 us a
  // row against a second launch of 5)
  if (groups <= 2) return 1;
  // workgroups that a compute unit holds: short rows need more of them in flight
  const int64_t most = (int64_t)cus * (cols > 8192 ? 1 : cols > 2048 ? 2 : 4);
  return (int)(groups < most ? groups : most);
}

void launch_rmsnorm_grad(int x_dtype, const NormGradParams& p, int grid, hipStream_t s) {
  if (x_dtype == T_F16) grad_cols<T_F16>(p, grid, s);
  else if (x_dtype == T_BF16) grad_cols<T_BF16>(p, grid, s);
  else grad_cols<T_F32>(p, grid, s);
}

}  // namespace gemm_epi
