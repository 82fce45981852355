// gemm_adapter_down.hip -- the rows' inner products with their own adapters:
//   U[m][j] = scale[g] sum_k A[m][k] down[g][j][k],  g = ids[m].
//
// Few rows (M * rank up to 8192): a wave takes one product of one row, so rows of
// as many adapters cost the same, and every weight is read once per row that has
// it, from the cache but for the first time.
//
// More rows: 16 or 32 rows per workgroup, K split over its 8 waves, whose partial
// sums are joined through LDS in wave order; fragments come straight from memory,
// 128 bytes of a row in one load of 4 lanes.  Bound by the one read of A.  Rows of
// several adapters take one pass over K for each, and keep only their own.
#include "gemm_adapter.hpp"

namespace gemm_epi {

namespace {

template <int AB>
__device__ __forceinline__ float dot8(v4u a, v4u b, float s) {
  const v4f a0 = epi_dec<AB>(a, 0), a1 = epi_dec<AB>(a, 1), b0 = epi_dec<AB>(b, 0), b1 = epi_dec<AB>(b, 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __builtin_fmaf(a0[i], b0[i], s);
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __builtin_fmaf(a1[i], b1[i], s);
  return s;
}

// Workgroup (x, y): products 4 x .. 4 x + 3 of row y, one wave each.
template <int AB>
__global__ __launch_bounds__(256) void adapter_dots_kernel(AdapterDownParams p) {
  const int64_t m = blockIdx.y;
  const int g = p.ids[m];
  if (g < 0 || g >= p.adapters) return;
  const int lane = threadIdx.x & 63, j = blockIdx.x * 4 + (threadIdx.x >> 6);
  const uint16_t* a = (const uint16_t*)p.A + m * p.lda;
  const uint16_t* w = (const uint16_t*)p.down + ((int64_t)g * p.rank + j) * p.K;
  float s = 0.0f;
#pragma unroll 8
  for (int64_t k = lane * 8; k < p.K; k += 512) s = dot8<AB>(*(const v4u*)(a + k), *(const v4u*)(w + k), s);
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d);
  if (lane == 0) store_as(p.U, m * p.rank + j, AB, s * p.scale[g]);
}

// RB blocks of 16 rows, up to CB * 16 products of each.
template <int AB, int RB, int CB>
__global__ __launch_bounds__(512) void adapter_down_kernel(AdapterDownParams p) {
  using MM = Mma<AB, 16>;
  constexpr int NW = 8, ROWS = RB * 16;
  __shared__ v4f part[NW][RB * CB][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * ROWS;
  const int rows = (int)min(p.M - m0, (int64_t)ROWS);
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((const char*)p.A + m0 * p.lda * 2), (short)0, (int)(((rows - 1) * p.lda + p.K) * 2), 0x00020000);
  int id[RB];
  uint32_t oa[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int m = i * 16 + r;
    const int g = m < rows ? p.ids[m0 + m] : -1;
    id[i] = g >= 0 && g < p.adapters ? g : -1;
    oa[i] = m < rows ? (uint32_t)((m * p.lda + q * 16) * 2) : 0x80000000u;
  }
  uint32_t todo[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) todo[i] = (uint32_t)__ballot(id[i] >= 0) & 0xffffu;
  for (;;) {
    int g = -1;
    static_for<0, RB>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      if (g < 0 && todo[i]) g = __builtin_amdgcn_readlane(id[i], __ffs(todo[i]) - 1);
    });
    if (g < 0) break;
    const int64_t bytes = p.rank * p.K * 2;
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        (void*)((const char*)p.down + g * bytes), (short)0, (int)bytes, 0x00020000);
    v4f acc[RB][CB] = {};
#pragma unroll 2
    for (int64_t k = wave * 64; k < p.K; k += NW * 64) {
      // lane (q, r): k + 16 q .. + 15 of its rows; each half is one product
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = k + q * 16 + h * 8 < p.K;
        const uint32_t at = (uint32_t)(k + h * 8) * 2;
        v4i fa[RB], fb[CB];
#pragma unroll
        for (int i = 0; i < RB; ++i)
          fa[i] = adapter_load(ra, in && oa[i] != 0x80000000u ? oa[i] + at : 0x80000000u);
#pragma unroll
        for (int c = 0; c < CB; ++c)
          fb[c] = adapter_load(rb, in && c * 16 + r < p.rank ? (uint32_t)(((c * 16 + r) * p.K + q * 16) * 2) + at
                                                             : 0x80000000u);
        // (products are the matrix core's rows: a lane ends with four of a token)
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
          for (int c = 0; c < CB; ++c) acc[i][c] = MM::mma(fb[c], fa[i], acc[i][c]);
      }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int c = 0; c < CB; ++c) part[wave][i * CB + c][lane] = acc[i][c];
    __syncthreads();
    for (int b = wave; b < RB * CB; b += NW) {
      v4f s = part[0][b][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) s += part[w][b][lane];
      const int m = (b / CB) * 16 + r, j = (b % CB) * 16 + 4 * q;
      int mine = -1;
      static_for<0, RB>([&](auto i_c) {
        if (b / CB == decltype(i_c)::value) mine = id[decltype(i_c)::value];
      });
      if (mine != g || j >= p.rank) continue;
      const float f = p.scale[g];
      uint16_t* out = (uint16_t*)p.U + (m0 + m) * p.rank + j;
#pragma unroll
      for (int e = 0; e < 4; ++e) store_as(out, e, AB, s[e] * f);
    }
    __syncthreads();
    static_for<0, RB>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      todo[i] &= ~((uint32_t)__ballot(id[i] == g) & 0xffffu);
    });
  }
}

template <int AB, int RB, int CB>
void down(const AdapterDownParams& p, hipStream_t s) {
  hipLaunchKernelGGL((adapter_down_kernel<AB, RB, CB>), dim3((unsigned)((p.M + RB * 16 - 1) / (RB * 16))), dim3(512), 0, s,
                     p);
}

template <int AB>
void launch(const AdapterDownParams& p, hipStream_t s) {
  if (p.M * p.rank <= 8192)
    hipLaunchKernelGGL(adapter_dots_kernel<AB>, dim3((unsigned)(p.rank / 4), (unsigned)p.M), dim3(256), 0, s, p);
  else if (p.rank <= 16) down<AB, 2, 1>(p, s);
  else if (p.rank <= 32) down<AB, 2, 2>(p, s);
  else if (p.rank <= 64) down<AB, 2, 4>(p, s);
  else down<AB, 1, 8>(p, s);
}

}  // namespace

void launch_adapter_down(int ab, const AdapterDownParams& p, hipStream_t s) {
  if (ab == T_F16) launch<T_F16>(p, s);
  else launch<T_BF16>(p, s);
}

}  // namespace gemm_epi
