// gemm_adapter_rows.hip -- the few-row kernel (gemm_linear_rows.hip) with
// adapters: up to 64 tokens, each with one of its own.  While a wave's first runs
// of the weight are on their way it adds its share of the tokens' adapters to its
// sums: 16 rows of up[g] against the tokens of g, the other tokens' columns zero.
// 16 tokens of 12 adapters of rank 16, 4096 x 4096 bf16: 10.6 us (the linear layer's 8.0),
// behind 4.8 for the inner products.
#include "gemm_adapter.hpp"
#include "gemm_linear_rows.hpp"

namespace gemm_epi {

namespace {

template <int AB, int MB, int NW, int NS>
__global__ __launch_bounds__(NW * 64) void adapter_rows_kernel(AdapterParams p) {
  constexpr int NB = (MB + 3) / 4;
  using MM = RowsMma<AB>;
  __shared__ __attribute__((aligned(1024))) char lds[RowsLds<AB, MB, NW, NS>::BYTES];
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  linear_rows_body<AB, MB, NW, NS, false>(p, n0, lds, [&](auto& acc) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int token = row_adapter(p, lane);  // lane's token's, M <= 64
    int id[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) id[j] = __shfl(token, j * 16 + r);
    const __amdgpu_buffer_rsrc_t ru =
        __builtin_amdgcn_make_buffer_rsrc((void*)p.U, (short)0, (int)p.M * p.rank * 2, 0x00020000);
    const uint32_t row = (uint32_t)p.rank * 2, ub = (uint32_t)r * row + 16 * q, nb = (uint32_t)(n0 + r) * row + 16 * q;
    int turn = 0;  // (adapter, 32 of the rank) pairs go round the waves
    for (uint64_t todo = __ballot(token >= 0); todo;) {
      const int g = __builtin_amdgcn_readlane(token, __ffsll((unsigned long long)todo) - 1);
      todo &= ~__ballot(token == g);
      const __amdgpu_buffer_rsrc_t rp = adapter_up(p, g);
      for (int k = 0; k < p.rank; k += 32) {
        if (turn++ % NW != wave) continue;
        const bool in = k + 8 * q < p.rank;
        const v4i b = adapter_load(rp, in ? nb + 2 * k : 0x80000000u);
        v4i a[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) a[j] = adapter_load(ru, in && id[j] == g ? ub + j * 16 * row + 2 * k : 0x80000000u);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const typename MM::acc_t t = MM::mma(__builtin_bit_cast(v4u, b), __builtin_bit_cast(v4u, a[j]), typename MM::acc_t{});
          // (a NaN of up[g] times another token's zero is not added)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[j][v] += id[j] == g ? t[v] : 0.0f;
        }
      }
    }
  });
}

template <int AB, int MB, int NW, int NS>
void rows(const AdapterParams& p, hipStream_t s) {
  hipLaunchKernelGGL((adapter_rows_kernel<AB, MB, NW, NS>), dim3((unsigned)((p.N + 15) / 16)), dim3(NW * 64), 0, s, p);
}

template <int AB>
void rows_ab(int nw, const AdapterParams& p, hipStream_t s) {
  if (p.M <= 4) rows<AB, 1, 8, 2>(p, s);
  else if (p.M <= 8) rows<AB, 2, 8, 2>(p, s);
  else if (p.M <= 16) nw == 8 ? rows<AB, 4, 8, 2>(p, s) : rows<AB, 4, 4, 2>(p, s);
  else if (p.M <= 32) nw == 8 ? rows<AB, 8, 8, 1>(p, s) : rows<AB, 8, 4, 1>(p, s);
  else nw == 8 ? rows<AB, 16, 8, 1>(p, s) : rows<AB, 16, 4, 1>(p, s);
}

}  // namespace

void launch_adapter_rows(int ab, int nw, const AdapterParams& p, hipStream_t s) {
  if (ab == T_F16) rows_ab<T_F16>(nw, p, s);
  else rows_ab<T_BF16>(nw, p, s);
}

}  // namespace gemm_epi
