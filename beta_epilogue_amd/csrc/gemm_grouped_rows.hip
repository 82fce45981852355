// gemm_grouped_rows.hip -- the experts' linear layer with few rows per expert
// (decoding): the few-row kernel (gemm_linear_rows.hip) on chunks of an expert's
// rows.  The time is the weights' of the experts that have rows; a workgroup
// streams 16 weight rows of one of them past a chunk of up to 4 * MB of its rows
// (8 rows of 8 experts, bf16, 512 x 4096: 8.7 us, in 64x64 tiles 15.6; 1536 x 2048: 14.3
// and 15.0).
#include "gemm_grouped.hpp"
#include "gemm_linear_rows.hpp"

namespace gemm_epi {

namespace {

template <int AB, int MB, int NW, int NS>
__global__ __launch_bounds__(NW * 64) void grouped_rows_kernel(GroupParams p) {
  constexpr int ES = AB == T_F16 || AB == T_BF16 ? 2 : 1;
  __shared__ __attribute__((aligned(1024))) char lds[RowsLds<AB, MB, NW, NS>::BYTES];
  const GroupTile t = group_chunk(p, blockIdx.y, 4 * MB);
  if (t.group < 0) return;
  LinParams q = p;
  const int64_t r = t.begin, g = t.group;
  const int sh = epi_shift(p.d_dtype);
  q.M = t.end - t.begin;
  q.A = (const char*)p.A + r * p.lda * ES;
  q.B = (const char*)p.B + g * p.N * p.K * ES;
  q.D = (char*)p.D + (r * p.ldd << sh);
  if (p.R) q.R = (const char*)p.R + (r * p.ldr << sh);
  if (p.Z) q.Z = (char*)p.Z + (r * p.ldz << sh);
  if (p.bias) q.bias = (const char*)p.bias + (g * p.N << epi_shift(p.bias_dtype));
  if (p.scale_a) q.scale_a = p.scale_a + r;
  if (p.scale_b) q.scale_b = p.scale_b + g * p.N;
  linear_rows_body<AB, MB, NW, NS, true>(q, (int64_t)blockIdx.x * 16, lds, [](auto&) {});
}

template <int AB, int MB, int NW, int NS>
void rows(const GroupParams& p, int slots, hipStream_t s) {
  hipLaunchKernelGGL((grouped_rows_kernel<AB, MB, NW, NS>), dim3((unsigned)((p.N + 15) / 16), (unsigned)slots),
                     dim3(NW * 64), 0, s, p);
}

template <int AB>
void rows_ab(int mb, const GroupParams& p, int slots, hipStream_t s) {
  if (mb == 1) rows<AB, 1, 8, 2>(p, slots, s);
  else rows<AB, 4, 4, 2>(p, slots, s);
}

}  // namespace

void launch_grouped_rows(int ab, int mb, const GroupParams& p, int slots, hipStream_t s) {
  if (ab == T_F16) rows_ab<T_F16>(mb, p, slots, s);
  else if (ab == T_BF16) rows_ab<T_BF16>(mb, p, slots, s);
  else if (ab == T_E4M3) rows_ab<T_E4M3>(mb, p, slots, s);
  else rows_ab<T_I8>(mb, p, slots, s);
}

}  // namespace gemm_epi
