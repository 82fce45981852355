// gemm_grouped_part.hip -- compiles the tile kernels of
// gemm_grouped_variants.inc whose `part` equals GEMM_GROUPED_PART (the build
// compiles this file once per part, in parallel).
//
// The linear layer's main loop and epilogue (gemm_epi_kernel.hpp) with each tile's rows
// ending at its expert's end.  Bound by the MFMAs where experts have hundreds of rows:
// 16384 rows of 8 experts, bf16, N 4096, K 2048, silu, U and Z, 309 us (890 TFLOP/s;
// the epilogue is 13 of a tile's 55 us, with nothing to hide behind), and by the weights'
// bytes below that: 2048 rows of 64 experts, e4m3, 1536 x 2048, 48 us (4.3 TB/s) in
// 64x64 tiles.
#include "gemm_grouped.hpp"

#ifndef GEMM_GROUPED_PART
#error "GEMM_GROUPED_PART must be defined (0 .. 6)"
#endif

namespace gemm_epi {

namespace {
// Persistent workgroups, an equal share of the tiles each.  Only the device knows
// how many tiles there are, and a last round of 256x256 tiles that leaves half of
// the compute units or more idle runs as quarters on the 128x128 kernel: a
// quarter takes under half of a tile's time.  (Quarters first in every other
// workgroup, so that not all of them write at the same time, changed nothing.)
template <class CF>
__global__ __launch_bounds__(CF::THREADS, CF::OCC) void grouped_kernel(GroupParams p) {
  __shared__ __attribute__((aligned(1024))) char lds[CF::LDS_BYTES + kGroupTableBytes];
  int* first = (int*)(lds + CF::LDS_BYTES);
  const int G = gridDim.x, total = group_table_rows(p, first, CF::BM) * p.tiles_n;
  if constexpr (CF::BM == 256) {
    const int left = total % G, whole = left <= G / 2 ? total - left : total;
    using Q = GroupedQuarter<CF::AB>;
    static_assert(Q::LDS_BYTES <= CF::LDS_BYTES && Q::THREADS == CF::THREADS, "one workgroup for both");
    gemm_epi_body<CF>(p, lds, blockIdx.x, G, GroupWork{first, 0, whole, 0});
    gemm_epi_body<Q>(p, lds, blockIdx.x, G, GroupWork{first, 4 * whole, 4 * total, 1});
  } else {
    gemm_epi_body<CF>(p, lds, blockIdx.x, G, GroupWork{first, 0, total, 0});
  }
}

template <int PART, class CF>
void launch_if(bool wanted, const GroupParams& p, int grid, hipStream_t s) {
  if constexpr (PART == GEMM_GROUPED_PART) {
    if (wanted) hipLaunchKernelGGL(grouped_kernel<CF>, dim3(grid), dim3(CF::THREADS), 0, s, p);
  }
}
}  // namespace

template <>
void launch_grouped_part<GEMM_GROUPED_PART>(int variant, const GroupParams& p, int grid, hipStream_t s) {
  int i = 0;
#define X(PART, AB, BM, BN, S, OCC, BL, NAME) launch_if<PART, GroupedCfg<AB, BM, BN, S, OCC, BL>>(variant == i++, p, grid, s);
#include "gemm_grouped_variants.inc"
#undef X
}

}  // namespace gemm_epi
