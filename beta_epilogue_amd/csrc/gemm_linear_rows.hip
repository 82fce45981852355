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
#include "gemm_linear_rows.hpp"

namespace gemm_epi {

namespace {

template <int AB, int MB, int NW, int NS>
__global__ __launch_bounds__(NW * 64) void linear_rows_kernel(LinParams p) {
  __shared__ __attribute__((aligned(1024))) char lds[RowsLds<AB, MB, NW, NS>::BYTES];
  linear_rows_body<AB, MB, NW, NS, false>(p, (int64_t)blockIdx.x * 16, lds, [](auto&) {});
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
    Epi4<> epi;
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
