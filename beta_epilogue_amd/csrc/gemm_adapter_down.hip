// gemm_adapter_down.hip -- the rows' inner products with their own adapters:
//   U[m][j] = scale[g] sum_k A[m][k] down[g][j][k],  g = ids[m].
//
// Few rows (kAdapterDots): a wave takes one product of one row, so rows of
// as many adapters cost the same, and every weight is read once per row that has
// it, from the cache but for the first time.
//
// More rows are sorted by adapter (gemm_experts_kernels.hip), so that a workgroup
// has 16 rows of one, streamed past the adapter's weights by the few-row kernel
// (gemm_linear_rows.hip): 4001 x 4096, rank 64, 16 us (17 to 19 with eight waves,
// whose LDS leaves room for one workgroup only, so that the ones below came in a round
// of their own; 24 with fragments straight from memory).  What bounds it is each adapter's
// weights, once from the cache for every 16 rows.  With up to two adapters the rows stay
// as they are, and a workgroup takes one after the other: a launch less.  (With four,
// all mixed, 1000 x 1024, rank 32, that is 14.4 us against 3.1 and 6.3.)
//
// Further workgroups of the same launch look whether the up[g] that the rows meet
// are finite (AdapterTiles): a read of each beside the rows' (4001 x 4096 x 4096: 7 adapters
// of rank 64 nothing, 300 of them, 157 MB, 15 of 219 us; 512 x 2048 x 2048, 200 of them, 6
// of 50).
#include "gemm_adapter.hpp"
#include "gemm_linear_rows.hpp"

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

// Whether any thread of the workgroup says so; red: a word per wave.
__device__ __forceinline__ bool any_thread(bool v, int* red) {
  const bool any = __any(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = any;
  __syncthreads();
  bool all = false;
  for (int w = 0; w < (int)blockDim.x / 64; ++w) all |= red[w] != 0;
  return all;
}

// Whether part `block % kFiniteParts` of up[block / kFiniteParts] is finite; an
// adapter that no row has is not read (and nobody asks), unless it takes a pass over
// many rows to know.
template <int AB>
__device__ __forceinline__ void finite_block(const AdapterDownParams& p, int block, int* red) {
  const int g = block / kFiniteParts, part = block % kFiniteParts, threads = blockDim.x;
  bool met = true;
  if (p.offsets) {
    met = p.offsets[g + 1] > p.offsets[g];
  } else if (p.M * p.rank <= kAdapterDots) {
    met = false;
    for (int64_t m = threadIdx.x; m < p.M; m += threads) met |= p.ids[m] == g;
    met = any_thread(met, red);
  }
  if (!met) return;
  constexpr uint32_t kExp = AB == T_F16 ? 0x7c00u : 0x7f80u;
  const int64_t n = p.N * p.rank / 8;  // 16-byte pieces
  const v4u* w = (const v4u*)((const char*)p.up + g * n * 16);
  bool bad = false;
#pragma unroll 8
  for (int64_t i = part * (int64_t)threads + threadIdx.x; i < n; i += (int64_t)kFiniteParts * threads) {
    const v4u v = w[i];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      bad |= (v[k] & kExp) == kExp || (v[k] & (kExp << 16)) == kExp << 16;
  }
  bad = any_thread(bad, red);
  if (threadIdx.x == 0) p.finite[g * kFiniteParts + part] = bad ? 0 : 1;
}

// Products 4 x .. 4 x + 3 of a row, one wave each.
template <int AB>
__global__ __launch_bounds__(256) void adapter_dots_kernel(AdapterDownParams p, int blocks) {
  __shared__ int red[4];
  if ((int)blockIdx.x >= blocks) {
    finite_block<AB>(p, blockIdx.x - blocks, red);
    return;
  }
  const int per = p.rank / 4, m = blockIdx.x / per;
  const int g = p.ids[m];
  if (g < 0 || g >= p.adapters) return;
  const int lane = threadIdx.x & 63, j = (blockIdx.x - m * per) * 4 + (threadIdx.x >> 6);
  const uint16_t* a = (const uint16_t*)p.A + m * p.lda;
  const uint16_t* w = (const uint16_t*)p.down + ((int64_t)g * p.rank + j) * p.K;
  float s = 0.0f;
#pragma unroll 8
  for (int64_t k = lane * 8; k < p.K; k += 512) s = dot8<AB>(*(const v4u*)(a + k), *(const v4u*)(w + k), s);
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d);
  if (lane == 0) store_as(p.U, (int64_t)m * p.rank + j, AB, s * p.scale[g]);
}

// 16 rows, 64 of their products (4 * MB at most): the few-row kernel with the rows in
// the weight's place and the adapter's in the tokens'.  Sorted rows have one adapter,
// others are taken one adapter at a time.
template <int AB, int MB, int NW, int NS>
__global__ __launch_bounds__(NW * 64) void adapter_down_kernel(AdapterDownParams p, int blocks, int per) {
  __shared__ __attribute__((aligned(1024))) char lds[RowsLds<AB, MB, NW, NS>::BYTES];
  if ((int)blockIdx.x >= blocks * per) {
    finite_block<AB>(p, blockIdx.x - blocks * per, (int*)lds);
    return;
  }
  const int chunk = blockIdx.x / per, j0 = (blockIdx.x - chunk * per) * 64;
  const int lane = threadIdx.x & 63;
  int mine = -1, id = -1;  // lane i (and 16 + i, ...): the chunk's row i and its adapter
  int first = chunk * 16, end = (int)p.M;
  if (p.order) {
    GroupParams gp;
    gp.offsets = p.offsets;
    gp.groups = p.adapters;
    gp.rows = (int)p.M;
    const GroupTile t = group_chunk(gp, chunk, 16);
    if (t.group < 0) return;
    first = t.begin;
    end = t.end;
    if (first + (lane & 15) < end) mine = p.order[first + (lane & 15)], id = t.group;
  } else if (first + (lane & 15) < end) {
    mine = first + (lane & 15);
    id = p.ids[mine];
    if (id < 0 || id >= p.adapters) id = -1;
  }
  // one adapter of the chunk's rows after the other
  for (uint64_t todo = __ballot(id >= 0); todo;) {
    const int g = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)todo) - 1);
    todo &= ~__ballot(id == g);
    const int row = id == g ? mine : -1;
    LinParams q;
    q.A = (const char*)p.down + ((int64_t)g * p.rank + j0) * p.K * 2;
    q.M = min(p.rank - j0, 64);
    q.K = q.lda = p.K;
    const float f = p.scale[g];
    rows_products<AB, MB, NW, NS>(
        q, make_rsrc(p.A, (uint32_t)(((p.M - 1) * p.lda + p.K) * 2)),
        [&](int i) {
          const int m = __shfl(row, i);
          return m >= 0 ? (uint32_t)(m * p.lda * 2) : 0x80000000u;
        },
        lds, [](int, int) {}, [](auto&) {},
        [&](int j, int i, v4f sum) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = first + i + e;
            if (at >= end || (!p.order && p.ids[at] != g)) continue;
            const int64_t m = p.order ? p.order[at] : at;
            store_as(p.U, m * p.rank + j0 + j, AB, sum[e] * f);
          }
        });
    __syncthreads();  // the sums' join is read: the ring may be filled again
  }
}

// Workgroups that look at up.
int looks(const AdapterDownParams& p) { return p.finite ? p.adapters * kFiniteParts : 0; }

template <int AB, int MB, int NW, int NS>
void down(const AdapterDownParams& p, hipStream_t s) {
  // chunks; sorted: of the worst distribution
  const int64_t n = p.M < p.adapters ? p.M : p.adapters;
  const int blocks = (int)(p.order ? n + (p.M - n) / 16 : (p.M + 15) / 16), per = (p.rank + 63) / 64;
  hipLaunchKernelGGL((adapter_down_kernel<AB, MB, NW, NS>), dim3((unsigned)(blocks * per + looks(p))), dim3(NW * 64), 0, s, p,
                     blocks, per);
}

template <int AB>
void launch(const AdapterDownParams& p, hipStream_t s) {
  if (p.M * p.rank <= kAdapterDots) {
    const int blocks = (int)(p.M * p.rank / 4);
    hipLaunchKernelGGL(adapter_dots_kernel<AB>, dim3((unsigned)(blocks + looks(p))), dim3(256), 0, s, p, blocks);
    return;
  }
  if (p.order) {
    SortParams q = {};
    q.ids = p.ids;
    q.offsets = p.offsets;
    q.order = p.order;
    q.counts = p.counts;
    q.tokens = p.M;
    q.top_k = 1;
    q.experts = p.adapters;
    q.chunks = (int32_t)sort_chunks(p.M);
    launch_expert_sort(q, s);
  }
  if (p.rank <= 16) down<AB, 4, 4, 2>(p, s);
  else if (p.rank <= 32) down<AB, 8, 4, 1>(p, s);
  else down<AB, 16, 4, 1>(p, s);
}

}  // namespace

void launch_adapter_down(int ab, const AdapterDownParams& p, hipStream_t s) {
  if (ab == T_F16) launch<T_F16>(p, s);
  else launch<T_BF16>(p, s);
}

}  // namespace gemm_epi
