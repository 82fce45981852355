// gemm_experts_kernels.hip -- tokens sorted by expert, their results brought
// back with the router's weights, and the gradient of that.
//
// The sort is a stable counting sort of the T * top_k choices: row = offsets[e]
// + the number of earlier choices of e.  Counts and ranks come from ballots (LDS
// atomics of choices that are alike queue up: 4001 choices of 5 runs took 8.7 us
// with one per choice, 6.1 now).  One workgroup ranks up to 8192 choices (4 to 10 us);
// of more, every workgroup counts a chunk of 4096 and a second launch ranks it behind the
// counts of the chunks before it (98760 choices of 128 experts: 5 and 7 us).  Those
// sums read every chunk's counts in every workgroup, which grows with the square of
// the chunks (10^6 choices of 128 experts 23 us, of 1024 29, 10^7 of 128 370 to 470).
// Moving the rows is bound by memory: a token's row is read once and stored top_k times.
#include "gemm_experts.hpp"
#include "gemm_linear.hpp"

namespace gemm_epi {

namespace {

constexpr int kSortThreads = 1024, kSortWaves = 16;

// Choice i's expert; -1: none.
__device__ __forceinline__ int choice(const SortParams& p, int64_t i, int64_t n) {
  if (i >= n) return -1;
  const int64_t e = p.ids64 ? ((const int64_t*)p.ids)[i] : (int64_t)((const int32_t*)p.ids)[i];
  return e >= 0 && e < p.experts ? (int)e : -1;
}

struct SortLds {
  int cnt[kSortWaves][kMaxExperts];  // a wave's choices of an expert, then its next row
  int wave_sum[kSortWaves];
};

// A wave's part of a chunk: `steps` (up to IT) times 64 consecutive choices.
template <int IT>
struct SortPart {
  int64_t first;       // this lane's first choice
  int steps;
  int e[IT];           // experts
  uint64_t same[IT];   // the lanes of the same expert (without one: anything)

  // Reads the choices and counts them.
  __device__ __forceinline__ void count(const SortParams& p, SortLds& s, int chunk) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = p.tokens * p.top_k, c0 = (int64_t)chunk * (IT * 1024);
    steps = (int)((min(n - c0, (int64_t)IT * 1024) + 1023) >> 10);  // few choices: one step of every wave
    first = c0 + wave * (steps * 64) + lane;
#pragma unroll
    for (int k = 0; k < IT; ++k) e[k] = k < steps ? choice(p, first + k * 64, n) : -1;
    for (int x = lane; x < p.experts; x += 64) s.cnt[wave][x] = 0;
    const int bits = 32 - __clz(p.experts);
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      if (k >= steps) break;
      // by one ballot per bit of the expert's number
      same[k] = __ballot(e[k] >= 0);
      for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((e[k] >> b) & 1);
        same[k] &= (e[k] >> b) & 1 ? one : ~one;
      }
      if (e[k] >= 0 && earlier(k) == 0) atomicAdd(&s.cnt[wave][e[k]], __popcll(same[k]));
    }
    __syncthreads();
  }
  // Lanes before this one with the same expert in step k.
  __device__ __forceinline__ int earlier(int k) const {
    return __popcll(same[k] & ((uint64_t(1) << (threadIdx.x & 63)) - 1));
  }
};

template <int IT>
__global__ __launch_bounds__(kSortThreads) void expert_count_kernel(SortParams p) {
  __shared__ SortLds s;
  SortPart<IT> part;
  part.count(p, s, blockIdx.x);
  for (int x = threadIdx.x; x < p.experts; x += kSortThreads) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) n += s.cnt[w][x];
    p.counts[(int64_t)blockIdx.x * p.experts + x] = n;
  }
}

// 16 bytes of a row of X, for the token's choices.
__device__ __forceinline__ void move_piece(const SortParams& p, int64_t t, uint32_t c, const int32_t* rows) {
  const v4u v = __builtin_nontemporal_load((const v4u*)((const char*)p.X + t * p.ldx + (int64_t)c * 16));
  const float sc = p.scale && c == 0 ? p.scale[t] : 0.0f;
#pragma unroll 4
  for (int j = 0; j < p.top_k; ++j) {
    const int r = rows[j];
    if (r < 0) continue;
    __builtin_nontemporal_store(v, (v4u*)((char*)p.Y + r * p.ldy + (int64_t)c * 16));
    if (p.scale && c == 0) p.scale_out[r] = sc;
  }
}

// Ranks the choices of chunk blockIdx.x: rows, the choice of each row, and (the
// first workgroup) offsets.  MOVE (one chunk): every workgroup ranks all choices
// and moves its share of the rows, which saves a launch (16 tokens, 8 of 64
// experts, 2048 columns of bf16: 9.5 us with two).
template <int IT, bool MOVE>
__global__ __launch_bounds__(kSortThreads) void expert_rank_kernel(SortParams p) {
  __shared__ SortLds s;
  __shared__ int32_t mine[MOVE ? IT * 1024 : 1];
  const int block = MOVE ? 0 : blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = threadIdx.x;
  SortPart<IT> part;
  part.count(p, s, block);
  // expert t's choices in all, and in the chunks before this one
  int all = 0, before = 0;
  if (t < p.experts) {
    if (p.chunks == 1) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) all += s.cnt[w][t];
    } else {
#pragma unroll 8
      for (int c = 0; c < p.chunks; ++c) {
        const int n = p.counts[(int64_t)c * p.experts + t];
        all += n;
        before += c < block ? n : 0;
      }
    }
  }
  // an exclusive sum over the experts
  const int sum = wave_scan(all);
  if (lane == 63) s.wave_sum[wave] = sum;
  __syncthreads();
  int first = sum - all;
  for (int w = 0; w < wave; ++w) first += s.wave_sum[w];
  if (t < p.experts) {
    if (blockIdx.x == 0) {
      p.offsets[t] = first;
      if (t == p.experts - 1) p.offsets[t + 1] = first + all;
    }
    int at = first + before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = s.cnt[w][t];
      s.cnt[w][t] = at;
      at += n;
    }
  }
  __syncthreads();
  // a wave's choices in order, 64 at a time: the first lane of each expert takes
  // the rows of its equals
  const int64_t n = p.tokens * p.top_k;
#pragma unroll
  for (int k = 0; k < IT; ++k) {
    if (k >= part.steps) break;
    const int e = part.e[k], earlier = part.earlier(k);
    int at = 0;
    if (e >= 0 && earlier == 0) at = atomicAdd(&s.cnt[wave][e], __popcll(part.same[k]));
    at = __shfl(at, e >= 0 ? __ffsll((unsigned long long)part.same[k]) - 1 : lane) + earlier;
    const int64_t i = part.first + k * 64;
    if (i >= n) continue;
    if constexpr (MOVE) mine[i] = e >= 0 ? at : -1;
    if (MOVE && blockIdx.x != 0) continue;
    if (p.rows) p.rows[i] = e >= 0 ? at : -1;
    if (p.order && e >= 0) p.order[at] = (int32_t)i;
  }
  if constexpr (MOVE) {
    __syncthreads();
    const uint32_t per = (uint32_t)(p.row_bytes / 16);
    const int64_t pieces = p.tokens * per;
    for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * kSortThreads) {
      const int64_t t = i / per;
      move_piece(p, t, (uint32_t)(i - t * per), mine + t * p.top_k);
    }
  }
}

// A thread for every 16 bytes of X: 12345 rows of 4096 bytes to 8 experts each, 455 MB
// in 88 us (5.2 TB/s, a large copy's rate).
__global__ __launch_bounds__(256) void expert_gather_kernel(SortParams p) {
  const uint32_t per = (uint32_t)(p.row_bytes / 16);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / per;
  if (t < p.tokens) move_piece(p, t, (uint32_t)(i - t * per), p.rows + t * p.top_k);
}

// ---------------------------------------------------------------------------
// The way back
// ---------------------------------------------------------------------------
template <int T> struct Vec {
  static constexpr int N = T == T_F32 ? 4 : 8;  // elements of a 16-byte access
  float v[N];
  __device__ __forceinline__ void decode(v4u r) {
    const v4f lo = epi_dec<T>(r, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lo[i];
    if constexpr (N == 8) {
      const v4f hi = epi_dec<T>(r, 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 + i] = hi[i];
    }
  }
  __device__ __forceinline__ v4u pack() const {
    return epi_pack<T>(v4f{v[0], v[1], v[2], v[3]}, N == 8 ? v4f{v[N - 4], v[N - 3], v[N - 2], v[N - 1]} : v4f{});
  }
};

// A thread makes 16 bytes of a token's row, summed in fp32 in the order of the
// token's choices; G choices' rows are in flight at a time.  Bound by memory: 12345
// tokens, 8 rows of 2048 bf16 each, 503 MB in 79 us, some of them from the last-level
// cache.
template <int T>
__global__ __launch_bounds__(256) void expert_combine_kernel(CombineParams p) {
  using V = Vec<T>;
  constexpr int ES = EpiElem<T>::SIZE, G = 4;
  const uint32_t per = (uint32_t)(p.cols / V::N);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / per;
  if (t >= p.tokens) return;
  const int64_t c = (i - t * per) * V::N;
  const uint32_t total = (uint32_t)(p.tokens * p.top_k);
  V sum;
#pragma unroll
  for (int k = 0; k < V::N; ++k) sum.v[k] = 0.0f;
  if (p.R) sum.decode(*(const v4u*)((const char*)p.R + (t * p.ldr + c) * ES));
  const int32_t* rows = p.rows + t * p.top_k;
  const float* w = p.weights ? p.weights + t * p.top_k : nullptr;
  for (int j0 = 0; j0 < p.top_k; j0 += G) {
    v4u y[G];
    float f[G];
    bool live[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int j = j0 + g;
      const uint32_t r = j < p.top_k ? (uint32_t)rows[j] : ~0u;
      live[g] = r < total;
      f[g] = w && j < p.top_k ? w[j] : 1.0f;
      if (live[g]) y[g] = __builtin_nontemporal_load((const v4u*)((const char*)p.Y + ((int64_t)r * p.ldy + c) * ES));
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (!live[g]) continue;
      V x;
      x.decode(y[g]);
#pragma unroll
      for (int k = 0; k < V::N; ++k) sum.v[k] = __builtin_fmaf(f[g], x.v[k], sum.v[k]);
    }
  }
  __builtin_nontemporal_store(sum.pack(), (v4u*)((char*)p.D + (t * p.ldd + c) * ES));
}

// The gradient: W waves take a token (W == 4: a workgroup, W == 1: four tokens
// per workgroup) and G of its choices at a time, so that dD is read once for
// them; the products with the rows are summed over lanes, then waves, in a
// fixed order.  Bound by memory: 8192 tokens of 2 choices, 4096 columns of bf16, 336 MB
// in 51 to 55 us.
template <int T, int W>
__global__ __launch_bounds__(256) void expert_combine_grad_kernel(CombineParams p) {
  using V = Vec<T>;
  constexpr int ES = EpiElem<T>::SIZE, G = 4;
  __shared__ float red[4][G];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = W == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
  if (W == 1 && t >= p.tokens) return;
  const uint32_t total = (uint32_t)(p.tokens * p.top_k);
  const char* dd = (const char*)p.dD + t * p.ldd * ES;
  for (int j0 = 0; j0 < p.top_k; j0 += G) {
    uint32_t r[G];
    float w[G], sum[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const bool there = j0 + g < p.top_k;
      r[g] = there ? (uint32_t)p.rows[t * p.top_k + j0 + g] : ~0u;
      w[g] = there ? p.weights[t * p.top_k + j0 + g] : 0.0f;
      sum[g] = 0.0f;
    }
    for (int64_t c = (int64_t)((W == 4 ? wave * 64 : 0) + lane) * V::N; c < p.cols; c += W * 64 * V::N) {
      V d;
      d.decode(*(const v4u*)(dd + c * ES));
      v4u y[G];
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (r[g] < total) y[g] = __builtin_nontemporal_load((const v4u*)((const char*)p.Y + ((int64_t)r[g] * p.ldy + c) * ES));
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (r[g] >= total) continue;
        V x, o;
        x.decode(y[g]);
#pragma unroll
        for (int k = 0; k < V::N; ++k) {
          sum[g] = __builtin_fmaf(d.v[k], x.v[k], sum[g]);
          o.v[k] = w[g] * d.v[k];
        }
        __builtin_nontemporal_store(o.pack(), (v4u*)((char*)p.dY + ((int64_t)r[g] * p.ldg + c) * ES));
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) sum[g] += __shfl_xor(sum[g], d);
    if constexpr (W == 4) {
      if (lane == 0) {
#pragma unroll
        for (int g = 0; g < G; ++g) red[wave][g] = sum[g];
      }
      __syncthreads();
      if (threadIdx.x < G && j0 + (int)threadIdx.x < p.top_k)
        p.dweights[t * p.top_k + j0 + threadIdx.x] =
            (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
      __syncthreads();
    } else if (lane == 0) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (j0 + g < p.top_k) p.dweights[t * p.top_k + j0 + g] = sum[g];
    }
  }
}

template <int T>
void combine(const CombineParams& p, hipStream_t s) {
  const int64_t n = p.tokens * (p.cols / Vec<T>::N);
  hipLaunchKernelGGL(expert_combine_kernel<T>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, p);
}

// A workgroup per token where a row has 16 bytes for each of its threads (and a
// launch has the threads), else a wave (8192 tokens of 2 choices, bf16: 55 and 61 us
// with 4096 columns, 14.6 and 10.2 with 512).
template <int T>
void combine_grad(const CombineParams& p, hipStream_t s) {
  if (p.cols >= 256 * Vec<T>::N && p.tokens < int64_t(1) << 24)
    hipLaunchKernelGGL((expert_combine_grad_kernel<T, 4>), dim3((unsigned)p.tokens), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((expert_combine_grad_kernel<T, 1>), dim3((unsigned)((p.tokens + 3) / 4)), dim3(256), 0, s, p);
}

}  // namespace

void launch_expert_sort(const SortParams& p, hipStream_t s) {
  const int64_t pieces = p.X ? p.tokens * (p.row_bytes / 16) : 0;
  if (p.chunks > 1) {
    hipLaunchKernelGGL(expert_count_kernel<4>, dim3(p.chunks), dim3(kSortThreads), 0, s, p);
    hipLaunchKernelGGL((expert_rank_kernel<4, false>), dim3(p.chunks), dim3(kSortThreads), 0, s, p);
  } else if (p.tokens * p.top_k > kSortChunk) {
    hipLaunchKernelGGL((expert_rank_kernel<8, false>), dim3(1), dim3(kSortThreads), 0, s, p);
  } else if (p.X) {
    const int64_t blocks = (pieces + kSortThreads - 1) / kSortThreads;
    hipLaunchKernelGGL((expert_rank_kernel<4, true>), dim3((unsigned)(blocks < 256 ? blocks : 256)), dim3(kSortThreads), 0, s, p);
    return;
  } else {
    hipLaunchKernelGGL((expert_rank_kernel<4, false>), dim3(1), dim3(kSortThreads), 0, s, p);
  }
  if (p.X) hipLaunchKernelGGL(expert_gather_kernel, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, s, p);
}

void launch_expert_combine(int t, const CombineParams& p, hipStream_t s) {
  if (t == T_F16) combine<T_F16>(p, s);
  else if (t == T_BF16) combine<T_BF16>(p, s);
  else combine<T_F32>(p, s);
}

void launch_expert_combine_grad(int t, const CombineParams& p, hipStream_t s) {
  if (t == T_F16) combine_grad<T_F16>(p, s);
  else if (t == T_BF16) combine_grad<T_BF16>(p, s);
  else combine_grad<T_F32>(p, s);
}

}  // namespace gemm_epi
