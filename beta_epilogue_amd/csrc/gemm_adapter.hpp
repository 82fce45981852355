// gemm_adapter.hpp -- device code of the linear layer with low-rank adapters as
// its host code (gemm_adapters.hip) sees it:
//   D = act(A . B^T + bias + scale[g] (A . down[g]^T) . up[g]^T) + R,
// g = ids[m], the adapter of row m (none outside 0 .. adapters - 1).
//
// Two launches.  The first makes U[m] = scale[g] A[m] . down[g]^T (M x rank,
// gemm_adapter_down.hip), rounded once to the operands' type, which the matrix
// cores read next; the second is the linear layer's kernel, whose accumulators
// take U . up[g]^T on top of A . B^T, so D is read and written once and the sum is
// rounded once.
#pragma once

#include "gemm_grouped.hpp"

namespace gemm_epi {

struct AdapterParams : LinParams {
  const void* U;          // M x rank
  const void* up;         // adapters x N x rank
  const int32_t* ids;     // M
  const uint32_t* finite; // adapters: a byte for each part of up[g], 1 where it is finite
  int32_t rank, adapters;
};

constexpr int kFiniteParts = 4;
constexpr uint32_t kFinite = 0x01010101u;  // all of them
constexpr int kMaxRank = 128;

// The adapter of row m; -1: none, or no such row.
__device__ __forceinline__ int row_adapter(const AdapterParams& p, int64_t m) {
  const int g = m < p.M ? p.ids[m] : -1;
  return g >= 0 && g < p.adapters ? g : -1;
}

// A fragment's 16 bytes of 16 rows: lane (q, r) has k = k0 + 8 q .. + 7 of its row.
__device__ __forceinline__ v4i adapter_load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t adapter_up(const AdapterParams& p, int g) {
  const int64_t bytes = p.N * p.rank * 2;
  return __builtin_amdgcn_make_buffer_rsrc((void*)((const char*)p.up + g * bytes), (short)0, (int)bytes, 0x00020000);
}

// The adapters of a tile's rows.  U . up[g]^T is a contraction like A . B^T, so the
// adapters that the tile's rows have add K tiles to the tile's, staged and
// multiplied by the same loop: A's rows are U's, zero for rows of other adapters,
// B's are up[g]'s.  A K tile of 64 holds as many adapters as fit (rank 16: four).
// Packed prompts have one or two adapters per tile (4001 x 4096 x 4096, rank 64: 110 us,
// a plain projection 95 to 101); a batch of single tokens has up to one per row
// (256 rows of 48 adapters, rank 16: 34 us with both launches).
//
// A zero times an infinity or a NaN in up[g] would reach the other rows, so an
// adapter whose up[g] is not finite (the first launch has looked) is left out
// there and added by `step`, which keeps its own rows only.
template <class CF>
struct AdapterTiles {
  using MM = typename CF::MM;
  static_assert(CF::BLK == 16 && MM::KSB == 64 && CF::ROWB == 128 && CF::BM <= CF::THREADS, "16-bit operands, 16x16 blocks");
  // behind the ring, in words: the rows' ids, the adapters' finite words, the rows'
  // adapters, a list of them, a bit for each, counts
  static constexpr int BITS = kMaxExperts / 32, FINITE = CF::BM, ROW = FINITE + kMaxExperts, LIST = ROW + CF::BM,
                       SEEN = LIST + CF::BM, COUNT = SEEN + BITS;
  static constexpr int LDS_BYTES = (COUNT + 4) * 4;
  int tiles;        // K tiles
  bool apart;       // some row's adapter is not finite
  int m0, n0;       // the tile's first row and column
  int slot;         // of this lane's 16 bytes of a K tile: which of its adapters,
  uint32_t k;       // and which byte of the rank (past it: at least 2 * rank)
  int shift;        // adapters in a K tile: 1 << shift; -1: two K tiles for one
  uint32_t bytes;   // of a row of U and of up
  int listed;       // adapters in the list
  uint32_t at;      // the byte in up of the adapter being staged, 0x80000000: none
  uint32_t mine;    // bit Q: the row that instruction Q stages has it

  static __device__ __forceinline__ int* words(char* lds) { return (int*)(lds + CF::LDS_BYTES); }

  // 64 words from byte `from` of r to byte `to` of LDS.
  static __device__ __forceinline__ void fetch64(v4i r, uint32_t from, uint32_t to, int lane) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %1, %2, 0 offen lds"
        :
        : "s"(to), "v"(from + 4u * (uint32_t)lane), "s"(r)
        : "memory", "m0");
  }
  // Starts to load what `setup` looks at, ahead of the tile's first loads, whose
  // latency is then behind that of these.  on: this item adds adapters at all (one K
  // slice of a tile does).
  __device__ __forceinline__ void fetch(const AdapterParams& p, char* lds, int row0, bool on, int wave, int lane) {
    m0 = row0;
    tiles = 0;
    apart = false;
    if (!on) return;
    const uint32_t at = (uint32_t)(uintptr_t)(lds_void_t*)words(lds);
    const int rows = (int)min((int64_t)CF::BM, p.M - m0);
    if (wave < CF::BM / 64)
      fetch64(make_rsrc((const char*)(p.ids + m0), (uint32_t)rows * 4), (uint32_t)wave * 256, at + (uint32_t)wave * 256, lane);
    const v4i rf = make_rsrc((const char*)p.finite, (uint32_t)p.adapters * 4);
    for (int c = wave; c * 64 < p.adapters; c += CF::NW)
      fetch64(rf, (uint32_t)c * 256, at + FINITE * 4 + (uint32_t)c * 256, lane);
    if (threadIdx.x < BITS + 2) words(lds)[SEEN + threadIdx.x] = 0;
  }

  // After a wait for the loads of `fetch`.  cb: the byte of K that this lane stages.
  __device__ __forceinline__ void setup(const AdapterParams& p, char* lds, int column0, bool on, uint32_t cb) {
    n0 = column0;
    if (!on) return;
    int* w = words(lds);
    const int t = threadIdx.x;
    barrier_lds();
    if (t < CF::BM) {
      int g = (int64_t)m0 + t < p.M ? w[t] : -1;
      if (g < 0 || g >= p.adapters) g = -1;
      if (g >= 0) {
        if ((uint32_t)w[FINITE + g] == kFinite) atomicOr(&w[SEEN + (g >> 5)], 1 << (g & 31));
        else g = -1, atomicOr(&w[COUNT + 1], 1);
      }
      w[ROW + t] = g;
    }
    barrier_lds();
    if (t < 64) {
      uint32_t word = t < BITS ? (uint32_t)w[SEEN + t] : 0u;
      const int n = __popc(word), sum = wave_scan(n);
      for (int i = sum - n; word; ++i, word &= word - 1) w[LIST + i] = t * 32 + __ffs(word) - 1;
      if (t == 63) w[COUNT] = sum;
    }
    barrier_lds();
    listed = __builtin_amdgcn_readfirstlane(w[COUNT]);
    apart = __builtin_amdgcn_readfirstlane(w[COUNT + 1]) != 0;
    bytes = (uint32_t)p.rank * 2;
    shift = p.rank <= 8 ? 3 : p.rank <= 16 ? 2 : p.rank <= 32 ? 1 : p.rank <= 64 ? 0 : -1;
    tiles = shift < 0 ? 2 * listed : (listed + (1 << shift) - 1) >> shift;
    slot = shift < 0 ? 0 : (int)(cb >> (7 - shift));
    k = shift < 0 ? cb : cb & (127u >> shift);
    at = 0x80000000u;
    mine = 0;
  }

  // The row that this lane stages by instruction Q.
  template <int Q>
  static __device__ __forceinline__ uint32_t stage_row() {
    const int lane = __lane_id(), wave = threadIdx.x >> 6;
    return (uint32_t)((Q * CF::NW + wave) * CF::ROWS_PER_DMA + lane / CF::CH);
  }
  // Instruction Q of K tile t (a K tile's instructions are issued in order, the rows'
  // first).  The rows' adapters are looked up together, for one wait for LDS between
  // the MFMAs (4001 x 4096 x 4096, rank 64: 136.5 us in all with one each, 134.4 so).
  template <int Q>
  __device__ __forceinline__ void issue_rows(const AdapterParams& p, char* lds, uint32_t sbase, int t) {
    const uint32_t kk = k + (shift < 0 && (t & 1) ? 128u : 0u);
    if constexpr (Q == 0) {
      const int a = shift < 0 ? t >> 1 : (t << shift) + slot;
      const bool any = a < listed && kk < bytes;
      const int cur = any ? words(lds)[LIST + a] : -2;
      mine = 0;
      static_for<0, CF::BM / (CF::NW * CF::ROWS_PER_DMA)>([&](auto q_c) {
        constexpr int q = decltype(q_c)::value;
        mine |= words(lds)[ROW + stage_row<q>()] == cur ? 1u << q : 0u;
      });
      at = any ? (uint32_t)cur * (uint32_t)p.N * bytes + kk : 0x80000000u;
    }
    const v4i ru = make_rsrc((const char*)p.U + (int64_t)m0 * bytes, (uint32_t)min((int64_t)CF::BM, p.M - m0) * bytes);
    dma16s<(uint32_t)Q * CF::NW * 1024u>(ru, sbase, mine >> Q & 1 ? stage_row<Q>() * bytes + kk : 0x80000000u, 0);
  }
  template <int Q>
  __device__ __forceinline__ void issue_columns(const AdapterParams& p, uint32_t sbase) {
    const int64_t first = (int64_t)n0 * bytes;
    const v4i rp = make_rsrc((const char*)p.up + first, (uint32_t)((int64_t)p.adapters * p.N * bytes - first));
    // (columns past the matrix get something else's weights, and are never stored)
    dma16s<(uint32_t)Q * CF::NW * 1024u>(rp, sbase, at != 0x80000000u ? at + stage_row<Q>() * bytes : 0x80000000u, 0);
  }

  // Adds what was left out to a wave's accumulators (rows mw .., columns nw ..):
  // block row by block row, fragments straight from the cache.
  template <class ACC>
  __device__ __forceinline__ void step(const AdapterParams& p, ACC (&acc)[CF::FM][CF::FN], int mw, int nw) const {
    const int lane = __lane_id(), r = lane & 15, q = lane >> 4;
    const int rows = (int)min(max(p.M - mw, (int64_t)0), (int64_t)CF::WM);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)((const char*)p.U + (int64_t)mw * p.rank * 2), (short)0, rows * p.rank * 2, 0x00020000);
    const uint32_t row = (uint32_t)p.rank * 2, ub = (uint32_t)r * row + 16 * q, nb = (uint32_t)(nw + r) * row + 16 * q;
    static_for<0, CF::FM>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      int id = row_adapter(p, mw + i * 16 + r);
      if (id >= 0 && p.finite[id] == kFinite) id = -1;
      uint32_t todo = (uint32_t)__ballot(id >= 0) & 0xffffu;  // rows whose adapter is still to come
      while (todo) {
        const int g = __builtin_amdgcn_readlane(id, __ffs(todo) - 1);
        const uint32_t mine = (uint32_t)__ballot(id == g) & 0xffffu;
        todo &= ~mine;
        const __amdgpu_buffer_rsrc_t rp = adapter_up(p, g);
        for (int k = 0; k < p.rank; k += 32) {
          const bool in = k + 8 * q < p.rank;
          const v4i fa = adapter_load(rw, in && id == g ? ub + i * 16 * row + 2 * k : 0x80000000u);
          v4i fb[CF::FN];
          // (columns past the matrix lie outside the resource)
#pragma unroll
          for (int j = 0; j < CF::FN; ++j) fb[j] = adapter_load(rp, in ? nb + j * 16 * row + 2 * k : 0x80000000u);
#pragma unroll
          for (int j = 0; j < CF::FN; ++j) {
            const typename MM::acc_t t = MM::mma(fa, fb[j], typename MM::acc_t{});
#pragma unroll
            for (int v = 0; v < MM::ACCN; ++v) acc[i][j][v] += mine >> MM::acc_row(lane, v) & 1 ? t[v] : 0.0f;
          }
        }
      }
    });
  }
};

// U[m] = scale[g] A[m] . down[g]^T of type ab (T_F16 or T_BF16); rows without an
// adapter are left as they are.  finite (NULL: not wanted): whether each part of
// up[g] is, for the adapters that some row has.
struct AdapterDownParams {
  const void* A;
  const void* down;    // adapters x rank x K
  const void* up;      // adapters x N x rank
  const float* scale;  // adapters
  const int32_t* ids;
  void* U;
  uint8_t* finite;     // kFiniteParts each
  int32_t* order;      // workspace, with adapter_sorted (else NULL): the rows by adapter,
  int32_t* offsets;    // where each adapter's begin,
  int32_t* counts;     // and the sort's
  int64_t M, N, K, lda;
  int32_t rank, adapters;
};
// Up to so many products (rows times rank) a wave makes each by itself; of more the
// rows are sorted by adapter first, where there are more than two.  (256 rows of rank
// 64, 4096 x 4096, 4 adapters, in all: 37.5 against 38.8 us; 1024 of rank 32, 8 adapters:
// 77.6 against 68.1.)
constexpr int64_t kAdapterDots = 16384;
inline bool adapter_sorted(int64_t M, int rank, int adapters) { return M * rank > kAdapterDots && adapters > 2; }
void launch_adapter_down(int ab, const AdapterDownParams& p, hipStream_t s);

// The linear layer's kernels with the rows' adapters.
template <int AB, int BM, int BN, int S, int OCC>
using AdapterCfg = Cfg<AB, true, true, true, BM, BN, 128, 2, 2, S, 0, 16, 6, OCC>;
// Tile kernel bm x bn of the linear layer's plan (one of part PART).
constexpr int kAdapterParts = 4;
template <int PART>
void launch_adapter_part(int ab, int bm, const AdapterParams& p, int grid, hipStream_t s);
void launch_adapter_rows(int ab, int nw, const AdapterParams& p, hipStream_t s);

}  // namespace gemm_epi
