// gemm_linear_cost.hpp -- the cost model (host) of the linear layer's tile kernels,
// from which plans are chosen.
#pragma once

#include <stdint.h>

#include "gemm_linear.hpp"

namespace gemm_epi {

// The plan's cost model (us), fitted per type to 1054 forced plans (24 shapes, M
// 90 to 8192, N 704 to 8192, K 512 to 8192; every tile, 1 to 6 slices), weighted
// towards each shape's best ones: 3 to 6 % rms from the measured times there, and
// the plans that it chooses of them take under 1 % longer on the mean, 17 % at worst,
// than the best measured ones.  An item (a tile or a K slice of one) takes its
// K tiles times tk plus an epilogue of e0 + e1 * area (in 256x256 tiles); rounds
// of items fill the compute units.  Smaller tiles of which two or three share a
// compute unit take pair or three together.  Slices add a second launch, `join`
// us and their partial sums at bw TB/s.
struct LinearCost {
  double start, join, bw, e0, e1;
  double tk256, tk192, tk128x256, tk128, tk64, pair128, pair64, three64;
};
constexpr LinearCost kCost16 = {0.98, 3.65, 21.9, 3.11, 10.4, 1.296, 1.032, 0.0, 0.592, 0.231, 0.821, 0.344, 0.0};
constexpr LinearCost kCostE4m3 = {1.89, 4.93, 32.2, 2.6, 11.4, 1.373, 1.007, 0.685, 0.407, 0.218, 0.0, 0.329, 0.0};
constexpr LinearCost kCostI8 = {1.1, 4.2, 21.8, 3.36, 10.8, 1.287, 1.027, 0.0, 0.61, 0.259, 0.856, 0.361, 0.509};
constexpr LinearCost kCostWide = {2.41, 3.49, 14.5, 2.14, 14.3, 0.0, 0.0, 0.0, 0.796, 0.349, 1.43, 0.53, 0.0};

inline const LinearCost& linear_cost(int ab) {
  return ab == T_E4M3 ? kCostE4m3 : ab == T_I8 ? kCostI8 : ab == T_E4M3_WIDE ? kCostWide : kCost16;
}

inline double linear_epilogue_time(const LinearCost& w, int bm, int bn) {
  return w.e0 + w.e1 * ((double)bm * bn / 65536.0);
}

// The adapters of a projection's rows (gemm_adapter.hpp), and the K tiles of 64 that
// they add to a tile of bm rows, or to the first K slice of one: for as many adapters
// as the tile's rows meet where those of each adapter lie together, of which rows in
// any other order meet more.  Over 84 shapes (24 to 4001 rows, 1 to 300 adapters of rank
// 8 to 128, N 256 to 8192, K 256 to 8192) the plans with them take 0.4 % longer than the
// best ones with packed rows and 0.8 % with mixed ones, 17 % at worst; without them 1.9
// and 2.3 %, 40 % (64 rows of 48 adapters of rank 32, 512 x 4096: K slices for 30 us, the
// few-row kernel takes 21; 512 rows of 300 of rank 8, 1024 x 8192: 52 and 40).
struct LinearAdapters {
  int rank, adapters;
  double k_tiles(int64_t M, int bm) const {
    const double rows = (double)(M < bm ? M : bm), met = 1.0 + rows * adapters / (double)M;
    const double n = met < adapters ? met : adapters;
    if (rank > 64) return 2.0 * n;
    const double tiles = n / (rank <= 8 ? 8 : rank <= 16 ? 4 : rank <= 32 ? 2 : 1);
    return tiles < 1.0 ? 1.0 : tiles;
  }
};

// Rounds of `items` tiles of bm x bn over `ktiles` K tiles, occ workgroups to a
// compute unit.
inline double linear_rounds(const LinearCost& w, int bm, int bn, int occ, int64_t items, double ktiles, int64_t cus) {
  if (items == 0) return 0.0;
  double tk = bm == 256 ? w.tk256 : bm == 192 ? w.tk192 : bn == 256 ? w.tk128x256 : bm == 128 ? w.tk128 : w.tk64;
  int64_t slots = cus;
  if (occ >= 2 && items > cus) tk = bm == 128 ? w.pair128 : w.pair64, slots = 2 * cus;
  if (occ >= 3 && items > 2 * cus) tk = w.three64, slots = 3 * cus;
  return (double)((items + slots - 1) / slots) * (tk * ktiles + linear_epilogue_time(w, bm, bn));
}

}  // namespace gemm_epi
