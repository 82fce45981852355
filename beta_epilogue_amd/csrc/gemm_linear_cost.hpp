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

// Rounds of `items` tiles of bm x bn over `ktiles` K tiles, occ workgroups to a
// compute unit.
inline double linear_rounds(const LinearCost& w, int bm, int bn, int occ, int64_t items, int64_t ktiles, int64_t cus) {
  if (items == 0) return 0.0;
  double tk = bm == 256 ? w.tk256 : bm == 192 ? w.tk192 : bn == 256 ? w.tk128x256 : bm == 128 ? w.tk128 : w.tk64;
  int64_t slots = cus;
  if (occ >= 2 && items > cus) tk = bm == 128 ? w.pair128 : w.pair64, slots = 2 * cus;
  if (occ >= 3 && items > 2 * cus) tk = w.three64, slots = 3 * cus;
  return (double)((items + slots - 1) / slots) * (tk * (double)ktiles + linear_epilogue_time(w, bm, bn));
}

}  // namespace gemm_epi
