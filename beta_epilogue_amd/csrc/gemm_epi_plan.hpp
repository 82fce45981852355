// gemm_epi_plan.hpp -- the plan's cost model (host): tile shape and K split,
// shared by the GEMM's and the linear layer's plans.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace gemm_epi {

// A plan's problem as the model sees it.
struct PlanProblem {
  int64_t M, N, K, L;
  double epi_bytes;  // bytes per output element that the epilogue moves
  bool may_split;    // false: never split (uint8)
};

// Plan cost model (measured on MI355X, fp16 with C, X, D, Y; times in us).
// A K tile of one output tile takes 1.1 us with 256x256 tiles; with the
// smaller tiles their share of the work at a lower per-CU rate (192x256:
// 0.75 at 0.9, 128x256: 0.5 at 0.67, 128x128: 0.25 at ~0.46).  The split-K
// reduction costs 4 us plus its bytes (S partial-sum slots and C, X, D, Y
// per split tile) at 5 TB/s.
inline double ktile_us(int bm, int bn) {
  if (bm == 256 && bn == 256) return 1.1;
  if (bm == 192 && bn == 256) return 1.1 * 0.75 / 0.9;
  if (bm == 128 && bn == 256) return 1.1 * 0.75;
  return 0.6;
}

struct SplitChoice {
  int64_t splits, tail;  // K slices of the split tiles (1: none), split tiles
  double us;             // modelled time of the launch
};

// The split choice for bm x bn tiles (K tiles of bk) and the modelled time:
// when the
// last round of tiles (tiles % cus, all of them with fewer tiles than CUs)
// would leave at least half of the CUs idle, those tiles may run in S K
// slices after whole-K rounds of the others; S (2 .. min(cus / last,
// K tiles / 4, 16)) maximises the time saved in the last round,
// (K tiles - ceil(K tiles / S)) K-tile times, less the reduction's cost; no S
// with a positive balance, no split.
inline SplitChoice split_choice(int bm, int bn, int bk, const PlanProblem& d, int64_t cus) {
  const int64_t tiles = ((d.M + bm - 1) / bm) * ((d.N + bn - 1) / bn) * d.L;
  const int64_t ktiles = (d.K + bk - 1) / bk;
  const double tk = ktile_us(bm, bn);
  const int64_t last = tiles % cus;
  SplitChoice c{1, 0, (double)((tiles + cus - 1) / cus) * ktiles * tk};
  if (last == 0 || last * 2 > cus || !d.may_split) return c;
  const double slot_bytes = 4.0 * bm * bn;
  const double epi_bytes = d.epi_bytes * bm * bn;
  const int64_t smax = std::min<int64_t>(std::min<int64_t>(cus / last, ktiles / 4), 16);
  double best = 0.0;
  for (int64_t s = 2; s <= smax; ++s) {
    const double saved_us = (double)(ktiles - (ktiles + s - 1) / s) * tk;
    const double cost_us = 4.0 + (double)last * (s * slot_bytes + epi_bytes) / 5.0e6;
    if (saved_us - cost_us > best) {
      best = saved_us - cost_us;
      c.splits = s;
    }
  }
  if (c.splits > 1) {
    c.tail = last;
    c.us -= best;
  }
  return c;
}

}  // namespace gemm_epi
