// heads_plan.h -- how the per-head kernels spread over waves (host code alone).
//
// A head of dim elements lies on 2^lane_bits lanes, a chunk of 8 elements in
// each; a wave takes 2^slot_bits heads of a token side by side, and, where a
// token has fewer heads than fit, 64 >> (lane_bits + slot_bits) tokens.  A
// token's heads are walked in `steps` steps by each of `slices` waves.
#pragma once

#include <stdint.h>

namespace hdq {

constexpr int kHeadMaxDim = 512;           // 64 lanes
constexpr int64_t kHeadMaxHeads = 1 << 20;  // of one call

struct HeadPlan {
  int lane_bits, slot_bits;
  int steps, slices;
  int64_t waves;
};

inline int bits_for(int64_t n) {  // smallest b with 2^b >= n
  int b = 0;
  while ((int64_t(1) << b) < n) ++b;
  return b;
}

// Waves wanted before a wave takes more than one step: 2048 are eight for each
// CU.  Fewer, longer waves compute a token's angles less often, more waves
// hide latency.
constexpr int64_t kHeadWaves = 2048;

inline HeadPlan plan_heads(int64_t tokens, int64_t heads, int dim) {
  HeadPlan p;
  p.lane_bits = bits_for((dim + 7) / 8);
  const int fit = 6 - p.lane_bits;
  p.slot_bits = heads >= (int64_t(1) << fit) ? fit : bits_for(heads);
  const int64_t per_wave = int64_t(1) << (6 - p.lane_bits - p.slot_bits);
  const int64_t groups = (tokens + per_wave - 1) / per_wave;
  const int64_t total = (heads + (int64_t(1) << p.slot_bits) - 1) >> p.slot_bits;
  int64_t slices = (kHeadWaves + groups - 1) / groups;
  if (slices > total) slices = total;
  p.steps = (int)((total + slices - 1) / slices);
  p.slices = (int)((total + p.steps - 1) / p.steps);
  p.waves = groups * p.slices;
  return p;
}

}  // namespace hdq
