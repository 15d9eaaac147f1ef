// heads_plan.h -- how the per-head kernels spread over waves (host code alone).
//
// A head of dim elements lies on 2^lane_bits lanes, one or two chunks of 8
// elements in each; a wave takes 2^slot_bits heads of a token side by side, and, where a
// token has fewer heads than fit, 64 >> (lane_bits + slot_bits) tokens.  A
// token's heads are walked in steps within one tensor (queries, keys or
// values), the values' by waves of their own.
#pragma once

#include <stdint.h>

namespace hdq {

constexpr int kHeadMaxDim = 512;           // 64 lanes
constexpr int64_t kHeadMaxHeads = 1 << 20;  // of one call
constexpr int64_t kMaxSlices = 16384;       // waves of a token: grids have fewer than 2^16 layers

struct HeadPlan {
  int lane_bits, slot_bits;
  int step_end[3];  // steps of the first tensor, of the first two, of all: a step is one tensor's
  int steps;        // of a wave
  int slices[2];    // waves of a token (or group of tokens) for the first two tensors, and for the third
  int64_t groups;   // of tokens
};

inline int bits_for(int64_t n) {  // smallest b with 2^b >= n
  int b = 0;
  while ((int64_t(1) << b) < n) ++b;
  return b;
}

// Waves wanted before a wave takes more than one step, of the kernels that may have
// angles to compute (fewer, longer waves do that less often; calls without angles
// take the same) and of the cache's reader: eight and 32 a CU.  With 512 and 8192 in
// place of 2048, 1350 tokens of 60 heads, rotated, took 9.7 and 9.7 us (8.3), 4050 of 90
// into the cache 22.7 and 25.3 (22.9, now 20); reading 5400 tokens of 30 with 2048
// and 32768 in place of 8192 14.5 and 16.1 (14.3).
constexpr int64_t kHeadWaves = 2048, kReadWaves = 8192;

// log2 of the lanes a group's maximum is taken over: all of a head's when the
// group is the head, else a chunk of 8 in each.
inline int group_lane_bits(int dim, int group, int lane_bits) { return group == dim ? lane_bits : bits_for(group / 8); }

// Tensors of h0, h1 and h2 heads (0: not there), 8 or 16 elements a lane.
inline HeadPlan plan_heads(int64_t tokens, int64_t h0, int64_t h1, int64_t h2, int dim, int per_lane, int64_t wanted) {
  HeadPlan p;
  const int64_t h[3] = {h0, h1, h2};
  int64_t most = h0 > h1 ? h0 : h1;
  if (h2 > most) most = h2;
  p.lane_bits = bits_for((dim + per_lane - 1) / per_lane);
  const int fit = 6 - p.lane_bits;
  p.slot_bits = most >= (int64_t(1) << fit) ? fit : bits_for(most);
  const int64_t per_wave = int64_t(1) << (6 - p.lane_bits - p.slot_bits);
  p.groups = (tokens + per_wave - 1) / per_wave;
  int64_t total = 0;
  for (int t = 0; t < 3; ++t) {
    total += (h[t] + (int64_t(1) << p.slot_bits) - 1) >> p.slot_bits;
    p.step_end[t] = (int)total;
  }
  int64_t slices = (wanted + p.groups - 1) / p.groups;
  if (slices > total) slices = total;
  int64_t steps = (total + slices - 1) / slices;
  if (steps < (total + kMaxSlices - 1) / kMaxSlices) steps = (total + kMaxSlices - 1) / kMaxSlices;
  p.steps = (int)steps;
  p.slices[0] = (int)((p.step_end[1] + steps - 1) / steps);
  p.slices[1] = (int)((total - p.step_end[1] + steps - 1) / steps);
  return p;
}

}  // namespace hdq
