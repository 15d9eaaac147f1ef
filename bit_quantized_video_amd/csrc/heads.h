// heads.h -- arguments and device helpers shared by the per-head kernels
// (heads.hip, kv_cache.hip).
#pragma once

#include "fp8_device.h"
#include "heads_plan.h"
#include "hdq_internal.h"

namespace hdq {

enum HeadNorm : int { kHeadNormNone = 0, kHeadNormLayer = 1, kHeadNormRms = 2 };
enum CacheFmt : int { kCacheInt8 = 0, kCacheFp8 = 1, kCacheInt4 = 2 };

// One of a call's tensors: [batch, length, heads, dim] elements, strides in elements.
struct HeadRows {
  const void* x;
  int64_t xb, xt, xh;
  void* y;  // null: not written as floats (keys and values that go to the cache)
  int64_t yb, yt, yh;
  const float* weight;
  const float* bias;
};

struct HeadArgs {
  HeadRows q, k, v;
  int heads[3];  // of q; of q and k; of q, k and v
  int64_t tokens, length;
  int dim;
  bool y_f32;
  int norm;
  float eps, inv_dim;
  // rotation: `half` pairs (0: none), pairs j and j + half (split) or neighbours
  int half;
  bool split;
  int axes, axis_end[2];  // pairs of the first axis, and of the first two
  float scale;
  const double* turns;
  const int64_t* positions;
  int64_t pos_axis, pos_batch, pos_token;
  // cache
  int fmt, group, groups, group_bits, hb;  // groups: of a head; group_bits: log2 of a group's lanes
  float c_b, top;
  const int64_t* slots;
  int64_t n_slots;
  uint8_t* codes[2];
  float* scales[2];
  // the plan's
  int lane_bits, slot_bits, steps, slices;
};

// Reading slots back: token t's keys and values go to row t of the outputs.
struct CacheReadArgs {
  const uint8_t* codes[2];
  const float* scales[2];
  void* y[2];
  int64_t tokens, n_slots;
  const int64_t* slots;
  int heads, dim, fmt, group, groups, hb;
  float c_b;
  bool y_f32;
  int lane_bits, slot_bits, steps, slices;
};

hipError_t launch_heads(HeadArgs g, bool f32, bool vec, bool cache, hipStream_t s);
hipError_t launch_cache_read(CacheReadArgs g, hipStream_t s);

// Lanes of a group: all of a head's when the group is the head, else group / 8.
inline int cache_group_bits(int dim, int group) { return bits_for(((group == dim ? dim : group) + 7) / 8); }
inline float cache_top(int fmt) { return fmt == kCacheInt8 ? 127.0f : fmt == kCacheFp8 ? kFp8Max : 7.0f; }

// Sum over the 2^bits lanes (aligned) that hold a head; the same in each.
__device__ __forceinline__ float lanes_sum(float v, int bits) {
  if (bits > 0) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true));   // quad_perm [1,0,3,2]
  if (bits > 1) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true));   // quad_perm [2,3,0,1]
  if (bits > 2) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true));  // row_half_mirror
  if (bits > 3) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true));  // row_mirror
  if (bits > 4) v += xor_lane<16>(v);
  if (bits > 5) v += __shfl_xor(v, 32);
  return v;
}

// Maximum over them; NaN wins.
__device__ __forceinline__ float lanes_max(float v, int bits) {
  auto take = [&](float o) { v = __builtin_elementwise_maximum(v, o); };
  if (bits > 0) take(__int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true)));
  if (bits > 1) take(__int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true)));
  if (bits > 2) take(__int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true)));
  if (bits > 3) take(__int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true)));
  if (bits > 4) take(xor_lane<16>(v));
  if (bits > 5) take(__shfl_xor(v, 32));
  return v;
}

// Scale of a group with maximum a and the factor its values are coded with;
// as the FP8 blocks': below 2^-100 both 0, not finite: scale NaN, factor 0.
__device__ __forceinline__ void code_scales(float a, float top, float& scale, float& inv) {
  const bool finite = a < __builtin_inff();
  const bool live = finite && a >= kTiny;
  scale = live ? a / top : (finite ? 0.0f : __builtin_nanf(""));
  inv = live ? top / a : 0.0f;
}

// Eight integer codes of y * inv, rounded to even, |code| <= top; inv 0: zeros.
__device__ __forceinline__ void int_codes(const float (&y)[8], float inv, float top, int (&q)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = inv != 0.0f ? (int)fminf(fmaxf(rintf(y[e] * inv), -top), top) : 0;
}

// Codes the lane's chunk at element `at` (a multiple of 8) of a cache's codes.
__device__ __forceinline__ void store_codes(uint8_t* codes, int64_t at, const float (&y)[8], float inv, int fmt) {
  if (fmt == kCacheFp8) {
    *reinterpret_cast<uint2*>(codes + at) = fp8_encode8(y, inv);
    return;
  }
  int q[8];
  int_codes(y, inv, fmt == kCacheInt8 ? 127.0f : 7.0f, q);
  if (fmt == kCacheInt8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = (uint32_t)(q[4 * i] & 255) | (uint32_t)(q[4 * i + 1] & 255) << 8 | (uint32_t)(q[4 * i + 2] & 255) << 16 |
             (uint32_t)q[4 * i + 3] << 24;
    *reinterpret_cast<uint2*>(codes + at) = make_uint2(w[0], w[1]);
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= (uint32_t)(q[e] & 15) << (4 * e);
    *reinterpret_cast<uint32_t*>(codes + at / 2) = w;
  }
}

}  // namespace hdq
