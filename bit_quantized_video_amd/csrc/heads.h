// heads.h -- arguments and device helpers shared by the per-head kernels
// (heads.hip, kv_cache.hip).
#pragma once

#include "fp8_device.h"
#include "heads_plan.h"
#include "hdq_internal.h"

namespace hdq {

enum HeadNorm : int { kHeadNormNone = 0, kHeadNormLayer = 1, kHeadNormRms = 2 };
enum CacheFmt : int { kCacheInt8 = 0, kCacheFp8 = 1, kCacheInt4 = 2 };
// The cache's Hadamard blocks, of kernels for heads of 16 << LL elements: none, whole heads, or g.hb.
enum Hadamard : int { kHadamardNone = 0, kHadamardWhole = 1, kHadamardAny = 2 };
// Its groups: a head each, within half a head, or g.group.
enum Group : int { kGroupHead = 0, kGroupPart = 1, kGroupAny = 2 };

// One of a call's tensors: [batch, length, heads, dim] elements, strides in elements.
struct HeadRows {
  const void* x;
  int64_t xb, xt, xh;
  void* y;  // null: not written as floats (keys and values that go to the cache)
  int64_t yb, yt, yh;
  const float* weight;
  const float* bias;
  int heads;
};

struct HeadArgs {
  HeadRows q, k, v;
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
  // the plan's: the first `qk_slices` layers of the grid take the queries' and keys' steps
  int lane_bits, slot_bits, steps, qk_slices, step_end[3];
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
  int lane_bits, slot_bits, steps;  // the plan's: layers z and z + half of the grid take step z * steps of keys and values
};

// heads16*.hip, for launch_heads
void run_heads16(const HeadArgs& g, dim3 grid, hipStream_t s);
void run_heads16_cache(const HeadArgs& g, dim3 grid, hipStream_t s);
void run_heads16_cache64(const HeadArgs& g, dim3 grid, hipStream_t s);
void run_heads16_cache128(const HeadArgs& g, dim3 grid, hipStream_t s);
void run_heads16_f32(const HeadArgs& g, bool cache, dim3 grid, hipStream_t s);
hipError_t launch_heads(HeadArgs g, bool f32, bool vec, bool cache, hipStream_t s);
hipError_t launch_cache_read(CacheReadArgs g, hipStream_t s);

// Whether two chunks, half a head apart, can lie in a lane: Hadamard blocks and
// groups within half a head, or the whole.
inline bool cache_pairs(int dim, int hb, int group) {
  const int half = dim / 2;
  return dim % 16 == 0 && (hb == dim || half % hb == 0) && (group == dim || half % group == 0);
}
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

// Stores 16 bytes.
template <typename V>
__device__ __forceinline__ void put16(void* p, const V& v) {
  *static_cast<V*>(p) = v;
}

// Integer codes of eight values, rounded to even, in the low bytes of words:
// adding 1.5 2^23 leaves the rounded value in the sum's low bits, two's
// complement; |y * inv| passes top by less than half.
__device__ __forceinline__ void int_codes(const float (&y)[8], float inv, uint32_t (&q)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = __float_as_uint(y[e] * inv + 12582912.0f);
}
// Byte 0 of each of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u), 0x05040100u);
}
__device__ __forceinline__ uint2 int8_word(const float (&y)[8], float inv) {
  uint32_t q[8];
  int_codes(y, inv, q);
  const uint2 w = make_uint2(low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7]));
  return inv != 0.0f ? w : make_uint2(0u, 0u);
}
__device__ __forceinline__ uint32_t int4_word(const float (&y)[8], float inv) {
  uint32_t q[8];
  int_codes(y, inv, q);
  const uint32_t w = (low_bytes(q[0], q[2], q[4], q[6]) & 0x0f0f0f0fu) | (low_bytes(q[1], q[3], q[5], q[7]) & 0x0f0f0f0fu) << 4;
  return inv != 0.0f ? w : 0u;
}

// Codes the lane's chunk at element `at` (a multiple of 8) of a cache's codes;
// inv 0 gives zeros whatever y holds.
__device__ __forceinline__ void store_codes(uint8_t* codes, int64_t at, const float (&y)[8], float inv, int fmt) {
  if (fmt == kCacheFp8)
    *reinterpret_cast<uint2*>(codes + at) = fp8_encode8(y, inv);
  else if (fmt == kCacheInt8)
    *reinterpret_cast<uint2*>(codes + at) = int8_word(y, inv);
  else
    *reinterpret_cast<uint32_t*>(codes + at / 2) = int4_word(y, inv);
}

// The same for chunks x at `at` and y at `at` + far.
__device__ __forceinline__ void store_codes2(uint8_t* codes, int64_t at, int far, const float (&x)[8], const float (&y)[8],
                                             float inv, float inv2, int fmt) {
  if (fmt == kCacheFp8) {
    *reinterpret_cast<uint2*>(codes + at) = fp8_encode8(x, inv);
    *reinterpret_cast<uint2*>(codes + at + far) = fp8_encode8(y, inv2);
  } else if (fmt == kCacheInt8) {
    *reinterpret_cast<uint2*>(codes + at) = int8_word(x, inv);
    *reinterpret_cast<uint2*>(codes + at + far) = int8_word(y, inv2);
  } else {
    *reinterpret_cast<uint32_t*>(codes + at / 2) = int4_word(x, inv);
    *reinterpret_cast<uint32_t*>(codes + at / 2 + far / 2) = int4_word(y, inv2);
  }
}

}  // namespace hdq
