// fp8_device.h -- FP8 (OCP E4M3) block-128 coding shared by the quantizers and
// the fused producers.
//
// A lane holds 32 consecutive elements of a row, so a block of 128 is four
// adjacent lanes (a DPP quad): its maximum is two quad_perm steps, and every
// lane stores its 32 code bytes as two 16-byte words.
#pragma once

#include "hdq_device.h"

namespace hdq {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;

inline int64_t fp8_blocks(int64_t cols) { return (cols + kFp8Block - 1) / kFp8Block; }

// Maximum over the four lanes of a quad; NaN wins.
__device__ __forceinline__ float quad_max(float v) {
  v = __builtin_elementwise_maximum(
      v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true)));  // quad_perm [1,0,3,2]
  v = __builtin_elementwise_maximum(
      v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true)));  // quad_perm [2,3,0,1]
  return v;
}

// Maximum over the 16 lanes of a DPP row; NaN wins.
__device__ __forceinline__ float row16_max(float v) {
  v = __builtin_elementwise_maximum(
      v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x128, 0xF, 0xF, true)));  // row_ror:8
  v = __builtin_elementwise_maximum(
      v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x124, 0xF, 0xF, true)));  // row_ror:4
  return quad_max(v);
}

// max |y| of the lane's 32 values; NaN wins.
__device__ __forceinline__ float absmax32(const float (&y)[32]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = __builtin_elementwise_maximum(m, fabsf(y[i]));
  return m;
}

// Scale of a block with maximum a, and the factor its values are coded with.
// Not finite: scale NaN, factor 0 (the caller's values then code to zero, see
// fp8_encode32); a below 2^-100: both 0.
__device__ __forceinline__ void fp8_scales(float a, float& scale, float& inv) {
  const bool finite = a < __builtin_inff();  // false for NaN
  const bool live = finite && a >= kTiny;
  scale = live ? a / kFp8Max : (finite ? 0.0f : __builtin_nanf(""));
  inv = live ? kFp8Max / a : 0.0f;
}

// Eight codes (two words), as fp8_encode32.
__device__ __forceinline__ uint2 fp8_encode8(const float (&y)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * q] * inv, y[4 * q + 1] * inv, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * q + 2] * inv, y[4 * q + 3] * inv, v, true);
    w[q] = inv != 0.0f ? (uint32_t)v : 0u;
  }
  return make_uint2(w[0], w[1]);
}

// E4M3 codes of y * inv (|y * inv| <= 448 (1 + 2^-23), which rounds to 448);
// inv 0 gives zeros whatever y holds.
__device__ __forceinline__ void fp8_encode32(const float (&y)[32], float inv, uint4 (&out)[2]) {
  uint32_t w[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * q] * inv, y[4 * q + 1] * inv, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * q + 2] * inv, y[4 * q + 3] * inv, v, true);
    w[q] = inv != 0.0f ? (uint32_t)v : 0u;
  }
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Loads 32 bf16 at chunk `c` (8 elements each) of a row of nch chunks; chunks
// past the row read zero.
__device__ __forceinline__ void load_row32(const uint4* __restrict__ row, int c, int nch, float (&y)[32]) {
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = c + i < nch ? row[c + i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float t[8];
    bf16x8_to_f32(w[i], t);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[8 * i + e] = t[e];
  }
}

// Rotates the lane's 32 values in blocks of HB and scales by fl32(1/sqrt(HB)).
template <int HB>
__device__ __forceinline__ void rotate32(float (&y)[32], int lane, float c_b) {
  if constexpr (HB > 1) {
    const float sc = fwht_w32<HB>(y, lane) * c_b;
#pragma unroll
    for (int i = 0; i < 32; ++i) y[i] = y[i] * sc;
  }
}

}  // namespace hdq
