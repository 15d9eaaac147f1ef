// heads_device.h -- device parts shared by the kernels for heads in registers
// (heads.hip, heads16.h): loads, norms, angles, stores.
#pragma once

#include "heads.h"

namespace hdq {

namespace {

constexpr int kWaves = 4;        // waves of a workgroup
constexpr int kUnroll = 2;       // head steps whose loads are in flight together
constexpr int kMaxPairs = 256;   // rotated pairs a wave's tokens have (dim 512, or more tokens of smaller heads)

// Eight elements, the chunk a lane holds, as loaded.
template <bool F32>
struct Chunk;
template <>
struct Chunk<false> {
  uint4 w;
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  template <bool VEC>
  __device__ __forceinline__ void load(const void* p, int n) {
    if constexpr (VEC) {
      w = *static_cast<const uint4*>(p);
    } else {
      const uint16_t* s = static_cast<const uint16_t*>(p);
      uint32_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < n ? s[e] : 0u;
      w = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
  }
  __device__ __forceinline__ void to_f32(float (&x)[8]) const { bf16x8_to_f32(w, x); }
};
template <>
struct Chunk<true> {
  float v[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  }
  template <bool VEC>
  __device__ __forceinline__ void load(const void* p, int n) {
    if constexpr (VEC) {
      const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < n ? static_cast<const float*>(p)[e] : 0.0f;
    }
  }
  __device__ __forceinline__ void to_f32(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v[e];
  }
};

// Rounds (to bf16: to nearest even) and stores n of the eight elements.
template <bool VEC>
__device__ __forceinline__ void store_chunk(void* p, bool f32, const float (&y)[8], int n) {
  if (f32) {
    float* d = static_cast<float*>(p);
    if constexpr (VEC) {
      put16(d, make_float4(y[0], y[1], y[2], y[3]));
      put16(d + 4, make_float4(y[4], y[5], y[6], y[7]));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) d[e] = y[e];
    }
  } else {
    const uint4 w = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    if constexpr (VEC) {
      put16(p, w);
    } else {
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
      uint16_t* d = static_cast<uint16_t*>(p);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) d[e] = (uint16_t)(v[e >> 1] >> ((e & 1) * 16));
    }
  }
}

__device__ __forceinline__ float sum8(const float (&x)[8]) {
  return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}

__device__ __forceinline__ float squares8(const float (&x)[8]) {
  float a = x[0] * x[0], b = x[1] * x[1];
#pragma unroll
  for (int e = 2; e < 8; e += 2) {
    a = fmaf(x[e], x[e], a);
    b = fmaf(x[e + 1], x[e + 1], b);
  }
  return a + b;
}

// The power of two that brings a head of largest magnitude m, and eps with it, near 1.
__device__ __forceinline__ int norm_exponent(float m, float eps) {
  const float big = fmaxf(m, sqrtf(eps));
  return big > 0.0f && big < __builtin_inff() ? ilogbf(big) + 1 : 0;
}

// Whether a sum of squares about `mean` is one that float32 holds well.  The mean's
// error goes with the head's elements, so it has to lie within a deviation of 0:
// heads further off (a constant one is, however small) are taken again.
__device__ __forceinline__ bool squares_hold(float ss, float mean, float inv_dim, float eps) {
  return ss < 0x1p100f && (ss > 0x1p-80f || eps > 0x1p-60f) && mean * mean <= ss * inv_dim;
}

// v of the first of the 2^bits lanes that hold a head (swizzles, which need no
// register for an address).
template <int BITS>
__device__ __forceinline__ float first_of(float v) {
  return __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x1F & ~((1 << BITS) - 1)));
}
__device__ __forceinline__ float lanes_first(float v, int bits) {
  switch (bits) {
    case 0: return v;
    case 1: return first_of<1>(v);
    case 2: return first_of<2>(v);
    case 3: return first_of<3>(v);
    case 4: return first_of<4>(v);
    case 5: return first_of<5>(v);
    default: return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
  }
}

// 1 / sqrt(mean square + eps), a step past the instruction's accuracy (1 unit).
// Sums outside squares_hold's range come scaled, with a largest element near 1, so
// the argument is normal but for a head without deviations, whose eps may be 0, or
// subnormal once scaled, which the instruction takes for 0: 0 for that one.
__device__ __forceinline__ float norm_scale(float ss, float inv_dim, float eps) {
  const float d = fmaf(ss, inv_dim, eps);
  const float r = __builtin_amdgcn_rsqf(d);
  return d < 0x1p-126f ? 0.0f : fmaf(0.5f * r, fmaf(-(d * r), r, 1.0f), r);
}

// A head's scale and its centred values in place.  Sums that do not hold
// are taken again from values scaled by a power of two, which cancels in the
// result, and about a mean in two steps: an element and the mean difference from
// it (of a constant head 0), then the mean of what is left.  A head with a NaN or
// an infinity becomes NaN.
template <bool F32>
__device__ __forceinline__ float head_norm(const Chunk<F32>& raw, float (&x)[8], int n, bool layer, float inv_dim,
                                           float eps, int ll) {
  // the lane's n elements of v less c
  auto less = [&](float (&v)[8], float c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? v[e] - c : 0.0f;
  };
  float mean = 0.0f;
  if (layer) {
    mean = lanes_sum(sum8(x), ll) * inv_dim;
    less(x, mean);
  }
  float ss = lanes_sum(squares8(x), ll);
  const bool ok = squares_hold(ss, mean, inv_dim, eps);
  if (__ballot(!ok) != 0) {
    float v[8], m = 0.0f;
    raw.to_f32(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, fabsf(v[e]));
    m = lanes_max(m, ll);
    const int k = norm_exponent(m, eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], -k);
    if (layer) {
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = v[e];
      const float first = lanes_first(v[0], ll);
      less(d, first);
      less(v, first + lanes_sum(sum8(d), ll) * inv_dim);
      less(v, lanes_sum(sum8(v), ll) * inv_dim);
    }
    const float again = lanes_sum(squares8(v), ll);
    if (!ok) {
      ss = again;
      eps = m < __builtin_inff() ? ldexpf(ldexpf(eps, -k), -k) : __builtin_nanf("");
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = v[e];
    }
  }
  return norm_scale(ss, inv_dim, eps);
}

// LDS between lanes of one wave: what was written is there, and stays until read.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Scaled cosine and sine of pair j at a token's positions.
__device__ __forceinline__ float2 pair_angle(const HeadArgs& g, int64_t p0, int64_t p1, int64_t p2, int j) {
  const double p = (double)(j < g.axis_end[0] ? p0 : j < g.axis_end[1] ? p1 : p2);
  const double f = g.turns[j];
  const double t = p * f, lost = fma(p, f, -t);  // the product in two parts
  // the fraction in two floats, the second in first order: rounded to one, it alone
  // would be half of a rotated element's error
  const double part = (t - rint(t)) + lost;
  const float r = (float)part, rest = 6.2831853f * (float)(part - (double)r);
  float s, co;
  sincospif(2.0f * r, &s, &co);
  return make_float2(fmaf(-rest, s, co) * g.scale, fmaf(rest, co, s) * g.scale);
}

// A token's sequence and place in it; one past the last stands in the first.
struct Token {
  bool in;
  uint32_t batch, pos;
};
__device__ __forceinline__ Token token_of(const HeadArgs& g, int64_t token) {
  Token t;
  t.in = token < g.tokens;
  const uint32_t i = t.in ? (uint32_t)token : 0u;
  t.batch = g.length == g.tokens ? 0u : i / (uint32_t)g.length;
  t.pos = i - t.batch * (uint32_t)g.length;
  return t;
}

// Its positions on the axes; live: it is rotated.
struct Positions {
  int64_t p0, p1, p2;
  bool live;
  __device__ __forceinline__ Positions(const HeadArgs& g, const Token& t) {
    const int64_t* p = g.positions + t.batch * g.pos_batch + t.pos * g.pos_token;
    p0 = p[0];
    p1 = g.axes > 1 ? p[g.pos_axis] : 0;
    p2 = g.axes > 2 ? p[2 * g.pos_axis] : 0;
    live = (p0 | p1 | p2) >= 0;
  }
};

// Weights and biases of a lane's chunk (null: 1 and 0), aligned to an element.
__device__ __forceinline__ void load_weights(const float* p, int at, float other, float (&w)[8]) {
  if (p != nullptr) {
    __builtin_memcpy(w, p + at, 32);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = other;
  }
}

// The wave's steps, of the layer of the grid it is in.
struct Steps {
  int first, end;
};
__device__ __forceinline__ Steps wave_steps(const HeadArgs& g) {
  const int z = (int)blockIdx.z, qk = g.qk_slices;
  const int first = z < qk ? z * g.steps : g.step_end[1] + (z - qk) * g.steps;
  return Steps{first, min(first + g.steps, z < qk ? g.step_end[1] : g.step_end[2])};
}

}  // namespace

}  // namespace hdq
