// heads.hip -- what lies between a QKV projection and the attention (gfx950):
// norms of queries and keys over each head, rotary positions, and keys and
// values quantized into a cache, all in one pass over the data.
//
// For a head x[0 .. dim) of a token at position p:
//   norm     x <- (x - mean) / sqrt(var + eps) * w + b   (layer), or
//            x <- x / sqrt(mean(x^2) + eps) * w + b      (RMS);
//   rotation pair j (elements 2j, 2j + 1, or j, j + R/2):
//            (a, b) <- s (a cos t - b sin t, b cos t + a sin t),
//            t = 2 pi frac(p * turns[j]), the product and its fraction in float64;
//   cache    y = H_b x / sqrt(b) in blocks of b, code = rne(y * (top / a)) with
//            a = max|y| of a group, scale a / top (top 127, 448 or 7).
// Bound by HBM: every element is read and written once.
#include "heads.h"

#include "fp8_device.h"
#include "hdq_internal.h"

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
      reinterpret_cast<float4*>(d)[0] = make_float4(y[0], y[1], y[2], y[3]);
      reinterpret_cast<float4*>(d)[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) d[e] = y[e];
    }
  } else {
    const uint4 w = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    if constexpr (VEC) {
      *static_cast<uint4*>(p) = w;
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

// Centres the lane's n elements (layer) and returns the head's sum of squares.
__device__ __forceinline__ float centred_squares(float (&x)[8], int n, bool layer, float inv_dim, int ll) {
  if (layer) {
    const float mean = lanes_sum(sum8(x), ll) * inv_dim;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = e < n ? x[e] - mean : 0.0f;
  }
  return lanes_sum(squares8(x), ll);
}

// The power of two that brings a head of largest magnitude m, and eps with it, near 1.
__device__ __forceinline__ int norm_exponent(float m, float eps) {
  const float big = fmaxf(m, sqrtf(eps));
  return big > 0.0f && big < __builtin_inff() ? ilogbf(big) + 1 : 0;
}

// Whether a sum of squares is one that float32 holds well.
__device__ __forceinline__ bool squares_hold(float ss, float eps) { return ss < 0x1p100f && (ss > 0x1p-80f || eps > 0x1p-60f); }

// 1 / sqrt(mean square + eps); sums outside that range come scaled, so the
// argument is normal (or 0: a head of zeros stays zero at eps 0).
__device__ __forceinline__ float norm_scale(float ss, float inv_dim, float eps) {
  const float d = fmaf(ss, inv_dim, eps);
  return d == 0.0f ? 0.0f : __builtin_amdgcn_rsqf(d);
}

// A head's scale and its centred values in place.  Sums that do not hold
// are taken again from values scaled by a power of two, which cancels in the
// result; a head with a NaN or an infinity becomes NaN.
template <bool F32>
__device__ __forceinline__ float head_norm(const Chunk<F32>& raw, float (&x)[8], int n, bool layer, float inv_dim,
                                           float eps, int ll) {
  float ss = centred_squares(x, n, layer, inv_dim, ll);
  const bool ok = squares_hold(ss, eps);
  if (__ballot(!ok) != 0) {
    float v[8], m = 0.0f;
    raw.to_f32(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, fabsf(v[e]));
    m = lanes_max(m, ll);
    const int k = norm_exponent(m, eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], -k);
    const float again = centred_squares(v, n, layer, inv_dim, ll);
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

// What a chunk's elements allow: element loads and any rotation; vector loads;
// and also a rotation whose pairs are whole chunks
// (k_heads), or whole heads on 16 elements a lane (k_heads16).
enum Mode : int { kElements = 0, kVectors = 1, kChunks = 2, kPairs = 3 };

// Scaled cosine and sine of pair j at a token's positions.
__device__ __forceinline__ float2 pair_angle(const HeadArgs& g, int64_t p0, int64_t p1, int64_t p2, int j) {
  const double p = (double)(j < g.axis_end[0] ? p0 : j < g.axis_end[1] ? p1 : p2);
  const double f = g.turns[j];
  const double t = p * f, lost = fma(p, f, -t);  // the product in two parts
  const float r = (float)((t - rint(t)) + lost);
  float s, co;
  sincospif(2.0f * r, &s, &co);
  return make_float2(co * g.scale, s * g.scale);
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

template <bool F32, int MODE, bool CACHE>
__global__ __launch_bounds__(64 * kWaves) void k_heads(const HeadArgs g) {
  constexpr bool VEC = MODE != kElements;
  __shared__ __align__(16) float2 s_trig[kWaves][kMaxPairs];
  __shared__ __align__(16) float s_swap[kWaves][64 * 8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ll = g.lane_bits, sl = g.slot_bits;
  // lane l of a head holds chunk c (in an order that the Hadamard stages like)
  const int c = CACHE ? (int)fwht_src(lane & ((1 << ll) - 1), lane, g.hb) : lane & ((1 << ll) - 1);
  const int hslot = (lane >> ll) & ((1 << sl) - 1);
  const int64_t group0 = ((int64_t)wide_block() * kWaves + wave) * (64 >> (ll + sl)), token = group0 + (lane >> (ll + sl));
  if (group0 >= g.tokens) return;  // whole waves
  const Token at = token_of(g, token);
  const int n = min(8, g.dim - c * 8);  // the lane's elements, <= 0 past the head
  const bool in = at.in && n > 0;

  // Steps: 2^sl heads of a tensor each, the queries' first.  A step's tensor is
  // the same for the whole wave.
  const Steps steps = wave_steps(g);
  auto tensor = [&](int s) { return s < g.step_end[0] ? 0 : !CACHE || s < g.step_end[1] ? 1 : 2; };
  auto block = [&](int t, int s) { return (s - (t == 0 ? 0 : t == 1 ? g.step_end[0] : g.step_end[1])) << sl; };
  auto rows = [&](int t) -> const HeadRows& { return t == 0 ? g.q : !CACHE || t == 1 ? g.k : g.v; };
  constexpr int kIn = F32 ? 4 : 2;
  const int out_size = g.y_f32 ? 4 : 2;

  int x_of = -1;  // whose lane base this is
  const char* x_base = nullptr;
  auto load = [&](Chunk<F32>& raw, int s) {
    if (s >= steps.end) return;
    const int t = tensor(s), h0 = block(t, s);
    const HeadRows& r = rows(t);
    if (t != x_of) {
      x_of = t;
      x_base = static_cast<const char*>(r.x) + (at.batch * r.xb + at.pos * r.xt + hslot * r.xh + c * 8) * kIn;
    }
    if (in && h0 + hslot < r.heads) raw.template load<VEC>(x_base + h0 * r.xh * kIn, n);
  };

  Chunk<F32> raw[kUnroll];  // lanes past a head's end keep zeros
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) raw[u].zero(), load(raw[u], steps.first + u);

  // angles of the wave's tokens: pair j of a token by lane j, j + lanes, ... of it
  float cs[8], sn[8];
  bool live = false;
  if (g.half > 0 && steps.first < g.step_end[1]) {
    const Positions pos(g, at);
    live = pos.live;
    const int per = 1 << (ll + sl);
    float2* trig = s_trig[wave] + (lane >> (ll + sl)) * g.half;
    for (int j = lane & (per - 1); j < g.half; j += per) trig[j] = pair_angle(g, pos.p0, pos.p1, pos.p2, j);
    wave_lds_fence();
    if (g.split) {  // element i of pair i or i - half, the sine negative for the first
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = c * 8 + e, j = i < g.half ? i : i - g.half;
        const float2 v = j < g.half ? trig[j] : make_float2(1.0f, 0.0f);
        cs[e] = v.x;
        sn[e] = i < g.half ? -v.y : v.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = c * 4 + e;
        const float2 v = j < g.half ? trig[j] : make_float2(1.0f, 0.0f);
        cs[e] = v.x;
        sn[e] = v.y;
      }
    }
    if (MODE == kChunks) live = live && c * 8 < 2 * g.half;
  }

  float wt[8], bs[8];
  int w_of = -1, y_of = -1;  // whose weights, whose lane base
  char* y_base = nullptr;
  const int64_t slot = CACHE && in ? g.slots[token] : -1;
  const bool in_cache = slot >= 0 && slot < g.n_slots;

  auto process = [&](const Chunk<F32>& raw, int s) {
    const int t = tensor(s), h = block(t, s) + hslot;
    const HeadRows& r = rows(t);
    const bool ok = in && h < r.heads;
    float x[8];
    raw.to_f32(x);
    if (g.norm != kHeadNormNone && t != 2) {
      if (w_of != t) {
        w_of = t;
        if (VEC) {
          load_weights(r.weight, n > 0 ? c * 8 : 0, 1.0f, wt);
          load_weights(r.bias, n > 0 ? c * 8 : 0, 0.0f, bs);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            wt[e] = r.weight != nullptr && e < n ? r.weight[c * 8 + e] : 1.0f;
            bs[e] = r.bias != nullptr && e < n ? r.bias[c * 8 + e] : 0.0f;
          }
        }
      }
      const float rs = head_norm<F32>(raw, x, n, g.norm == kHeadNormLayer, g.inv_dim, g.eps, ll);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e] * rs, wt[e], bs[e]);
    }
    if (g.half > 0 && t != 2) {
      if (g.split) {
        float p[8];
        float* sw = s_swap[wave] + (lane >> ll << ll) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) sw[c * 8 + e] = x[e];
        wave_lds_fence();
        if (MODE == kChunks || g.half % 4 == 0) {
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const int i = c * 8 + e;
            const float4 v = *reinterpret_cast<const float4*>(sw + (i < g.half ? i + g.half : i < 2 * g.half ? i - g.half : i));
            p[e] = v.x, p[e + 1] = v.y, p[e + 2] = v.z, p[e + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = c * 8 + e;
            p[e] = sw[i < g.half ? i + g.half : i < 2 * g.half ? i - g.half : i];
          }
        }
        wave_lds_fence();
        if (live) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (MODE == kChunks || c * 8 + e < 2 * g.half) x[e] = fmaf(p[e], sn[e], x[e] * cs[e]);
        }
      } else if (live) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (MODE == kChunks || c * 4 + e < g.half) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = fmaf(-b, sn[e], a * cs[e]);
            x[2 * e + 1] = fmaf(a, sn[e], b * cs[e]);
          }
      }
    }
    if (CACHE && t != 0) {
      const float sc = fwht8(x, lane, g.hb) * g.c_b;
      float a = 0.0f;
      if (g.hb > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], sc, 0.0f);  // a difference of 0 has either sign: + 0 is coded
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) a = __builtin_elementwise_maximum(a, fabsf(x[e]));
      float scale, inv;
      code_scales(lanes_max(a, g.group_bits), g.top, scale, inv);
      if (ok && in_cache) {
        const int64_t row = slot * r.heads + h;
        store_codes(g.codes[t - 1], row * g.dim + c * 8, x, inv, g.fmt);
        if ((c * 8) % g.group == 0) g.scales[t - 1][row * g.groups + c * 8 / g.group] = scale;
      }
    } else {
      if (y_of != t) {
        y_of = t;
        y_base = static_cast<char*>(r.y) + (at.batch * r.yb + at.pos * r.yt + hslot * r.yh + c * 8) * out_size;
      }
      if (ok) store_chunk<VEC>(y_base + (h - hslot) * r.yh * out_size, g.y_f32, x, n);
    }
  };

  for (int s = steps.first; s < steps.end; s += kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (s + u < steps.end) {
        process(raw[u], s + u);
        load(raw[u], s + kUnroll + u);
      }
  }
}

// The same for heads of 16 elements a lane, most calls' form: a lane holds
// chunks c and c + dim / 16 of a head, so both elements of a pair, in either
// layout, are its own, and a step's addresses, reductions and tests serve
// twice the elements (half the instructions an element).  dim is a
// multiple of 16 on LL bits of lanes (LL < 0: g.lane_bits), the rotation none,
// interleaved in whole chunks or split over the whole head, a Hadamard block
// and a group within half a head or the whole.
template <bool F32, int LL, bool CACHE>
__global__ __launch_bounds__(64 * kWaves) void k_heads16(const HeadArgs g) {
  __shared__ __align__(16) float2 s_trig[kWaves][2 * kMaxPairs];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ll = LL < 0 ? g.lane_bits : LL, sl = g.slot_bits;
  const int far = g.dim >> 4;  // chunks from a lane's first to its second
  const int hb1 = CACHE ? min(g.hb, g.dim >> 1) : 1;
  const int c = CACHE ? (int)fwht_src(lane & ((1 << ll) - 1), lane, hb1) : lane & ((1 << ll) - 1);
  const int hslot = (lane >> ll) & ((1 << sl) - 1);
  const int64_t group0 = ((int64_t)wide_block() * kWaves + wave) * (64 >> (ll + sl)), token = group0 + (lane >> (ll + sl));
  if (group0 >= g.tokens) return;  // whole waves
  const Token at = token_of(g, token);
  const bool in = at.in && c < far;

  const Steps steps = wave_steps(g);
  auto tensor = [&](int s) { return s < g.step_end[0] ? 0 : !CACHE || s < g.step_end[1] ? 1 : 2; };
  auto block = [&](int t, int s) { return (s - (t == 0 ? 0 : t == 1 ? g.step_end[0] : g.step_end[1])) << sl; };
  auto rows = [&](int t) -> const HeadRows& { return t == 0 ? g.q : !CACHE || t == 1 ? g.k : g.v; };
  constexpr int kIn = F32 ? 4 : 2;
  const int out_size = g.y_f32 ? 4 : 2;

  struct Pair {
    Chunk<F32> a, b;
  };
  int x_of = -1;  // whose lane base this is
  const char* x_base = nullptr;
  auto load = [&](Pair& raw, int s) {
    if (s >= steps.end) return;
    const int t = tensor(s), h0 = block(t, s);
    const HeadRows& r = rows(t);
    if (t != x_of) {
      x_of = t;
      x_base = static_cast<const char*>(r.x) + (at.batch * r.xb + at.pos * r.xt + hslot * r.xh + c * 8) * kIn;
    }
    if (in && h0 + hslot < r.heads) {
      const char* p = x_base + h0 * r.xh * kIn;
      raw.a.template load<true>(p, 8);
      raw.b.template load<true>(p + far * (8 * kIn), 8);
    }
  };

  Pair raw[kUnroll];  // lanes past a head's end keep zeros
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) raw[u].a.zero(), raw[u].b.zero(), load(raw[u], steps.first + u);

  // angles of the wave's tokens, as above; cs, sn: of the lane's eight pairs
  // (what lies past the rotated ones is not used)
  float cs[8], sn[8];
  bool live = false, live2 = false;
  if (g.half > 0 && steps.first < g.step_end[1]) {
    const Positions pos(g, at);
    const int per = 1 << (ll + sl);
    float2* trig = s_trig[wave] + (lane >> (ll + sl)) * (8 << ll);
    for (int j = lane & (per - 1); j < g.half; j += per) trig[j] = pair_angle(g, pos.p0, pos.p1, pos.p2, j);
    wave_lds_fence();
    const int j0 = g.split ? c * 8 : c * 4, j1 = g.split ? c * 8 + 4 : (c + far) * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = trig[j0 + e], w = trig[j1 + e];
      cs[e] = v.x, sn[e] = v.y;
      cs[4 + e] = w.x, sn[4 + e] = w.y;
    }
    live2 = pos.live && (c + far) * 8 < 2 * g.half;  // interleaved: each chunk is turned or not
    live = pos.live && c * 8 < 2 * g.half;
  }

  float wt[2][8], bs[2][8];
  int w_of = -1, y_of = -1;  // whose weights, whose lane base
  char* y_base = nullptr;
  const int64_t slot = CACHE && in ? g.slots[token] : -1;
  const bool in_cache = slot >= 0 && slot < g.n_slots;
  // the groups of the lane's chunks, and whether the lane is their first
  const bool whole = g.group == g.dim;
  const int group1 = CACHE && !whole ? c * 8 / g.group : 0, group2 = CACHE && !whole ? (c + far) * 8 / g.group : 0;
  const bool heads_group = CACHE && (whole ? c == 0 : group1 * g.group == c * 8);

  auto process = [&](const Pair& raw, int s) {
    const int t = tensor(s), h = block(t, s) + hslot;
    const HeadRows& r = rows(t);
    const bool ok = in && h < r.heads;
    float x[8], y[8];
    raw.a.to_f32(x);
    raw.b.to_f32(y);
    if (g.norm != kHeadNormNone && t != 2) {
      if (w_of != t) {
        w_of = t;
        const int at = c < far ? c * 8 : 0;
        load_weights(r.weight, at, 1.0f, wt[0]);
        load_weights(r.weight, at + far * 8, 1.0f, wt[1]);
        load_weights(r.bias, at, 0.0f, bs[0]);
        load_weights(r.bias, at + far * 8, 0.0f, bs[1]);
      }
      float eps = g.eps;
      auto squares = [&]() {
        if (g.norm == kHeadNormLayer) {
          const float mean = lanes_sum(sum8(x) + sum8(y), ll) * g.inv_dim;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = x[e] - mean;
            y[e] = y[e] - mean;
          }
          const float q = squares8(x) + squares8(y);
          return lanes_sum(c < far ? q : 0.0f, ll);  // lanes past the head hold -mean
        }
        return lanes_sum(squares8(x) + squares8(y), ll);
      };
      float ss = squares();
      const bool holds = squares_hold(ss, eps);
      if (__ballot(!holds) != 0) {
        float keep[2][8], m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) keep[0][e] = x[e], keep[1][e] = y[e];
        raw.a.to_f32(x);
        raw.b.to_f32(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, __builtin_elementwise_maximum(fabsf(x[e]), fabsf(y[e])));
        m = lanes_max(m, ll);
        const int k = norm_exponent(m, eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = ldexpf(x[e], -k), y[e] = ldexpf(y[e], -k);
        const float again = squares();
        if (holds) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = keep[0][e], y[e] = keep[1][e];
        } else {
          ss = again;
          eps = m < __builtin_inff() ? ldexpf(ldexpf(eps, -k), -k) : __builtin_nanf("");
        }
      }
      const float rs = norm_scale(ss, g.inv_dim, eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = fmaf(x[e] * rs, wt[0][e], bs[0][e]);
        y[e] = fmaf(y[e] * rs, wt[1][e], bs[1][e]);
      }
    }
    if (g.half > 0 && t != 2) {
      if (g.split) {
        if (live) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = x[e], b = y[e];
            x[e] = fmaf(-b, sn[e], a * cs[e]);
            y[e] = fmaf(a, sn[e], b * cs[e]);
          }
        }
      } else {
        auto turn = [&](float (&v)[8], int at) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = v[2 * e], b = v[2 * e + 1];
            v[2 * e] = fmaf(-b, sn[at + e], a * cs[at + e]);
            v[2 * e + 1] = fmaf(a, sn[at + e], b * cs[at + e]);
          }
        };
        if (live) turn(x, 0);
        if (live2) turn(y, 4);
      }
    }
    if (CACHE && t != 0) {
      if (g.hb > 1) {
        float sc = fwht8(x, lane, hb1) * g.c_b;
        fwht8(y, lane, hb1);
        if (g.hb != hb1) {  // the last stage, half a head apart
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = x[e], b = y[e];
            x[e] = a + b;
            y[e] = a - b;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // + 0: a difference of 0 has either sign, + 0 is coded
          x[e] = fmaf(x[e], sc, 0.0f);
          y[e] = fmaf(y[e], sc, 0.0f);
        }
      }
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a = __builtin_elementwise_maximum(a, fabsf(x[e]));
        b = __builtin_elementwise_maximum(b, fabsf(y[e]));
      }
      if (whole) a = __builtin_elementwise_maximum(a, b);
      float scale, inv, scale2, inv2;
      code_scales(lanes_max(a, g.group_bits), g.top, scale, inv);
      if (whole)
        scale2 = scale, inv2 = inv;
      else
        code_scales(lanes_max(b, g.group_bits), g.top, scale2, inv2);
      if (ok && in_cache) {
        const int64_t row = slot * r.heads + h;
        store_codes(g.codes[t - 1], row * g.dim + c * 8, x, inv, g.fmt);
        store_codes(g.codes[t - 1], row * g.dim + (c + far) * 8, y, inv2, g.fmt);
        float* to = g.scales[t - 1] + row * g.groups;
        if (heads_group) to[group1] = scale;
        if (heads_group && !whole) to[group2] = scale2;
      }
    } else {
      if (y_of != t) {
        y_of = t;
        y_base = static_cast<char*>(r.y) + (at.batch * r.yb + at.pos * r.yt + hslot * r.yh + c * 8) * out_size;
      }
      if (ok) {
        char* p = y_base + (h - hslot) * r.yh * out_size;
        store_chunk<true>(p, g.y_f32, x, 8);
        store_chunk<true>(p + far * 8 * out_size, g.y_f32, y, 8);
      }
    }
  };

  for (int s = steps.first; s < steps.end; s += kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (s + u < steps.end) {
        process(raw[u], s + u);
        load(raw[u], s + kUnroll + u);
      }
  }
}

template <bool F32, bool CACHE>
void run(const HeadArgs& g, int mode, dim3 grid, hipStream_t s) {
  const dim3 block(64 * kWaves);
  if (mode == kPairs) {
    if (g.dim == 64)
      k_heads16<F32, 2, CACHE><<<grid, block, 0, s>>>(g);
    else if (g.dim == 128)
      k_heads16<F32, 3, CACHE><<<grid, block, 0, s>>>(g);
    else
      k_heads16<F32, -1, CACHE><<<grid, block, 0, s>>>(g);
  } else if (mode == kChunks) {
    k_heads<F32, kChunks, CACHE><<<grid, block, 0, s>>>(g);
  } else if (mode == kVectors) {
    k_heads<F32, kVectors, CACHE><<<grid, block, 0, s>>>(g);
  } else {
    k_heads<F32, kElements, CACHE><<<grid, block, 0, s>>>(g);
  }
}

// The kernel a call takes.
int mode_of(const HeadArgs& g, bool vec, bool cache) {
  if (!vec) return kElements;
  const bool chunks = g.half % (g.split ? 8 : 4) == 0;
  const bool pairs = cache ? cache_pairs(g.dim, g.hb, g.group) : g.dim % 16 == 0;
  if (pairs && chunks && (!g.split || g.half == 0 || 2 * g.half == g.dim)) return kPairs;
  return chunks ? kChunks : kVectors;
}

}  // namespace

hipError_t launch_heads(HeadArgs g, bool f32, bool vec, bool cache, hipStream_t s) {
  const int mode = mode_of(g, vec, cache);
  const HeadPlan p = plan_heads(g.tokens, g.q.heads, g.k.heads, g.v.heads, g.dim, mode == kPairs ? 16 : 8, kHeadWaves);
  g.lane_bits = p.lane_bits;
  g.slot_bits = p.slot_bits;
  g.steps = p.steps;
  g.qk_slices = p.slices[0];
  for (int i = 0; i < 3; ++i) g.step_end[i] = p.step_end[i];
  g.inv_dim = 1.0f / (float)g.dim;
  if (cache) g.group_bits = group_lane_bits(g.dim, g.group, p.lane_bits);
  dim3 grid = wide_grid((p.groups + kWaves - 1) / kWaves);
  grid.z = (unsigned)(p.slices[0] + p.slices[1]);
  if (cache)
    f32 ? run<true, true>(g, mode, grid, s) : run<false, true>(g, mode, grid, s);
  else
    f32 ? run<true, false>(g, mode, grid, s) : run<false, false>(g, mode, grid, s);
  return hipGetLastError();
}

}  // namespace hdq
