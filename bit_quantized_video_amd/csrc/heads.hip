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
constexpr int kUnroll = 4;       // head steps whose loads are in flight together
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

// A head's scale 1 / sqrt(mean square + eps) and its centred values in place.
// Sums outside what float32 squares hold (and NaN, infinities) are taken
// again from values scaled by a power of two, which cancels in the result;
// a head with a NaN or an infinity becomes NaN.
__device__ __forceinline__ float head_norm(float (&x)[8], int n, bool layer, float inv_dim, float eps, int ll) {
  float raw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) raw[e] = x[e];
  float scaled_eps = eps, ss = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    if (layer) {
      float s = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
      const float mean = lanes_sum(s, ll) * inv_dim;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < n ? x[e] - mean : 0.0f;
    }
    float a = x[0] * x[0], b = x[1] * x[1];
#pragma unroll
    for (int e = 2; e < 8; e += 2) {
      a = fmaf(x[e], x[e], a);
      b = fmaf(x[e + 1], x[e + 1], b);
    }
    ss = lanes_sum(a + b, ll);
    const bool ok = ss < 0x1p100f && (ss > 0x1p-80f || eps > 0x1p-60f);
    if (pass == 1 || __ballot(!ok) == 0) break;
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, fabsf(raw[e]));
    m = lanes_max(m, ll);
    int k = 0;
    if (m > 0.0f && m < __builtin_inff()) k = ilogbf(fmaxf(m, sqrtf(eps))) + 1;
    if (ok) k = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = ldexpf(raw[e], -k);
    scaled_eps = ldexpf(ldexpf(eps, -k), -k);
    if (!(m < __builtin_inff())) scaled_eps = __builtin_nanf("");
  }
  const float d = ss * inv_dim + scaled_eps;
  return d == 0.0f ? 0.0f : rsqrtf(d);  // a head of zeros stays zero at eps 0
}

template <bool F32, bool VEC, bool CACHE>
__global__ __launch_bounds__(64 * kWaves) void k_heads(const HeadArgs g) {
  __shared__ float2 s_trig[kWaves][kMaxPairs];
  __shared__ __align__(16) float s_swap[kWaves][64 * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // 32 bits hold the wave's number: one token a wave at most, and slices only with few tokens
  const uint32_t work = wide_block() * kWaves + wave;
  const uint32_t tgroup = work / (uint32_t)g.slices;
  const int slice = (int)(work - tgroup * (uint32_t)g.slices);
  const int ll = g.lane_bits, sl = g.slot_bits;
  // lane l of a head holds chunk c (in an order that the Hadamard stages like)
  const int c = CACHE ? (int)fwht_src(lane & ((1 << ll) - 1), lane, g.hb) : lane & ((1 << ll) - 1);
  const int hslot = (lane >> ll) & ((1 << sl) - 1);
  const int64_t first = (int64_t)tgroup * (64 >> (ll + sl)), token = first + (lane >> (ll + sl));
  if (first >= g.tokens) return;  // whole waves
  const bool in_token = token < g.tokens;
  const uint32_t tok = in_token ? (uint32_t)token : 0u, bi = tok / (uint32_t)g.length, ti = tok - bi * (uint32_t)g.length;
  const int n = min(8, g.dim - c * 8);  // the lane's elements, <= 0 past the head
  const bool in_head = n > 0;

  // angles of the wave's tokens: pair j of a token by lane j, j + lanes, ... of it
  float cs[8], sn[8];
  bool live = false;
  if (g.half > 0) {
    const int64_t* pp = g.positions + bi * g.pos_batch + ti * g.pos_token;
    int64_t pos[3];
    live = true;
#pragma unroll
    for (int a = 0; a < 3; ++a) {
      pos[a] = a < g.axes ? pp[a * g.pos_axis] : 0;
      live = live && pos[a] >= 0;
    }
    const int per = 1 << (ll + sl);
    float2* trig = s_trig[wave] + (lane >> (ll + sl)) * g.half;
    for (int j = lane & (per - 1); j < g.half; j += per) {
      const double p = (double)(j < g.axis_end[0] ? pos[0] : j < g.axis_end[1] ? pos[1] : pos[2]);
      const double f = g.turns[j];
      const double t = p * f, lost = fma(p, f, -t);  // the product in two parts
      const float r = (float)((t - rint(t)) + lost);
      float s, co;
      sincospif(2.0f * r, &s, &co);
      trig[j] = make_float2(co * g.scale, s * g.scale);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = c * 8 + e;
      const int j = g.split ? (i < g.half ? i : i - g.half) : (c * 4 + (e >> 1));
      const float2 v = j < g.half ? trig[j] : make_float2(1.0f, 0.0f);
      cs[e] = v.x;
      // y[i] = x[i] cos + x[partner] sin, the sine negative for a pair's first element
      sn[e] = (g.split ? i < g.half : (e & 1) == 0) ? -v.y : v.y;
    }
  }

  // head h of the call is head h - start of one of its tensors
  constexpr int kIn = F32 ? 4 : 2;
  const int out_size = g.y_f32 ? 4 : 2;
  const char* qx = static_cast<const char*>(g.q.x) + (bi * g.q.xb + ti * g.q.xt + c * 8) * kIn;
  const char* kx = static_cast<const char*>(g.k.x) + (bi * g.k.xb + ti * g.k.xt + c * 8) * kIn;
  const char* vx = CACHE ? static_cast<const char*>(g.v.x) + (bi * g.v.xb + ti * g.v.xt + c * 8) * kIn : nullptr;
  char* qy = static_cast<char*>(g.q.y) + (bi * g.q.yb + ti * g.q.yt + c * 8) * out_size;
  char* ky = CACHE ? nullptr : static_cast<char*>(g.k.y) + (bi * g.k.yb + ti * g.k.yt + c * 8) * out_size;
  const int heads = g.heads[2];
  auto tensor = [&](int h) { return h < g.heads[0] ? 0 : !CACHE || h < g.heads[1] ? 1 : 2; };
  auto start = [&](int t) { return t == 0 ? 0 : !CACHE || t == 1 ? g.heads[0] : g.heads[1]; };

  float wt[8], bs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) wt[e] = 1.0f, bs[e] = 0.0f;
  int loaded = -1;  // whose weights these are
  const int64_t slot = CACHE && in_token ? g.slots[tok] : -1;
  const bool in_cache = slot >= 0 && slot < g.n_slots;

  for (int i0 = 0; i0 < g.steps; i0 += kUnroll) {
    Chunk<F32> raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = (slice * g.steps + i0 + u) << sl | hslot;
      raw[u].zero();
      if (i0 + u < g.steps && h < heads && in_token && in_head) {
        const int t = tensor(h);
        const int64_t xh = t == 0 ? g.q.xh : !CACHE || t == 1 ? g.k.xh : g.v.xh;
        raw[u].template load<VEC>((t == 0 ? qx : !CACHE || t == 1 ? kx : vx) + (h - start(t)) * xh * kIn, n);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (i0 + u >= g.steps) break;
      const int h = (slice * g.steps + i0 + u) << sl | hslot;
      const bool ok = h < heads && in_token && in_head;
      const int t = tensor(h);
      float x[8];
      raw[u].to_f32(x);
      const bool plain = t == 2;  // values: neither norm nor rotation
      if (g.norm != 0 && __ballot(!plain) != 0) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e];
        const float r = head_norm(y, n, g.norm == 1, g.inv_dim, g.eps, ll);
        if (!plain && loaded != t && in_head) {
          loaded = t;
          const float* w = t == 0 ? g.q.weight : g.k.weight;
          const float* b = t == 0 ? g.q.bias : g.k.bias;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            wt[e] = w != nullptr && e < n ? w[c * 8 + e] : 1.0f;
            bs[e] = b != nullptr && e < n ? b[c * 8 + e] : 0.0f;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = plain ? x[e] : fmaf(y[e] * r, wt[e], bs[e]);
      }
      if (g.half > 0) {
        float p[8];
        if (g.split) {
          float* sw = s_swap[wave] + (lane >> ll << ll) * 8;
#pragma unroll
          for (int e = 0; e < 8; ++e) sw[c * 8 + e] = x[e];
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
          __builtin_amdgcn_wave_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
          if (g.half % 4 == 0) {
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
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
          __builtin_amdgcn_wave_barrier();
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = x[e ^ 1];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool turn = live && !plain && (g.split ? c * 8 + e < 2 * g.half : c * 4 + (e >> 1) < g.half);
          x[e] = turn ? fmaf(p[e], sn[e], x[e] * cs[e]) : x[e];
        }
      }
      if (CACHE) {
        const bool coded = t != 0;
        if (__ballot(coded) != 0) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e];
          const float sc = fwht8(y, lane, g.hb) * g.c_b;
          float a = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = g.hb > 1 ? fmaf(y[e], sc, 0.0f) : y[e];  // a difference of 0 has either sign: + 0 is coded
            a = __builtin_elementwise_maximum(a, fabsf(y[e]));
          }
          float scale, inv;
          code_scales(lanes_max(a, g.group_bits), g.top, scale, inv);
          if (coded && ok && in_cache) {
            const int64_t row = slot * (heads - g.heads[1]) + (h - start(t));
            store_codes(t == 1 ? g.codes[0] : g.codes[1], row * g.dim + c * 8, y, inv, g.fmt);
            if ((c * 8) % g.group == 0) (t == 1 ? g.scales[0] : g.scales[1])[row * g.groups + c * 8 / g.group] = scale;
          }
        }
        if (coded) continue;
      }
      if (ok) {
        char* y = t == 0 ? qy : ky;
        store_chunk<VEC>(y + (h - start(t)) * (t == 0 ? g.q.yh : g.k.yh) * out_size, g.y_f32, x, n);
      }
    }
  }
}

}  // namespace

hipError_t launch_heads(HeadArgs g, bool f32, bool vec, bool cache, hipStream_t s) {
  const HeadPlan p = plan_heads(g.tokens, g.heads[2], g.dim);
  g.lane_bits = p.lane_bits;
  g.slot_bits = p.slot_bits;
  g.steps = p.steps;
  g.slices = p.slices;
  g.inv_dim = 1.0f / (float)g.dim;
  const dim3 grid = wide_grid((p.waves + kWaves - 1) / kWaves), block(64 * kWaves);
  if (cache) {
    if (f32)
      vec ? k_heads<true, true, true><<<grid, block, 0, s>>>(g) : k_heads<true, false, true><<<grid, block, 0, s>>>(g);
    else
      vec ? k_heads<false, true, true><<<grid, block, 0, s>>>(g) : k_heads<false, false, true><<<grid, block, 0, s>>>(g);
  } else {
    if (f32)
      vec ? k_heads<true, true, false><<<grid, block, 0, s>>>(g) : k_heads<true, false, false><<<grid, block, 0, s>>>(g);
    else
      vec ? k_heads<false, true, false><<<grid, block, 0, s>>>(g) : k_heads<false, false, false><<<grid, block, 0, s>>>(g);
  }
  return hipGetLastError();
}

}  // namespace hdq
