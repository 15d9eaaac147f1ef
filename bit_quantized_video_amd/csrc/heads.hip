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
// Bound by HBM: every element is read and written once.  Queries and keys of
// 17776 tokens, 60 heads of 64, layer norm and rotation: 62 us, 4.4 TB/s (a copy
// 4.9); rotation of 30 of them 27 us, 5.0 TB/s (part from the memory-side cache);
// 4050 tokens of 90 heads, queries written back, keys and values to FP8 in
// blocks of 64: 20 us, 3.9 TB/s (a short launch: two rounds of waves, each
// beginning with positions, angles and loads, a thousand vector instructions
// each).  One token: 4 us, a chain of latencies (arguments, positions, angles,
// norm) of which an empty launch is 1.5.
//
// Two forms: k_heads16 (heads16.h), 16 elements a lane, for heads of a multiple
// of 16 in whole vectors, and k_heads here, 8 elements a lane, for the rest.
// With one form of 8 elements the largest calls took 86 us (62) and 49 (32 then, 20 now):
// a step's addresses, lane sums and tests served half as many elements.  What is left to
// k_heads: the rotation of 32 of 64 elements in halves, 17776 tokens of 30 heads, 28 us (a copy
// 28); norm and rotation of 52 heads of 72 115 us, of 40 heads of 96 on 16 elements 72;
// 4050 tokens into the cache, 72 heads of 80 in blocks of 16 41 us, 60 of 96 in blocks of 32 36.
// Rounding: everything is float32 until the output's type or the code; angles are
// float64 up to the fraction of a turn.
#include "heads_device.h"

namespace hdq {

namespace {

// What a chunk's elements allow: element loads and any rotation; vector loads;
// and also a rotation whose pairs are whole chunks (k_heads), or whole heads
// on 16 elements a lane (heads16.h).
enum Mode : int { kElements = 0, kVectors = 1, kChunks = 2, kPairs = 3 };

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
      if (n <= 0) a = 0.0f;  // lanes past the head hold biases
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

template <bool F32, bool CACHE>
void run(const HeadArgs& g, int mode, dim3 grid, hipStream_t s) {
  const dim3 block(64 * kWaves);
  if (mode == kChunks)
    k_heads<F32, kChunks, CACHE><<<grid, block, 0, s>>>(g);
  else if (mode == kVectors)
    k_heads<F32, kVectors, CACHE><<<grid, block, 0, s>>>(g);
  else
    k_heads<F32, kElements, CACHE><<<grid, block, 0, s>>>(g);
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
  if (mode == kPairs)
    f32 ? run_heads16_f32(g, cache, grid, s)
    : !cache ? run_heads16(g, grid, s)
    : g.dim == 64 ? run_heads16_cache64(g, grid, s)
    : g.dim == 128 ? run_heads16_cache128(g, grid, s)
                   : run_heads16_cache(g, grid, s);
  else if (cache)
    f32 ? run<true, true>(g, mode, grid, s) : run<false, true>(g, mode, grid, s);
  else
    f32 ? run<true, false>(g, mode, grid, s) : run<false, false>(g, mode, grid, s);
  return hipGetLastError();
}

}  // namespace hdq
