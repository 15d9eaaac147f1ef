// heads16.h -- heads of 16 elements a lane: the form most calls take.
//
// A lane holds chunks c and c + dim / 16 of a head, so both elements of a pair,
// in either layout, are its own, and a step's addresses, reductions and tests
// serve twice the elements.  Norm, rotation and the cache's blocks and groups
// are the kernel's template arguments and the values' waves a path of their own,
// so that a step is straight code: under conditions the compiler moved every
// element between registers (4050 tokens of 90 heads into the cache 32 -> 26 us
// without those of norm and rotation, 23 of the blocks, 20 of the groups).  Conditions: dim a multiple of 16, vectors throughout, the
// rotation none, interleaved in whole chunks or split over the whole head, a
// Hadamard block and a group within half a head or the whole.
//
// Not kept: fewer registers for more waves (weights loaded again for each step:
// 4050 tokens 22.6 -> 22.2 us, 17776 62 -> 68); one, three or four steps' loads in
// flight (no gain); stores past the caches (reading back 38.6 -> 42.7).
#pragma once

#include <type_traits>

#include "heads_device.h"

namespace hdq {

enum Rotation : int { kRotateNone = 0, kRotateSplit = 1, kRotatePairs = 2 };

namespace {

// LL: log2 of a head's lanes, or -1 for g.lane_bits.
template <bool F32, int LL, bool CACHE, bool NORM, int ROTATE, int HADAMARD, int GROUP>
__global__ __launch_bounds__(64 * kWaves) void k_heads16(const HeadArgs g) {
  __shared__ __align__(16) float2 s_trig[kWaves][ROTATE != kRotateNone ? 2 * kMaxPairs : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ll = LL < 0 ? g.lane_bits : LL, sl = g.slot_bits;
  // Chunks from a lane's first to its second.  A constant where it can be: a register less, and
  // with more than 128 a SIMD holds three waves for four (4050 tokens in blocks of 32 24.2 -> 21.3 us).
  const int far = LL < 0 ? g.dim >> 4 : 1 << LL;
  const int hb = HADAMARD == kHadamardNone ? 1 : HADAMARD == kHadamardWhole ? 16 << LL : g.hb;
  const int hb1 = HADAMARD == kHadamardWhole ? hb / 2 : HADAMARD == kHadamardNone ? 1 : min(hb, g.dim >> 1);
  const int c = CACHE ? (int)fwht_src(lane & ((1 << ll) - 1), lane, hb1) : lane & ((1 << ll) - 1);
  const int hslot = (lane >> ll) & ((1 << sl) - 1);
  const int64_t group0 = ((int64_t)wide_block() * kWaves + wave) * (64 >> (ll + sl)), token = group0 + (lane >> (ll + sl));
  if (group0 >= g.tokens) return;  // whole waves
  const Token at = token_of(g, token);
  const bool in = at.in && c < far;
  const Steps steps = wave_steps(g);
  constexpr int kIn = F32 ? 4 : 2;
  const int out_size = g.y_f32 ? 4 : 2;

  // cache: the token's slot, the groups of the lane's chunks, and whether the lane is their first
  const int64_t slot = CACHE && in ? g.slots[token] : -1;
  const bool in_cache = slot >= 0 && slot < g.n_slots;
  const bool whole = GROUP == kGroupAny ? g.group == g.dim : GROUP == kGroupHead;
  const int group1 = CACHE && !whole ? c * 8 / g.group : 0, group2 = CACHE && !whole ? (c + far) * 8 / g.group : 0;
  const bool heads_group = CACHE && (whole ? c == 0 : group1 * g.group == c * 8);

  struct Pair {
    Chunk<F32> a, b;
  };

  // A wave of the queries' and keys' steps, or (VALUES) of the values'.
  auto walk = [&](auto values) {
    constexpr bool VALUES = decltype(values)::value;
    auto tensor = [&](int s) { return VALUES ? 2 : s < g.step_end[0] ? 0 : 1; };
    auto block = [&](int t, int s) { return (s - (t == 0 ? 0 : t == 1 ? g.step_end[0] : g.step_end[1])) << sl; };
    auto rows = [&](int t) -> const HeadRows& { return VALUES ? g.v : t == 0 ? g.q : g.k; };

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

    // angles of the wave's tokens: pair j of a token by lane j, j + lanes, ... of it;
    // cs, sn: of the lane's eight pairs (what lies past the rotated ones is not used)
    float cs[8], sn[8];
    bool live = true, live2 = true, all_live = true;
    if (!VALUES && ROTATE != kRotateNone) {
      const Positions pos(g, at);
      const int per = 1 << (ll + sl);
      float2* trig = s_trig[wave] + (lane >> (ll + sl)) * (8 << ll);
      for (int j = lane & (per - 1); j < g.half; j += per) trig[j] = pair_angle(g, pos.p0, pos.p1, pos.p2, j);
      wave_lds_fence();
      const int j0 = ROTATE == kRotateSplit ? c * 8 : c * 4, j1 = ROTATE == kRotateSplit ? c * 8 + 4 : (c + far) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = trig[j0 + e], w = trig[j1 + e];
        cs[e] = v.x, sn[e] = v.y;
        cs[4 + e] = w.x, sn[4 + e] = w.y;
      }
      live = pos.live && c * 8 < 2 * g.half;  // interleaved: each chunk is turned or not
      live2 = pos.live && (ROTATE == kRotateSplit || (c + far) * 8 < 2 * g.half);
      all_live = __ballot(in && !(live && live2)) == 0;
    }

    float wt[2][8], bs[2][8];
    int w_of = -1, y_of = -1;  // whose weights, whose lane base
    char* y_base = nullptr;

    auto process = [&](const Pair& raw, int s) {
      const int t = tensor(s), h = block(t, s) + hslot;
      const HeadRows& r = rows(t);
      const bool ok = in && h < r.heads;
      float x[8], y[8];
      raw.a.to_f32(x);
      raw.b.to_f32(y);
      if (!VALUES && NORM) {
        if (w_of != t) {
          w_of = t;
          const int first = c < far ? c * 8 : 0;
          load_weights(r.weight, first, 1.0f, wt[0]);
          load_weights(r.weight, first + far * 8, 1.0f, wt[1]);
          load_weights(r.bias, first, 0.0f, bs[0]);
          load_weights(r.bias, first + far * 8, 0.0f, bs[1]);
        }
        const bool layer = g.norm == kHeadNormLayer;
        auto less = [&](float v) {  // not in lanes past the head
          if (LL < 0 && c >= far) v = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = x[e] - v;
            y[e] = y[e] - v;
          }
        };
        auto average = [&]() { return lanes_sum(sum8(x) + sum8(y), ll) * g.inv_dim; };
        float eps = g.eps, mean = 0.0f;
        if (layer) mean = average(), less(mean);
        float ss = lanes_sum(squares8(x) + squares8(y), ll);
        const bool holds = squares_hold(ss, mean, g.inv_dim, eps);
        // As head_norm; once more the same where the sum holds.  17776 tokens of 60 heads, unrotated,
        // 52 us, and 57 where all are 3 deviations off.
        if (__ballot(!holds) != 0) {
          float m = 0.0f;
          auto scaled = [&](int k) {
            raw.a.to_f32(x);
            raw.b.to_f32(y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = ldexpf(x[e], -k), y[e] = ldexpf(y[e], -k);
          };
          scaled(0);
#pragma unroll
          for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, __builtin_elementwise_maximum(fabsf(x[e]), fabsf(y[e])));
          m = lanes_max(m, ll);
          const int k = holds ? 0 : norm_exponent(m, eps);
          eps = m < __builtin_inff() ? ldexpf(ldexpf(eps, -k), -k) : __builtin_nanf("");
          scaled(k);
          if (layer) {
            const float first = holds ? 0.0f : lanes_first(x[0], ll);
            less(first);
            mean = first + average();
            scaled(k);
            less(mean);
            mean = average();
            less(holds ? 0.0f : mean);
          }
          ss = lanes_sum(squares8(x) + squares8(y), ll);
        }
        const float rs = norm_scale(ss, g.inv_dim, eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = fmaf(x[e] * rs, wt[0][e], bs[0][e]);
          y[e] = fmaf(y[e] * rs, wt[1][e], bs[1][e]);
        }
      }
      if (!VALUES && ROTATE != kRotateNone) {
        float a[8], b[8];
        if (ROTATE == kRotateSplit) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            a[e] = fmaf(-y[e], sn[e], x[e] * cs[e]);
            b[e] = fmaf(x[e], sn[e], y[e] * cs[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[2 * e] = fmaf(-x[2 * e + 1], sn[e], x[2 * e] * cs[e]);
            a[2 * e + 1] = fmaf(x[2 * e], sn[e], x[2 * e + 1] * cs[e]);
            b[2 * e] = fmaf(-y[2 * e + 1], sn[4 + e], y[2 * e] * cs[4 + e]);
            b[2 * e + 1] = fmaf(y[2 * e], sn[4 + e], y[2 * e + 1] * cs[4 + e]);
          }
        }
        if (!all_live) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            a[e] = live ? a[e] : x[e];
            b[e] = live2 ? b[e] : y[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = a[e], y[e] = b[e];
      }
      if (CACHE && (VALUES || t != 0)) {
        if (hb > 1) {
          const float sc = fwht8(x, lane, hb1) * g.c_b;
          fwht8(y, lane, hb1);
          if (hb != hb1) {  // the last stage, half a head apart
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
        if (LL < 0 && c >= far) a = 0.0f;  // lanes past the head hold biases, turned by any angle
        float scale, inv;
        code_scales(lanes_max(a, g.group_bits), g.top, scale, inv);
        float scale2 = scale, inv2 = inv;
        if (!whole) code_scales(lanes_max(b, g.group_bits), g.top, scale2, inv2);
        if (ok && in_cache) {
          const int64_t row = slot * r.heads + h;
          uint8_t* codes = VALUES ? g.codes[1] : g.codes[0];
          float* to = (VALUES ? g.scales[1] : g.scales[0]) + row * g.groups;
          store_codes2(codes, row * g.dim + c * 8, far * 8, x, y, inv, inv2, g.fmt);
          if (heads_group) {
            to[group1] = scale;
            if (!whole) to[group2] = scale2;
          }
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
  };
  if (CACHE && steps.first >= g.step_end[1])
    walk(std::true_type());
  else
    walk(std::false_type());
}

template <bool F32, int LL, bool CACHE, bool NORM, int HADAMARD, int GROUP>
void run16_rotate(const HeadArgs& g, int rotate, dim3 grid, hipStream_t s) {
  const dim3 block(64 * kWaves);
  if (rotate == kRotateNone)
    k_heads16<F32, LL, CACHE, NORM, kRotateNone, HADAMARD, GROUP><<<grid, block, 0, s>>>(g);
  else if (rotate == kRotateSplit)
    k_heads16<F32, LL, CACHE, NORM, kRotateSplit, HADAMARD, GROUP><<<grid, block, 0, s>>>(g);
  else
    k_heads16<F32, LL, CACHE, NORM, kRotatePairs, HADAMARD, GROUP><<<grid, block, 0, s>>>(g);
}

template <bool F32, int LL, bool CACHE, int HADAMARD, int GROUP>
void run16_norm(const HeadArgs& g, dim3 grid, hipStream_t s) {
  const int rotate = g.half == 0 ? kRotateNone : g.split ? kRotateSplit : kRotatePairs;
  if (g.norm != kHeadNormNone)
    run16_rotate<F32, LL, CACHE, true, HADAMARD, GROUP>(g, rotate, grid, s);
  else
    run16_rotate<F32, LL, CACHE, false, HADAMARD, GROUP>(g, rotate, grid, s);
}

template <bool F32, int LL, bool CACHE, int HADAMARD>
void run16_group(const HeadArgs& g, dim3 grid, hipStream_t s) {
  if (g.group == g.dim)
    run16_norm<F32, LL, CACHE, HADAMARD, kGroupHead>(g, grid, s);
  else
    run16_norm<F32, LL, CACHE, HADAMARD, kGroupPart>(g, grid, s);
}

template <bool F32, int LL, bool CACHE>
void run16(const HeadArgs& g, dim3 grid, hipStream_t s) {
  if constexpr (!CACHE)
    run16_norm<F32, LL, CACHE, kHadamardNone, kGroupHead>(g, grid, s);
  else if constexpr (LL < 0)
    run16_norm<F32, LL, CACHE, kHadamardAny, kGroupAny>(g, grid, s);
  else if (g.hb == 1)
    run16_group<F32, LL, CACHE, kHadamardNone>(g, grid, s);
  else if (g.hb == g.dim)
    run16_group<F32, LL, CACHE, kHadamardWhole>(g, grid, s);
  else
    run16_group<F32, LL, CACHE, kHadamardAny>(g, grid, s);
}

}  // namespace

}  // namespace hdq
