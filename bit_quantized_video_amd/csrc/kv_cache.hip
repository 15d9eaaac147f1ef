// kv_cache.hip -- slots of a quantized key-value cache read back (gfx950):
// x = H_b (code * scale) / sqrt(b), the inverse of what heads.hip writes (the
// rotation is its own inverse).  Bound by HBM: the codes and scales read
// once, the elements written once.
#include "heads.h"

namespace hdq {

namespace {

constexpr int kWaves = 4;
constexpr int kUnroll = 4;  // head steps whose loads are in flight together

struct Coded {
  uint2 w;
  float scale;
};

__device__ __forceinline__ void decode8(const Coded& v, int fmt, float (&x)[8]) {
  if (fmt == kCacheFp8) {
    e4m3x4_to_f32(v.w.x, x);
    e4m3x4_to_f32(v.w.y, x + 4);
  } else if (fmt == kCacheInt8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)(int8_t)((e < 4 ? v.w.x : v.w.y) >> (8 * (e & 3)));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)((int)(v.w.x << (28 - 4 * e)) >> 28);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = x[e] * v.scale;
}

__global__ __launch_bounds__(64 * kWaves) void k_cache_read(const CacheReadArgs g) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t work = wide_block() * kWaves + wave;
  const uint32_t tgroup = work / (uint32_t)g.slices;
  const int slice = (int)(work - tgroup * (uint32_t)g.slices);
  const int ll = g.lane_bits, sl = g.slot_bits;
  const int c = (int)fwht_src(lane & ((1 << ll) - 1), lane, g.hb);
  const int hslot = (lane >> ll) & ((1 << sl) - 1);
  const int64_t first = (int64_t)tgroup * (64 >> (ll + sl)), token = first + (lane >> (ll + sl));
  if (first >= g.tokens) return;  // whole waves
  const bool in = token < g.tokens && c * 8 < g.dim;
  const int64_t slot = in ? g.slots[token] : -1;
  const bool cached = slot >= 0 && slot < g.n_slots;
  // the lane's element of head hslot, and its scale, in the cache and in the output
  const int64_t row = (cached ? slot : 0) * g.heads + hslot;
  const int64_t from = row * g.dim + c * 8, scale_from = row * g.groups + c * 8 / g.group;
  const int64_t to = (token * g.heads + hslot) * g.dim + c * 8;
  const int step0 = slice * g.steps, step1 = min(step0 + g.steps, g.step_end[2]);

  auto load = [&](Coded& v, int s) {
    v = Coded{make_uint2(0u, 0u), 0.0f};  // slots that are not there read zeros
    if (s >= step1) return;
    const int t = s < g.step_end[0] ? 0 : 1, h0 = (s - (t ? g.step_end[0] : 0)) << sl;
    if (cached && h0 + hslot < g.heads) {
      const int64_t at = from + (int64_t)h0 * g.dim;
      if (g.fmt == kCacheInt4)
        v.w.x = *reinterpret_cast<const uint32_t*>(g.codes[t] + at / 2);
      else
        v.w = *reinterpret_cast<const uint2*>(g.codes[t] + at);
      v.scale = g.scales[t][scale_from + (int64_t)h0 * g.groups];
    }
  };
  auto process = [&](const Coded& v, int s) {
    const int t = s < g.step_end[0] ? 0 : 1, h0 = (s - (t ? g.step_end[0] : 0)) << sl;
    float x[8];
    decode8(v, g.fmt, x);
    const float sc = fwht8(x, lane, g.hb) * g.c_b;
    if (g.hb > 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * sc;
    }
    if (in && h0 + hslot < g.heads) {
      const int64_t at = to + (int64_t)h0 * g.dim;
      if (g.y_f32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(g.y[t]) + at);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.y[t]) + at) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      }
    }
  };

  Coded raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) load(raw[u], step0 + u);
  for (int s = step0; s < step1; s += kUnroll) {
    Coded now[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) now[u] = raw[u];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load(raw[u], s + kUnroll + u);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (s + u < step1) process(now[u], s + u);
  }
}

}  // namespace

hipError_t launch_cache_read(CacheReadArgs g, hipStream_t s) {
  const HeadPlan p = plan_heads(g.tokens, g.heads, g.heads, 0, g.dim);
  g.lane_bits = p.lane_bits;
  g.slot_bits = p.slot_bits;
  g.steps = p.steps;
  g.slices = p.slices;
  for (int i = 0; i < 3; ++i) g.step_end[i] = p.step_end[i];
  k_cache_read<<<wide_grid((p.waves + kWaves - 1) / kWaves), dim3(64 * kWaves), 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace hdq
