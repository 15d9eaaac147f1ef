// kv_cache.hip -- slots of a quantized key-value cache read back (gfx950):
// x = H_b (code * scale) / sqrt(b), the inverse of what heads.hip writes (the
// rotation is its own inverse).  Bound by HBM: the codes and scales read
// once, the elements written once.  17550 tokens of 30 heads of 64 from INT8 to
// bf16 38 us, 5.5 TB/s (the codes partly from the memory-side cache; a copy
// 4.9); 5400 tokens from INT4, rotated back, 13.4 us, 4.0 TB/s, a short launch with the
// rotation's vector instructions beside it.
#include "heads.h"

namespace hdq {

namespace {

constexpr int kWaves = 4;
constexpr int kUnroll = 2;  // head steps whose loads are in flight together

// A chunk of eight codes as loaded.
template <int FMT>
struct Codes {
  uint2 w;
  __device__ __forceinline__ void load(const uint8_t* p) {
    if (FMT == kCacheInt4)
      w.x = *reinterpret_cast<const uint32_t*>(p);
    else
      w = *reinterpret_cast<const uint2*>(p);
  }
  __device__ __forceinline__ void to_f32(float scale, float (&x)[8]) const {
    if (FMT == kCacheFp8) {
      e4m3x4_to_f32(w.x, x);
      e4m3x4_to_f32(w.y, x + 4);
    } else if (FMT == kCacheInt8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (float)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (float)((int)(w.x << (28 - 4 * e)) >> 28);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * scale;
  }
};

__device__ __forceinline__ void store8(void* y, bool f32, int64_t at, const float (&x)[8]) {
  if (f32) {
    float* d = static_cast<float*>(y) + at;
    put16(d, make_float4(x[0], x[1], x[2], x[3]));
    put16(d + 4, make_float4(x[4], x[5], x[6], x[7]));
  } else {
    put16(static_cast<uint16_t*>(y) + at,
          make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
  }
}

// A layer of the grid takes `steps` steps of the keys' heads, or of the
// values'.  A lane holds one chunk of a head, or (PAIRS) chunks c and
// c + dim / 16, as the kernels that write the cache; LL: log2 of a head's
// lanes, or -1 for g.lane_bits.  A Hadamard block of the whole head is a template
// argument: under its conditions the compiler moved the elements between
// registers (5400 tokens from INT4 14.6 -> 13.4 us, of 24 heads of 128 18.5 -> 17.4);
// for blocks of 1 that gained nothing (17550 tokens from INT8 38.7 -> 41).
template <int FMT, int LL, bool PAIRS, int HADAMARD>
__global__ __launch_bounds__(64 * kWaves) void k_cache_read(const CacheReadArgs g) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ll = LL < 0 ? g.lane_bits : LL, sl = g.slot_bits;
  const int far = PAIRS ? g.dim >> 4 : 0;
  const int hb = HADAMARD == kHadamardWhole ? 16 << LL : g.hb;
  const int hb1 = HADAMARD == kHadamardWhole ? hb / 2 : PAIRS ? min(hb, g.dim >> 1) : hb;
  const int c = (int)fwht_src(lane & ((1 << ll) - 1), lane, hb1);
  const int hslot = (lane >> ll) & ((1 << sl) - 1);
  const int64_t group0 = ((int64_t)wide_block() * kWaves + wave) * (64 >> (ll + sl)), token = group0 + (lane >> (ll + sl));
  if (group0 >= g.tokens) return;  // whole waves
  const bool in = token < g.tokens && (PAIRS ? c < far : c * 8 < g.dim);
  const int64_t slot = in ? g.slots[token] : -1;
  const bool cached = slot >= 0 && slot < g.n_slots;
  const int layers = (int)gridDim.z >> 1, z = (int)blockIdx.z, t = z >= layers;
  const int heads = ((g.heads - 1) >> sl) + 1;  // steps of a tensor
  const int step0 = (t ? z - layers : z) * g.steps, step1 = min(step0 + g.steps, heads);

  // the lane's element of head hslot, and its scales, in the cache and in the output
  constexpr int kBits = FMT == kCacheInt4 ? 4 : 8;
  const int64_t row = (cached ? slot : 0) * g.heads + hslot;
  const uint8_t* from = g.codes[t] + (row * g.dim + c * 8) * kBits / 8;
  const float* scale_from = g.scales[t] + row * g.groups;
  const int group1 = c * 8 / g.group, group2 = (c + far) * 8 / g.group;
  const int64_t to = (token * g.heads + hslot) * g.dim + c * 8;
  void* y = g.y[t];

  struct Head {
    Codes<FMT> a, b;
    float scale, scale2;
  };
  auto load = [&](Head& v, int s) {
    if (s >= step1) return;
    const int h0 = s << sl;
    if (cached && h0 + hslot < g.heads) {
      const int64_t at = (int64_t)h0 * g.dim * kBits / 8;
      v.a.load(from + at);
      if (PAIRS) v.b.load(from + at + far * kBits);
      const float* p = scale_from + (int64_t)h0 * g.groups;
      v.scale = p[group1];
      if (PAIRS) v.scale2 = p[group2];
    }
  };
  auto process = [&](const Head& v, int s) {
    float x[8], w[8];
    v.a.to_f32(v.scale, x);
    if (PAIRS) v.b.to_f32(v.scale2, w);
    if (hb > 1) {
      const float sc = fwht8(x, lane, hb1) * g.c_b;
      if (PAIRS) {
        fwht8(w, lane, hb1);
        if (hb != hb1) {  // the last stage, half a head apart
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = x[e], b = w[e];
            x[e] = a + b;
            w[e] = a - b;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = w[e] * sc;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * sc;
    }
    const int h0 = s << sl;
    if (in && h0 + hslot < g.heads) {
      const int64_t at = to + (int64_t)h0 * g.dim;
      store8(y, g.y_f32, at, x);
      if (PAIRS) store8(y, g.y_f32, at + far * 8, w);
    }
  };

  Head raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    raw[u].a.w = raw[u].b.w = make_uint2(0u, 0u);  // slots that are not there read zeros
    raw[u].scale = raw[u].scale2 = 0.0f;
    load(raw[u], step0 + u);
  }
  for (int s = step0; s < step1; s += kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (s + u < step1) {
        process(raw[u], s + u);
        load(raw[u], s + kUnroll + u);
      }
  }
}

template <int FMT, int LL>
void run_dim(const CacheReadArgs& g, dim3 grid, hipStream_t s) {
  const dim3 block(64 * kWaves);
  if (g.hb == g.dim)
    k_cache_read<FMT, LL, true, kHadamardWhole><<<grid, block, 0, s>>>(g);
  else
    k_cache_read<FMT, LL, true, kHadamardAny><<<grid, block, 0, s>>>(g);
}

template <int FMT>
void run(const CacheReadArgs& g, bool pairs, dim3 grid, hipStream_t s) {
  if (!pairs)
    k_cache_read<FMT, -1, false, kHadamardAny><<<grid, dim3(64 * kWaves), 0, s>>>(g);
  else if (g.dim == 64)
    run_dim<FMT, 2>(g, grid, s);
  else if (g.dim == 128)
    run_dim<FMT, 3>(g, grid, s);
  else
    k_cache_read<FMT, -1, true, kHadamardAny><<<grid, dim3(64 * kWaves), 0, s>>>(g);
}

}  // namespace

hipError_t launch_cache_read(CacheReadArgs g, hipStream_t s) {
  const bool pairs = cache_pairs(g.dim, g.hb, g.group);
  // keys and values by waves of their own: the plan of one of them
  const HeadPlan p = plan_heads(2 * g.tokens, g.heads, 0, 0, g.dim, pairs ? 16 : 8, kReadWaves);
  g.lane_bits = p.lane_bits;
  g.slot_bits = p.slot_bits;
  g.steps = p.steps;
  const int64_t per_wave = int64_t(1) << (6 - p.lane_bits - p.slot_bits);
  const int64_t groups = (g.tokens + per_wave - 1) / per_wave;
  dim3 grid = wide_grid((groups + kWaves - 1) / kWaves);
  grid.z = (unsigned)(2 * p.slices[0]);
  if (g.fmt == kCacheFp8)
    run<kCacheFp8>(g, pairs, grid, s);
  else if (g.fmt == kCacheInt8)
    run<kCacheInt8>(g, pairs, grid, s);
  else
    run<kCacheInt4>(g, pairs, grid, s);
  return hipGetLastError();
}

}  // namespace hdq
