// w4.hip -- linear layer of few tokens with 4-bit weights in groups (gfx950).
//
//   y[m, n] = sum over groups g of s[n, g] sum_{k in g} (u[n, k] - z[n, g]) x[m, k],
// u the codes 0 .. 15, z the group's zero point (8 without).  Bound by HBM: half
// a byte a weight, each read once.  The matrix instruction takes 16 rows x 32
// columns of weights and 32 columns of 16 tokens at a time; fewer tokens leave
// its other columns unused, at no cost beside the loads.  A code becomes bf16
// in one operation a pair: nibble u in bits 6..3 of a bf16 16.0 is 16 + u,
// exact, so the product is sum (16 + u) x - (16 + z) sum x, and sum x comes from a
// second product with ones.  Sums are float32: the difference costs at most
// (31 + 31) / 8 times a float32 sum's rounding.
#include "hdq_device.h"
#include "hdq_internal.h"
#include "w4.h"

namespace hdq {

namespace {

struct W4Args {
  const uint16_t* x;  // bf16 [M, K]
  const uint8_t* codes;
  const uint16_t* scale;
  const uint8_t* zero;
  void* y;
  int64_t M, N, K;
  int64_t tiles_n, tiles_k;
  int wn, wk;
};

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));

// Codes to bf16 16 + u: eight columns of a word.
__device__ __forceinline__ v8bf decode(uint32_t w) {
  v4u r;
  r.x = ((w << 3) & 0x00780078u) | 0x41804180u;
  r.y = ((w >> 1) & 0x00780078u) | 0x41804180u;
  r.z = ((w >> 5) & 0x00780078u) | 0x41804180u;
  r.w = ((w >> 9) & 0x00780078u) | 0x41804180u;
  return __builtin_bit_cast(v8bf, r);
}

// One tile's operands as loaded: NT x 16 rows, MT x 16 tokens, 128 columns.
template <int MT, int NT, int GROUPS, bool ZERO>
struct Tile {
  v4u codes[NT];
  v4u x[MT][4];
  v2u scale[NT][GROUPS];
  uint32_t zero[ZERO ? NT : 1][GROUPS];
};

template <int MT, int NT, int GROUPS, bool ZERO, bool F32>
__global__ __launch_bounds__(1024) void k_w4(const W4Args g) {
  extern __shared__ float s_sum[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wn = wave / g.wk, wk = wave - wn * g.wk;
  const int col = lane & 15, quad = lane >> 4;
  const int64_t tn0 = ((int64_t)blockIdx.x * g.wn + wn) * NT;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const int tiles_k = (int)g.tiles_k;
  typedef Tile<MT, NT, GROUPS, ZERO> T;

  const uint8_t* codes[NT];
  const uint16_t* scale[NT];
  const uint8_t* zero[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t tile = (tn0 + i < g.tiles_n ? tn0 + i : g.tiles_n - 1) * tiles_k;  // a row tile past the end repeats the last
    codes[i] = g.codes + tile * 1024 + lane * 16;
    scale[i] = g.scale + tile * (16 * GROUPS) + quad * (4 * GROUPS);
    zero[i] = ZERO ? g.zero + tile * (16 * GROUPS) + quad * (4 * GROUPS) : nullptr;
  }
  const uint16_t* xr[MT];
  bool token[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    token[m] = m0 + m * 16 + col < g.M;
    xr[m] = g.x + (token[m] ? m0 + m * 16 + col : 0) * g.K + quad * 8;
  }

  auto load = [&](T& t, int kt) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      t.codes[i] = *reinterpret_cast<const v4u*>(codes[i] + (int64_t)kt * 1024);
#pragma unroll
      for (int q = 0; q < GROUPS; ++q) {
        t.scale[i][q] = *reinterpret_cast<const v2u*>(scale[i] + (int64_t)kt * (16 * GROUPS) + 4 * q);
        if (ZERO) t.zero[i][q] = *reinterpret_cast<const uint32_t*>(zero[i] + (int64_t)kt * (16 * GROUPS) + 4 * q);
      }
    }
    const int left = (int)(g.K - (int64_t)kt * 128) - quad * 8;  // columns from the lane's first on
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        t.x[m][s] = v4u{0u, 0u, 0u, 0u};
        if (token[m] && 32 * s < left) t.x[m][s] = *reinterpret_cast<const v4u*>(xr[m] + (int64_t)kt * 128 + 32 * s);
      }
  };

  v4f y[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) y[i][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const v8bf ones = __builtin_bit_cast(v8bf, v4u{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});

  auto multiply = [&](const T& t) {
    constexpr int STEPS = 4 / GROUPS;
#pragma unroll
    for (int q = 0; q < GROUPS; ++q) {
      v4f d[NT][MT], sum[MT];
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        v8bf b[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          b[m] = __builtin_bit_cast(v8bf, t.x[m][q * STEPS + s]);
          const v4f c = s == 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : sum[m];
          sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, b[m], c, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const v8bf a = decode(t.codes[i][q * STEPS + s]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const v4f c = s == 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : d[i][m];
            d[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[m], c, 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t w = t.scale[i][q][r >> 1];
          const float sc = (r & 1) ? bf16_hi(w) : bf16_lo(w);
          const float off = ZERO ? 16.0f + (float)((t.zero[ZERO ? i : 0][q] >> (8 * r)) & 255u) : 24.0f;
#pragma unroll
          for (int m = 0; m < MT; ++m) y[i][m][r] = fmaf(sc, fmaf(-off, sum[m][r], d[i][m][r]), y[i][m][r]);
        }
    }
  };

  // two tiles in flight
  T a, b;
  int kt = wk;
  if (kt < tiles_k) load(a, kt);
  while (kt < tiles_k) {
    if (kt + g.wk < tiles_k) load(b, kt + g.wk);
    multiply(a);
    kt += g.wk;
    if (kt >= tiles_k) break;
    if (kt + g.wk < tiles_k) load(a, kt + g.wk);
    multiply(b);
    kt += g.wk;
  }

  auto store = [&](int64_t tn, int64_t m, const v4f v) {
    const int64_t n = tn * 16 + quad * 4;
    if (m >= g.M || tn >= g.tiles_n || n >= g.N) return;
    const int count = (int)(g.N - n < 4 ? g.N - n : 4);
    if (F32) {
      float* p = static_cast<float*>(g.y) + m * g.N + n;
      if (count == 4) {
        __builtin_memcpy(p, &v, 16);
      } else {
#pragma unroll
        for (int r = 0; r < 3; ++r)
          if (r < count) p[r] = v[r];
      }
    } else {
      uint16_t* p = static_cast<uint16_t*>(g.y) + m * g.N + n;
      const v2u w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      if (count == 4) {
        __builtin_memcpy(p, &w, 8);
      } else {
#pragma unroll
        for (int r = 0; r < 3; ++r)
          if (r < count) p[r] = (uint16_t)(w[r >> 1] >> (16 * (r & 1)));
      }
    }
  };

  if (g.wk == 1) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) store(tn0 + i, m0 + m * 16 + col, y[i][m]);
    return;
  }
  // the waves along K join their sums, in order: tile t of the workgroup's
  // wn x NT x MT by wave t, t + waves, ...
  constexpr int TILES = NT * MT;
  v4f* sums = reinterpret_cast<v4f*>(s_sum);  // [wn][TILES][wk][64]
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) sums[((wn * TILES + i * MT + m) * g.wk + wk) * 64 + lane] = y[i][m];
  __syncthreads();
  for (int t = wave; t < g.wn * TILES; t += g.wn * g.wk) {
    const int tw = t / TILES, ti = t - tw * TILES;
    v4f v = sums[t * g.wk * 64 + lane];
    for (int k = 1; k < g.wk; ++k) v += sums[(t * g.wk + k) * 64 + lane];
    store(((int64_t)blockIdx.x * g.wn + tw) * NT + ti / MT, m0 + (ti % MT) * 16 + col, v);
  }
}

// ---- weights ----------------------------------------------------------------

// Position of column e of eight in a packed word.
__device__ __forceinline__ int nibble(int e) { return (e >> 1) + 4 * (e & 1); }

// Codes of checkpoints (bytes [N, K / 2], even columns in the low nibbles;
// scales and zero points [N, K / group]) to tiles: a lane's 16 bytes each.
__global__ __launch_bounds__(256) void k_w4_pack(const uint8_t* __restrict__ src, const uint16_t* __restrict__ scale,
                                                 const uint8_t* __restrict__ zero, int64_t N, int64_t K, int group,
                                                 int64_t tiles_k, int64_t tiles, W4Out out) {
  const int64_t tile = (int64_t)wide_block() * 4 + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int lane = threadIdx.x & 63;
  const int64_t tn = tile / tiles_k, tk = tile - tn * tiles_k;
  const int64_t row = tn * 16 + (lane & 15);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int64_t k = tk * 128 + 32 * s + 8 * (lane >> 4);
    if (row < N && k < K) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(src + (row * K + k) / 2);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[s] |= ((v >> (4 * e)) & 15u) << (4 * nibble(e));
    }
  }
  reinterpret_cast<uint4*>(out.codes)[tile * 64 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
  const int groups = 128 / group;
  if (lane < 16 * groups) {  // [4 quads][groups][4 rows]
    const int64_t r = tn * 16 + (lane / (4 * groups)) * 4 + lane % 4, kg = tk * groups + lane / 4 % groups, kgs = K / group;
    const bool in = r < N && kg < kgs;
    out.scale[tile * 16 * groups + lane] = in ? scale[r * kgs + kg] : (uint16_t)0;
    if (out.zero != nullptr) out.zero[tile * 16 * groups + lane] = in ? zero[r * kgs + kg] : (uint8_t)0;
  }
}

// bf16 weights to tiles, a thread for each group of a row:
//   without zero points  s = bf16(max|w| / 7), u = clamp(rne(w / s), -8, 7) + 8;
//   with                 s = bf16((max - min) / 15) (0 among the values),
//                        z = rne(-min / s), u = clamp(rne(w / s) + z, 0, 15).
// A group below 2^-100 gets s = 0; one with a NaN or an infinity s = NaN.
__global__ __launch_bounds__(256) void k_w4_quantize(const uint16_t* __restrict__ src, int64_t N, int64_t K, int group,
                                                     int64_t tiles_n, int64_t tiles_k, W4Out out) {
  const int groups = 128 / group;
  const int64_t kgs = tiles_k * groups, id = (int64_t)wide_block() * 256 + threadIdx.x;
  const int64_t row = id / kgs, kg = id - row * kgs;
  if (row >= tiles_n * 16) return;
  const bool in = row < N && kg * group < K;
  float lo = 0.0f, hi = 0.0f;
  bool finite = true;
  const uint4* p = reinterpret_cast<const uint4*>(src + (in ? row * K + kg * group : 0));
  for (int i = 0; in && i < group / 8; ++i) {
    float v[8];
    bf16x8_to_f32(p[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, v[e]);
      hi = fmaxf(hi, v[e]);
      finite = finite && fabsf(v[e]) < __builtin_inff();
    }
  }
  const bool zp = out.zero != nullptr;
  // halves: hi - lo may pass float32's range
  const float raw = zp ? (0.5f * hi - 0.5f * lo) / 7.5f : fmaxf(hi, -lo) / 7.0f;
  const uint32_t bits = pack_bf16x2(raw, 0.0f) & 0xffffu;
  const float s = finite && raw >= kTiny ? bf16_lo(bits) : 0.0f;
  const float z = zp ? (s > 0.0f ? fminf(rintf(-lo / s), 15.0f) : 0.0f) : 8.0f;
  const int64_t tile = (row >> 4) * tiles_k + kg / groups;
  const int q = (int)(kg % groups), n = (int)(row & 15);
  const int64_t at = (tile * 4 + (n >> 2)) * (groups * 4) + q * 4 + (n & 3);
  out.scale[at] = finite ? (s > 0.0f ? (uint16_t)bits : (uint16_t)0) : (uint16_t)0x7fc0;
  if (zp) out.zero[at] = in ? (uint8_t)z : (uint8_t)0;
  for (int i = 0; i < group / 8; ++i) {
    uint32_t w = 0;
    if (in) {
      float v[8];
      bf16x8_to_f32(p[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = s > 0.0f ? fminf(fmaxf(rintf(v[e] / s) + z, 0.0f), 15.0f) : z;
        w |= (uint32_t)u << (4 * nibble(e));
      }
    }
    const int k = q * group + 8 * i;  // column of the tile
    reinterpret_cast<uint32_t*>(out.codes)[(tile * 64 + ((k >> 3) & 3) * 16 + n) * 4 + (k >> 5)] = w;
  }
}

template <int MT, int NT, int GROUPS, bool ZERO>
hipError_t run(const W4Args& a, const W4Plan& p, bool f32, hipStream_t s) {
  const dim3 grid((unsigned)p.grid_x, (unsigned)p.grid_y), block((unsigned)(64 * p.wn * p.wk));
  const size_t lds = p.wk > 1 ? (size_t)p.wn * p.wk * NT * MT * 1024 : 0;
  if (f32)
    k_w4<MT, NT, GROUPS, ZERO, true><<<grid, block, lds, s>>>(a);
  else
    k_w4<MT, NT, GROUPS, ZERO, false><<<grid, block, lds, s>>>(a);
  return hipGetLastError();
}

template <int MT, int NT>
hipError_t run_tiles(const W4Args& a, const W4Plan& p, int group, bool f32, hipStream_t s) {
  const bool z = a.zero != nullptr;
  switch (group) {
    case 32: return z ? run<MT, NT, 4, true>(a, p, f32, s) : run<MT, NT, 4, false>(a, p, f32, s);
    case 64: return z ? run<MT, NT, 2, true>(a, p, f32, s) : run<MT, NT, 2, false>(a, p, f32, s);
    default: return z ? run<MT, NT, 1, true>(a, p, f32, s) : run<MT, NT, 1, false>(a, p, f32, s);
  }
}

}  // namespace

hipError_t launch_w4(const uint16_t* x, int64_t M, const W4Weights& w, void* y, bool f32, hipStream_t s) {
  const W4Plan p = plan_w4(M, w.N, w.K);
  const W4Args a{x, w.codes, w.scale, w.zero, y, M, w.N, w.K, w4_tiles_n(w.N), w4_tiles_k(w.K), p.wn, p.wk};
  if (p.mt == 1) return run_tiles<1, 1>(a, p, w.group, f32, s);
  if (p.mt == 2) return run_tiles<2, 2>(a, p, w.group, f32, s);
  return run_tiles<4, 2>(a, p, w.group, f32, s);
}

hipError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scale, const uint8_t* zero, int64_t N, int64_t K,
                          int group, const W4Out& out, hipStream_t s) {
  const int64_t tiles = w4_tiles_n(N) * w4_tiles_k(K);
  k_w4_pack<<<wide_grid((tiles + 3) / 4), dim3(256), 0, s>>>(codes, scale, zero, N, K, group, w4_tiles_k(K), tiles, out);
  return hipGetLastError();
}

hipError_t launch_w4_quantize(const uint16_t* w, int64_t N, int64_t K, int group, const W4Out& out, hipStream_t s) {
  const int64_t tn = w4_tiles_n(N), tk = w4_tiles_k(K), threads = tn * 16 * tk * (128 / group);
  k_w4_quantize<<<wide_grid((threads + 255) / 256), dim3(256), 0, s>>>(w, N, K, group, tn, tk, out);
  return hipGetLastError();
}

}  // namespace hdq
