// group_norm.hip -- group norm over channels-last data, with an optional SiLU,
// to bf16 / fp32 or straight to FP8 block-128 codes (gfx950).
//
// x [n, length, channels]; a group is channels / groups adjacent channels of
// one sample:
//   t = (x - mean) rsqrt(var + eps) weight + bias,  y = t or t / (1 + e^-t),
// mean and var over the group's length x channels / groups elements.
//
// Bound by HBM: x has to be read for the statistics before the first output,
// and again unless it is still in a cache.  Three kernels: partial statistics
// per chunk of rows, their join per group, and the normalization.
//
// Statistics: a thread sums d = x - s and d^2 in float32 over its rows, s its
// own first value of each channel, so neither a large mean nor an outlier in
// another thread's rows cancels digits; the (mean, sum of squared deviations)
// pairs are joined in float64, in a fixed order:
//   mean = sum n_i mean_i / n,  M2 = sum M2_i + sum n_i (mean_i - mean)^2.
#include "fp8_device.h"
#include "hdq_internal.h"

namespace hdq {

constexpr int kGnThreads = 512;

// V consecutive elements of bf16 or float data as float.
template <typename T, int V>
__device__ __forceinline__ void gn_load(const T* p, float (&v)[V]) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (V == 8) {
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), v);
    } else if constexpr (V == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    } else {
      v[0] = bf16_lo(*p);
    }
  } else {
    if constexpr (V == 1) {
      v[0] = *p;
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(p + i);
        v[i] = w.x; v[i + 1] = w.y; v[i + 2] = w.z; v[i + 3] = w.w;
      }
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void gn_store(T* p, const float (&v)[V]) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (V == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
      *p = (uint16_t)pack_bf16x2(v[0], 0.0f);
    }
  } else {
    if constexpr (V == 1) {
      *p = v[0];
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  }
}

// t / (1 + e^-t); e^-t past the float range gives 0.
__device__ __forceinline__ float gn_silu(float t) {
  return t * __builtin_amdgcn_rcpf(1.0f + __expf(-t));
}

// Joins `count` (mean, M2) pairs, pair i of weight n(i), over the P lanes of
// an aligned lane group (lane p takes pairs p, p + P, ...).
template <typename Pair, typename Weight>
__device__ __forceinline__ void gn_join(int count, int p, int P, Pair pair, Weight weight, double& n, double& mean,
                                        double& m2) {
  double sn = 0.0, sm = 0.0;
  for (int i = p; i < count; i += P) {
    const double w = weight(i);
    if (w > 0.0) {
      sn += w;
      sm += w * (double)pair(i).x;
    }
  }
  for (int o = 1; o < P; o <<= 1) {
    sn += __shfl_xor(sn, o);
    sm += __shfl_xor(sm, o);
  }
  const double mu = sm / sn;
  double s2 = 0.0;
  for (int i = p; i < count; i += P) {
    const double w = weight(i);
    if (w > 0.0) {
      const auto q = pair(i);
      const double d = (double)q.x - mu;
      s2 += (double)q.y + w * d * d;
    }
  }
  for (int o = 1; o < P; o <<= 1) s2 += __shfl_xor(s2, o);
  n = sn;
  mean = mu;
  m2 = s2;
}

// Lanes that share a group's join: the largest power of two that leaves every
// group its own lane group within `threads`.
__device__ __forceinline__ int gn_lanes(int groups, int threads) {
  int p = 64;
  while (p > 1 && p * groups > threads) p >>= 1;
  return p;
}

// Chunk `c` of sample `s` (blockIdx = s * chunks + c): partial (mean, M2) of
// every group to part[blockIdx][group].  Thread t of the first cv * rpar owns
// channel vector t % cv of rows t / cv, t / cv + rpar, ... (cv channel vectors
// a row, rpar rows at a time; rows of more than 512 vectors in several turns).
template <typename T, int V>
__global__ __launch_bounds__(kGnThreads) void k_gn_partial(const T* __restrict__ x, int64_t length, int C, int groups,
                                                           int chunks, int64_t rows_per, double2* __restrict__ part) {
  extern __shared__ float2 pair_s[];  // [rpar][C]
  const int64_t sample = blockIdx.x / (unsigned)chunks;
  const int chunk = (int)(blockIdx.x % (unsigned)chunks);
  const int64_t r0 = chunk * rows_per;
  const int rows = (int)min(rows_per, length - r0);
  const T* xr = x + (sample * length + r0) * C;
  const int cv = C / V, rpar = cv >= kGnThreads ? 1 : kGnThreads / cv;
  const int pr = rpar > 1 ? (int)threadIdx.x / cv : 0;
  // rows of row slot r: r, r + rpar, ...
  auto slot_rows = [&](int r) { return r < rows ? (rows - r + rpar - 1) / rpar : 0; };
  if (pr < rpar) {
    for (int c = (int)threadIdx.x - pr * cv; c < cv; c += kGnThreads) {
      float s[V], s1[V], s2[V];
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = s1[e] = s2[e] = 0.0f;
      const T* p = xr + (int64_t)pr * C + c * V;
      const int64_t step = (int64_t)rpar * C;
      const int cnt = slot_rows(pr);
      if (cnt > 0) gn_load<T, V>(p, s);
#pragma unroll 4
      for (int i = 1; i < cnt; ++i) {
        float v[V];
        gn_load<T, V>(p + i * step, v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = v[e] - s[e];
          s1[e] += d;
          s2[e] = __builtin_fmaf(d, d, s2[e]);
        }
      }
      const float inv = cnt > 0 ? 1.0f / (float)cnt : 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float dm = s1[e] * inv;
        pair_s[pr * C + c * V + e] = make_float2(s[e] + dm, fmaxf(s2[e] - s1[e] * dm, 0.0f) + 0.0f * s2[e]);
      }
    }
  }
  __syncthreads();
  const int cg = C / groups, P = gn_lanes(groups, kGnThreads);
  for (int g0 = 0; g0 < groups; g0 += kGnThreads / P) {
    const int g = g0 + (int)threadIdx.x / P;
    if (g >= groups) continue;  // lane groups of P leave together
    double n, mean, m2;
    gn_join(
        rpar * cg, (int)threadIdx.x % P, P, [&](int i) { return pair_s[(i / cg) * C + g * cg + i % cg]; },
        [&](int i) { return (double)slot_rows(i / cg); }, n, mean, m2);
    if (threadIdx.x % P == 0) part[(int64_t)blockIdx.x * groups + g] = make_double2(mean, m2);
  }
}

// Group g of sample s (one wave each): mean and 1 / sqrt(var + eps) from the
// chunks' pairs.
__global__ __launch_bounds__(256) void k_gn_final(const double2* __restrict__ part, int64_t total, int64_t length,
                                                  int cg, int groups, int chunks, int64_t rows_per, float eps,
                                                  float2* __restrict__ stat) {
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= total) return;
  const int64_t sample = id / groups;
  const int g = (int)(id - sample * groups), lane = threadIdx.x & 63;
  double n, mean, m2;
  gn_join(
      chunks, lane, 64, [&](int i) { return part[(sample * chunks + i) * groups + g]; },
      [&](int i) { return (double)min(rows_per, length - i * rows_per) * cg; }, n, mean, m2);
  if (lane == 0) stat[id] = make_float2((float)mean, (float)(1.0 / sqrt(m2 / n + (double)eps)));
}

// Rows [r0, r0 + rows_per) of a sample, one channel vector per thread as in
// k_gn_partial; the workgroups run through the rows from the end, so that
// what the statistics read last is still in the memory-side cache.
template <typename TI, typename TO, int V>
__global__ __launch_bounds__(kGnThreads) void k_gn_apply(const TI* x, int64_t length, int C, int groups, int chunks,
                                                         int64_t rows_per, const float2* __restrict__ stat,
                                                         const float* __restrict__ weight,
                                                         const float* __restrict__ bias, int act, TO* y) {
  const unsigned blk = gridDim.x - 1 - blockIdx.x;
  const int64_t sample = blk / (unsigned)chunks;
  const int64_t r0 = (blk % (unsigned)chunks) * rows_per;
  const int rows = (int)min(rows_per, length - r0);
  const int64_t base = (sample * length + r0) * C;
  const int cv = C / V, rpar = cv >= kGnThreads ? 1 : kGnThreads / cv;
  const int pr = rpar > 1 ? (int)threadIdx.x / cv : 0;
  if (pr >= rpar) return;
  const int cg = C / groups;
  for (int c = (int)threadIdx.x - pr * cv; c < cv; c += kGnThreads) {
    float mean[V], a[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int ch = c * V + e;
      const float2 st = stat[sample * groups + ch / cg];
      mean[e] = st.x;
      a[e] = weight != nullptr ? st.y * weight[ch] : st.y;
      b[e] = bias != nullptr ? bias[ch] : 0.0f;
    }
    const int64_t o = base + (int64_t)pr * C + c * V, step = (int64_t)rpar * C;
    const int cnt = pr < rows ? (rows - pr + rpar - 1) / rpar : 0;
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
      float v[V];
      gn_load<TI, V>(x + o + i * step, v);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float t = __builtin_fmaf(v[e] - mean[e], a[e], b[e]);
        v[e] = act ? gn_silu(t) : t;
      }
      gn_store<TO, V>(y + o + i * step, v);
    }
  }
}

// The normalization to FP8 codes: a wave owns one block of 128 channels (lane
// l: rows l / 4, l / 4 + 16, ... of its chunk, 32 channels of the block's
// quarter l % 4), keeping its channels' factors in registers over the rows.
template <typename TI, int HB>
__global__ __launch_bounds__(256) void k_gn_apply_fp8(const TI* __restrict__ x, int64_t length, int C, int groups,
                                                      int chunks, int64_t rows_per, const float2* __restrict__ stat,
                                                      const float* __restrict__ weight,
                                                      const float* __restrict__ bias, int act, float c_b, int kb,
                                                      int64_t total_rows, uint8_t* __restrict__ codes,
                                                      float* __restrict__ scale) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = lane & 3;
  const int kgroups = (kb + 3) >> 2;
  const unsigned blk = gridDim.x - 1 - blockIdx.x;
  const int b = (int)(blk % (unsigned)kgroups) * 4 + wave;
  const unsigned rest = blk / (unsigned)kgroups;
  const int64_t sample = rest / (unsigned)chunks;
  const int64_t r0 = (rest % (unsigned)chunks) * rows_per;
  const int rows = (int)min(rows_per, length - r0);
  if (b >= kb) return;
  const int ch0 = b * kFp8Block + part * 32, cg = C / groups;
  float mean[32], a[32], bs[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const int ch = min(ch0 + e, C - 1);
    const float2 st = stat[sample * groups + ch / cg];
    const bool in = ch0 + e < C;
    mean[e] = st.x;
    a[e] = in ? (weight != nullptr ? st.y * weight[ch] : st.y) : 0.0f;
    bs[e] = in && bias != nullptr ? bias[ch] : 0.0f;
  }
  for (int r = lane >> 2; r < rows; r += 16) {  // whole quads stay together
    const int64_t row = sample * length + r0 + r;
    float y[32];
    const TI* p = x + row * C + ch0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float t[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      const bool in = ch0 + 8 * i < C;  // C is a multiple of 8
      if (in) gn_load<TI, 8>(p + 8 * i, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = __builtin_fmaf(t[e] - mean[8 * i + e], a[8 * i + e], bs[8 * i + e]);
        y[8 * i + e] = in ? (act ? gn_silu(u) : u) : 0.0f;
      }
    }
    rotate32<HB>(y, lane, c_b);
    float s, inv;
    fp8_scales(quad_max(absmax32(y)), s, inv);
    uint4 out[2];
    // lanes past the channels (whole Hadamard blocks) hold rotated zeros of either sign
    fp8_encode32(y, ch0 < C ? inv : 0.0f, out);
    uint4* dst = reinterpret_cast<uint4*>(codes + row * ((int64_t)kb * kFp8Block) + ch0);
    dst[0] = out[0];
    dst[1] = out[1];
    if (part == 0) scale[(int64_t)b * total_rows + row] = s;
  }
}

// Chunks of a sample's rows for a pass of about 2048 workgroups that take `per`
// rows at least.
static void gn_chunks(int64_t n, int64_t length, int64_t per, int64_t& chunks, int64_t& rows_per) {
  int64_t want = (2048 + n - 1) / n;
  if (want > (length + per - 1) / per) want = (length + per - 1) / per;
  if (want < 1) want = 1;
  rows_per = (length + want - 1) / want;
  chunks = (length + rows_per - 1) / rows_per;
}

static int64_t gn_vec(int64_t C) { return C % 8 == 0 ? 8 : C % 4 == 0 ? 4 : 1; }
static int64_t gn_rpar(int64_t C) {
  const int64_t cv = C / gn_vec(C);
  return cv >= kGnThreads ? 1 : kGnThreads / cv;
}

static void gn_stat_chunks(int64_t n, int64_t length, int64_t C, int64_t& chunks, int64_t& rows_per) {
  gn_chunks(n, length, 8 * gn_rpar(C), chunks, rows_per);
}

static size_t gn_align(size_t v) { return (v + 255) / 256 * 256; }

size_t group_norm_ws_bytes(int64_t n, int64_t length, int64_t C, int64_t groups) {
  int64_t chunks, rows_per;
  gn_stat_chunks(n, length, C, chunks, rows_per);
  return gn_align((size_t)(n * chunks * groups) * sizeof(double2)) + gn_align((size_t)(n * groups) * sizeof(float2));
}

template <typename TI, int V>
static hipError_t gn_partial(const GroupNormArgs& g, double2* part, int64_t chunks, int64_t rows_per, hipStream_t s) {
  const size_t lds = (size_t)(gn_rpar(g.C) * g.C) * sizeof(float2);
  if (g.n * chunks > 0x7fffffff) return hipErrorInvalidValue;
  k_gn_partial<TI, V><<<dim3((unsigned)(g.n * chunks)), dim3(kGnThreads), lds, s>>>(
      static_cast<const TI*>(g.x), g.length, (int)g.C, (int)g.groups, (int)chunks, rows_per, part);
  return hipGetLastError();
}

// The statistics of every (sample, group) into ws; *stat points at them.
static hipError_t gn_statistics(const GroupNormArgs& g, void* ws, float2** stat, hipStream_t s) {
  int64_t chunks, rows_per;
  gn_stat_chunks(g.n, g.length, g.C, chunks, rows_per);
  double2* part = static_cast<double2*>(ws);
  *stat = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) +
                                    gn_align((size_t)(g.n * chunks * g.groups) * sizeof(double2)));
  hipError_t e;
  switch (gn_vec(g.C)) {
    case 8: e = g.x_f32 ? gn_partial<float, 8>(g, part, chunks, rows_per, s) : gn_partial<uint16_t, 8>(g, part, chunks, rows_per, s); break;
    case 4: e = g.x_f32 ? gn_partial<float, 4>(g, part, chunks, rows_per, s) : gn_partial<uint16_t, 4>(g, part, chunks, rows_per, s); break;
    default: e = g.x_f32 ? gn_partial<float, 1>(g, part, chunks, rows_per, s) : gn_partial<uint16_t, 1>(g, part, chunks, rows_per, s); break;
  }
  if (e != hipSuccess) return e;
  const int64_t total = g.n * g.groups;
  k_gn_final<<<dim3((unsigned)((total + 3) / 4)), dim3(256), 0, s>>>(part, total, g.length, (int)(g.C / g.groups),
                                                                     (int)g.groups, (int)chunks, rows_per, g.eps, *stat);
  return hipGetLastError();
}

template <typename TI, typename TO, int V>
static hipError_t gn_apply(const GroupNormArgs& g, const float2* stat, void* y, hipStream_t s) {
  int64_t chunks, rows_per;
  gn_chunks(g.n, g.length, 4 * gn_rpar(g.C), chunks, rows_per);
  if (g.n * chunks > 0x7fffffff) return hipErrorInvalidValue;
  k_gn_apply<TI, TO, V><<<dim3((unsigned)(g.n * chunks)), dim3(kGnThreads), 0, s>>>(
      static_cast<const TI*>(g.x), g.length, (int)g.C, (int)g.groups, (int)chunks, rows_per, stat, g.weight, g.bias,
      g.act, static_cast<TO*>(y));
  return hipGetLastError();
}

template <typename TI, typename TO>
static hipError_t gn_apply_v(const GroupNormArgs& g, const float2* stat, void* y, hipStream_t s) {
  switch (gn_vec(g.C)) {
    case 8: return gn_apply<TI, TO, 8>(g, stat, y, s);
    case 4: return gn_apply<TI, TO, 4>(g, stat, y, s);
    default: return gn_apply<TI, TO, 1>(g, stat, y, s);
  }
}

hipError_t launch_group_norm(const GroupNormArgs& g, void* y, bool y_f32, void* ws, hipStream_t s) {
  float2* stat;
  const hipError_t e = gn_statistics(g, ws, &stat, s);
  if (e != hipSuccess) return e;
  if (g.x_f32) return y_f32 ? gn_apply_v<float, float>(g, stat, y, s) : gn_apply_v<float, uint16_t>(g, stat, y, s);
  return y_f32 ? gn_apply_v<uint16_t, float>(g, stat, y, s) : gn_apply_v<uint16_t, uint16_t>(g, stat, y, s);
}

template <typename TI, int HB>
static hipError_t gn_apply_fp8(const GroupNormArgs& g, const float2* stat, uint8_t* codes, float* scale,
                               hipStream_t s) {
  const int64_t kb = fp8_blocks(g.C), kgroups = (kb + 3) / 4;
  int64_t chunks, rows_per;
  gn_chunks(g.n * kgroups, g.length, 16, chunks, rows_per);
  if (g.n * chunks * kgroups > 0x7fffffff) return hipErrorInvalidValue;
  k_gn_apply_fp8<TI, HB><<<dim3((unsigned)(g.n * chunks * kgroups)), dim3(256), 0, s>>>(
      static_cast<const TI*>(g.x), g.length, (int)g.C, (int)g.groups, (int)chunks, rows_per, stat, g.weight, g.bias,
      g.act, hadamard_scale(HB), (int)kb, g.n * g.length, codes, scale);
  return hipGetLastError();
}

template <typename TI>
static hipError_t gn_apply_fp8_hb(const GroupNormArgs& g, int hb, const float2* stat, uint8_t* codes, float* scale,
                                  hipStream_t s) {
  switch (hb) {
    case 1: return gn_apply_fp8<TI, 1>(g, stat, codes, scale, s);
    case 2: return gn_apply_fp8<TI, 2>(g, stat, codes, scale, s);
    case 4: return gn_apply_fp8<TI, 4>(g, stat, codes, scale, s);
    case 8: return gn_apply_fp8<TI, 8>(g, stat, codes, scale, s);
    case 16: return gn_apply_fp8<TI, 16>(g, stat, codes, scale, s);
    case 32: return gn_apply_fp8<TI, 32>(g, stat, codes, scale, s);
    case 64: return gn_apply_fp8<TI, 64>(g, stat, codes, scale, s);
    case 128: return gn_apply_fp8<TI, 128>(g, stat, codes, scale, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_group_norm_fp8(const GroupNormArgs& g, int hb, uint8_t* codes, float* scale, void* ws,
                                 hipStream_t s) {
  float2* stat;
  const hipError_t e = gn_statistics(g, ws, &stat, s);
  if (e != hipSuccess) return e;
  return g.x_f32 ? gn_apply_fp8_hb<float>(g, hb, stat, codes, scale, s)
                 : gn_apply_fp8_hb<uint16_t>(g, hb, stat, codes, scale, s);
}

}  // namespace hdq
