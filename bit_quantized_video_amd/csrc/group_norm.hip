// group_norm.hip -- group norm over channels-last data, with an optional SiLU,
// to bf16 / fp32 or straight to FP8 block-128 codes (gfx950).
//
// x [n, length, channels]; a group is channels / groups adjacent channels of
// one sample:
//   t = (x - mean) / sqrt(var + eps) weight + bias,  y = t or t / (1 + e^-t),
// mean and var over the group's length x channels / groups elements.
//
// Bound by HBM: x has to be read for the statistics before the first output,
// and again unless it is kept.  Three ways, by the size of a sample's slab (the
// channels of a few groups, see gn_plan): a slab that fits a workgroup's
// registers is read once, normalized and written in one launch; a slab that one
// workgroup can still stream takes one launch for the statistics and one for
// the normalization; else partial statistics per chunk of rows, their join (of
// few chunks in small inputs: by the normalization itself) and the
// normalization.  The FP8 form codes whole rows, so it has no slab form: its
// short samples take one launch whose workgroups each read the whole sample for
// the statistics (k_gn_short_fp8), the others the plain form's statistics.
// Measured: 691200 x 256 bf16 with SiLU 177 us (4.0 TB/s of bytes read and
// written once, where a large copy reaches 4.8), 13 x 1350 x 512 17.5 us (9 + 8:
// the statistics of 18 MB are two rounds of loads of 32-byte pieces in 416
// workgroups), to FP8 21 (9 + 12), 2 x 77 x 300 fp32 5.9 us (one launch's
// latency), 225 x 320 to FP8 10.9 (one launch whose 15 workgroups each read the
// sample's 144 KB).
//
// Statistics: a thread takes up to 16 rows at a time into registers, sums each
// channel's values (relative to the first) and then the squared deviations from
// their mean, in float32, so neither a large mean nor an outlier cancels
// digits; (mean, sum of squared deviations) pairs are joined by
//   mean = sum n_i mean_i / n,  M2 = sum M2_i + sum n_i (mean_i - mean)^2,
// in a fixed order: means in float64 throughout (rounded to float32 once, in a
// thread's pair), a thread's own M2 in float32 and the joined ones in float64.
// Where a thread's M2 leaves the float32 range, it sums its rows anew in float64,
// so every finite input has finite statistics.
#include "fp8_device.h"
#include "group_norm_plan.h"
#include "hdq_internal.h"

#include <algorithm>
#include <type_traits>

namespace hdq {

// a slab's pairs (one per thread and channel of its vector) and groups
constexpr int kGnSlabLds = kGnSlabThreads * 8 * 8 + 8 * 8192;
// a short sample's pairs, groups and coefficients (at most 512 channels)
constexpr int kGnShortLds = (kGnThreads * 8 + 512 + 2) * 8 + 3 * 512 * 4;

// NT: 16-byte stores that do not stay in the caches.
template <typename T, int V, bool NT = false>
__device__ __forceinline__ void gn_store(T* p, const float (&v)[V]) {
  constexpr int WORDS = (V * (int)sizeof(T) + 3) / 4;
  uint32_t w[WORDS];
#pragma unroll
  for (int i = 0; i < WORDS; ++i)
    w[i] = sizeof(T) == 4 ? __float_as_uint(v[i]) : pack_bf16x2(v[(2 * i) % V], v[(2 * i + 1) % V]);
  if constexpr (sizeof(T) == 2 && V == 1) {
    *p = (T)w[0];
  } else if constexpr (WORDS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const v4i q = v4i{(int)w[i], (int)w[i + 1], (int)w[i + 2], (int)w[i + 3]};
      v4i* d = reinterpret_cast<v4i*>(reinterpret_cast<uint32_t*>(p) + i);
      if constexpr (NT)
        __builtin_nontemporal_store(q, d);
      else
        *d = q;
    }
  } else if constexpr (WORDS == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

// V elements as loaded (bf16 stay packed).
template <typename T, int V>
struct GnRaw {
  static constexpr int WORDS = (V * (int)sizeof(T) + 3) / 4;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(T) == 2 && V == 1) {
      w[0] = *p;
    } else if constexpr (WORDS % 4 == 0) {
#pragma unroll
      for (int i = 0; i < WORDS; i += 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
      }
    } else if constexpr (WORDS == 2) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x; w[1] = q.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
    for (int e = 0; e < V; ++e)
      v[e] = sizeof(T) == 4 ? __uint_as_float(w[e]) : (e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
  }
};

// t / (1 + e^-t) from the hardware's exponential and reciprocal (one step each),
// for float32 outputs too: (2 |t| / (1 + e^t) + 6) 2^-24 of it at most, so about
// as good as its float32 t; library ones would only take longer.  e^-t past the
// float range gives 0.
__device__ __forceinline__ float gn_silu(float t) {
  return t * __builtin_amdgcn_rcpf(1.0f + __expf(-t));
}

// Lanes that share a group's join: the largest power of two that leaves every
// group its own lane group within `threads`.
__device__ __forceinline__ int gn_lanes(int groups, int threads) {
  int p = 64;
  while (p > 1 && p * groups > threads) p >>= 1;
  return p;
}

// A pair among a workgroup's: mean and variance in float32, or with the sign set
// the root of a variance that is not in the float32 range (or of NaN).
__device__ __forceinline__ float2 gn_wide_pair(double mean, double var) {
  return make_float2((float)mean, -(float)sqrt(var));
}
__device__ __forceinline__ double gn_pair_var(const float2& q) {
  return q.y >= 0.0f ? (double)q.y : (double)q.y * (double)q.y;
}

// A thread's (mean, M2) of each channel of one vector over n rows.  The mean is
// kept in float64: one workgroup may have a sample's every row, and a float32
// mean rounded again every eight rows drifts by 2e-3 deviations over 20000 of
// them when it is 2000 times the deviation.
template <int V>
struct GnSums {
  float n, m2[V];
  double mean[V];
  // The mean and M2 of the first cnt (1 .. K) of K rows held in q.
  template <typename T, int K>
  static __device__ __forceinline__ void rows(const GnRaw<T, V> (&q)[K], int cnt, float (&m)[V], float (&d2)[V]) {
    float x0[V];
    q[0].get(x0);
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = d2[e] = 0.0f;
#pragma unroll
    for (int u = 1; u < K; ++u)
      if (u < cnt) {
        float v[V];
        q[u].get(v);
#pragma unroll
        for (int e = 0; e < V; ++e) m[e] += v[e] - x0[e];
      }
    const float inv = 1.0f / (float)cnt;
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = __builtin_fmaf(m[e], inv, x0[e]);
#pragma unroll
    for (int u = 0; u < K; ++u)
      if (u < cnt) {
        float v[V];
        q[u].get(v);
#pragma unroll
        for (int e = 0; e < V; ++e) d2[e] = __builtin_fmaf(v[e] - m[e], v[e] - m[e], d2[e]);
      }
  }
  // Begins with the first cnt rows in q.
  template <typename T, int K>
  __device__ __forceinline__ void start(const GnRaw<T, V> (&q)[K], int cnt) {
    float m[V];
    rows(q, cnt, m, m2);
    n = (float)cnt;
#pragma unroll
    for (int e = 0; e < V; ++e) mean[e] = (double)m[e];
  }
  // Joins all K rows in q.
  template <typename T, int K>
  __device__ __forceinline__ void add(const GnRaw<T, V> (&q)[K]) {
    float m[V], d2[V];
    rows(q, K, m, d2);
    const float k = (float)K, f = k / (n + k), g = n * f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const double d = (double)m[e] - mean[e];
      const float df = (float)d;
      m2[e] += __builtin_fmaf(df * df, g, d2[e]);
      mean[e] = __builtin_fma(d, (double)f, mean[e]);
    }
    n += k;
  }
  // Whether M2 holds: not past the float32 range (then it is infinite, or NaN),
  // nor so small that squares may have underflowed.
  __device__ __forceinline__ bool holds(float least) const {
    bool ok = true;
#pragma unroll
    for (int e = 0; e < V; ++e) ok = ok & (m2[e] >= least) & (m2[e] < __builtin_inff());
    return ok;
  }
  // The pair of channel e, and of all V together (one group's), inv = 1 / n.
  __device__ __forceinline__ float2 one(int e, float inv) const { return make_float2((float)mean[e], m2[e] * inv); }
  __device__ __forceinline__ float2 all(float inv) const {
    float d[V], m = 0.0f, v = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      d[e] = (float)(mean[e] - mean[0]);
      m += d[e] * (1.0f / V);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) v += __builtin_fmaf(d[e] - m, d[e] - m, m2[e] * inv) * (1.0f / V);
    return make_float2((float)(mean[0] + (double)m), v);
  }
};

// Sums of squared deviations below this may have lost float32 squares to
// underflow; an eps above 2^-100 hides them.
__host__ __device__ inline float gn_least(float eps) { return eps < 0x1p-100f ? 0x1p-60f : 0.0f; }

__device__ __forceinline__ double gn_value(float v) { return v; }
__device__ __forceinline__ double gn_value(uint16_t v) { return bf16_lo(v); }

// A channel's mean and M2 over cnt rows, in float64, a value at a time: for the
// threads whose M2 float32 does not hold.
template <typename T>
__device__ __forceinline__ void gn_wide_sums(const T* p, int64_t step, int cnt, double& mean, double& m2) {
  const double first = gn_value(p[0]);
  mean = m2 = 0.0;
#pragma nounroll
  for (int i = 0; i < cnt; ++i) mean += gn_value(p[i * step]) - first;
  mean = first + mean / cnt;
#pragma nounroll
  for (int i = 0; i < cnt; ++i) {
    const double d = gn_value(p[i * step]) - mean;
    m2 = __builtin_fma(d, d, m2);
  }
}

// Sums cnt vectors at p, p + step, ...; eight loads are in flight at a time.  The
// odd ones come first, where there is nothing to join them with.
template <typename T, int V>
__device__ __forceinline__ void gn_stream(const T* p, int64_t step, int cnt, GnSums<V>& t) {
  if (cnt == 0) return;
  GnRaw<T, V> q[8];
  const int head = ((cnt - 1) & 7) + 1;
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (u < head) q[u].load(p + u * step);
  t.start(q, head);
  for (int i = head; i < cnt; i += 8) {
#pragma unroll
    for (int u = 0; u < 8; ++u) q[u].load(p + (i + u) * step);
    t.add(q);
  }
}

// A thread's pairs from sums made anew in float64 (gn_put).  That it is there costs
// the statistics of 13 x 1350 x 512 0.2 to 0.4 us of 9 (0.6 where the test for it
// branched for each channel).
template <bool MERGE, int V, typename T>
__device__ __forceinline__ void gn_put_wide(float2* to, const T* p, int64_t step, int cnt) {
  double sd = 0.0, s2 = 0.0, ref = 0.0;  // MERGE: sums of d and M2 / cnt + d^2, d a channel's distance from ref
#pragma nounroll
  for (int e = 0; e < V; ++e) {
    double mean, m2;
    gn_wide_sums(p + e, step, cnt, mean, m2);
    if constexpr (MERGE) {
      if (e == 0) ref = mean;
      const double d = mean - ref;
      sd += d;
      s2 += m2 / cnt + d * d;
    } else {
      to[e] = gn_wide_pair(mean, m2 / cnt);
    }
  }
  if constexpr (MERGE)
    to[0] = gn_wide_pair(ref + sd / V, fmax(s2 / V - (sd / V) * (sd / V), 0.0) + 0.0 * s2);
}

// Puts the pairs of a thread's sums (cnt rows at p, p + step, ...; row slot pr,
// channel vector c of cv) among a workgroup's: one pair per thread when a vector
// lies in one group (MERGE), else one per channel.
template <bool MERGE, typename T, int V>
__device__ __forceinline__ void gn_put(float2* pairs, const GnSums<V>& t, const T* p, int64_t step, int cnt,
                                       float least, int pr, int c, int cv) {
  if (cnt == 0) return;
  float2* const to = pairs + (pr * cv + c) * (MERGE ? 1 : V);
  const float inv = 1.0f / (float)cnt;
  bool ok = t.holds(least);
  if constexpr (MERGE) {
    const float2 q = t.all(inv);
    ok = ok & (q.y < __builtin_inff());
    to[0] = q;
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) to[e] = t.one(e, inv);
  }
  if (__builtin_expect(!ok, 0)) gn_put_wide<MERGE, V>(to, p, step, cnt);
}
// The end of a join over P lanes, from the lanes' sums of n, n d and M2 + n d^2.
__device__ __forceinline__ void gn_join_lanes(int P, double ref, double sn, double sd, double s2, double& n,
                                              double& mean, double& m2) {
  for (int o = 1; o < P; o <<= 1) {
    sn += __shfl_xor(sn, o);
    sd += __shfl_xor(sd, o);
    s2 += __shfl_xor(s2, o);
  }
  n = sn;
  mean = ref + sd / sn;
  m2 = fmax(s2 - sd * (sd / sn), 0.0) + 0.0 * s2;  // NaN stays NaN
}
// Joins group g's pairs of row slots 0 .. slots - 1 (slot r: rows(r) rows) over
// the P lanes of an aligned lane group, in one pass: sums of n, n d and
// n (variance + d^2) in float64, d the distance of a pair's mean from the first
// one's.
template <bool MERGE, int V, typename Rows>
__device__ __forceinline__ void gn_join_group(const float2* pairs, int g, int cg, int cv, int slots, int p, int P,
                                              Rows rows, double& n, double& mean, double& m2) {
  const int per = MERGE ? cg / V : cg, pitch = MERGE ? cv : cv * V;
  const float2* base = pairs + g * per;
  const double ref = (double)base[0].x;
  double sn = 0.0, sd = 0.0, s2 = 0.0;
  // lane p takes pairs p, p + P, ... of the group's slots x per
  int r = p / per, c = p - r * per;
  const int dr = P / per, dc = P - dr * per;
  while (r < slots) {
    const float2 q = base[r * pitch + c];
    const double w = (double)(rows(r) * (MERGE ? V : 1)), d = (double)q.x - ref;
    sn += w;
    sd += w * d;
    s2 += w * (gn_pair_var(q) + d * d);
    r += dr;
    c += dc;
    if (c >= per) {
      c -= per;
      ++r;
    }
  }
  gn_join_lanes(P, ref, sn, sd, s2, n, mean, m2);
}

// A group's (mean / 4, 4 rstd): t = (x / 4 - mean / 4) (4 rstd weight) + bias has
// the roundings of the formula without the fours, and neither the difference of
// two finite values overflows nor rstd underflows.
__device__ __forceinline__ float2 gn_stat(double mean, double m2, double n, float eps) {
  return make_float2((float)(0.25 * mean), (float)(4.0 / sqrt(m2 / n + (double)eps)));
}

// Chunk `c` of sample `s` (blockIdx = s * chunks + c): partial (mean, M2) of
// every group to part[blockIdx][group].  Thread t of the first cv * rpar owns
// channel vector t % cv of rows t / cv, t / cv + rpar, ... (cv channel vectors
// a row, rpar rows at a time; rows of more than 512 vectors in several turns).
template <typename T, int V, bool MERGE>
__global__ __launch_bounds__(kGnThreads) void k_gn_partial(const T* __restrict__ x, int64_t length, int C, int groups,
                                                           int chunks, int64_t rows_per, float least,
                                                           double2* __restrict__ part) {
  extern __shared__ float2 pair_s[];  // [rpar][C], or with MERGE [rpar][cv]
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
      const T* p = xr + (int64_t)pr * C + c * V;
      const int64_t step = (int64_t)rpar * C;
      const int cnt = slot_rows(pr);
      GnSums<V> t;
      gn_stream<T, V>(p, step, cnt, t);
      gn_put<MERGE>(pair_s, t, p, step, cnt, least, pr, c, cv);
    }
  }
  __syncthreads();
  const int cg = C / groups, P = gn_lanes(groups, kGnThreads);
  for (int g0 = 0; g0 < groups; g0 += kGnThreads / P) {
    const int g = g0 + (int)threadIdx.x / P;
    if (g >= groups) continue;  // lane groups of P leave together
    double n, mean, m2;
    gn_join_group<MERGE, V>(pair_s, g, cg, cv, min(rpar, rows), (int)threadIdx.x % P, P, slot_rows, n, mean, m2);
    if (threadIdx.x % P == 0) part[(int64_t)blockIdx.x * groups + g] = make_double2(mean, m2);
  }
}

// What the normalization reads per sample and channel, three rows of C floats:
// mean / 4, a = 4 rstd * weight, b = bias, so t = (x / 4 - mean / 4) a + b.
__device__ __forceinline__ void gn_write_coef(float* __restrict__ coef, int C, int ch, float2 st,
                                              const float* __restrict__ weight, const float* __restrict__ bias) {
  coef[ch] = st.x;
  coef[C + ch] = weight != nullptr ? st.y * weight[ch] : st.y;
  coef[2 * C + ch] = bias != nullptr ? bias[ch] : 0.0f;
}

// Group g of sample s (one wave each): the join of at most 512 chunks' pairs,
// and its channels' coefficients.
__global__ __launch_bounds__(kGnFinalThreads) void k_gn_final(const double2* __restrict__ part, int64_t total, int64_t length,
                                                  int cg, int groups, int chunks, int64_t rows_per, float eps,
                                                  const float* __restrict__ weight, const float* __restrict__ bias,
                                                  float* __restrict__ coef) {
  const int64_t id = (int64_t)wide_block() * kGnFinalGroups + (threadIdx.x >> 6);
  if (id >= total) return;
  const int64_t sample = id / groups;
  const int g = (int)(id - sample * groups), lane = threadIdx.x & 63;
  // all of the lane's pairs are loaded before the first is used
  constexpr int PER = kGnMaxChunks / 64;
  double2 q[PER];
  double w[PER];
  double sn = 0.0, sm = 0.0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int i = lane + 64 * k;
    w[k] = i < chunks ? (double)min(rows_per, length - i * rows_per) * cg : 0.0;
    q[k] = i < chunks ? part[(sample * chunks + i) * groups + g] : make_double2(0.0, 0.0);
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    sn += w[k];
    sm += w[k] * q[k].x;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    sn += __shfl_xor(sn, o);
    sm += __shfl_xor(sm, o);
  }
  const double mean = sm / sn;
  double m2 = 0.0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const double d = q[k].x - mean;
    m2 += w[k] > 0.0 ? q[k].y + w[k] * d * d : 0.0;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m2 += __shfl_xor(m2, o);
  const float2 st = gn_stat(mean, m2, sn, eps);
  const int C = cg * groups;
  for (int c = lane; c < cg; c += 64)
    gn_write_coef(coef + sample * 3 * C, C, g * cg + c, st, weight, bias);
}

// V consecutive coefficients (16-byte aligned when V is 4 or 8: C is then a multiple of 4).
template <int V>
__device__ __forceinline__ void gn_load_coef(const float* __restrict__ p, float (&v)[V]) {
  GnRaw<float, V> q;
  q.load(p);
  q.get(v);
}

template <int V>
__device__ __forceinline__ void gn_normalize(float (&v)[V], const float (&mean)[V], const float (&a)[V],
                                             const float (&b)[V], int act) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float t = __builtin_fmaf(__builtin_fmaf(v[e], 0.25f, -mean[e]), a[e], b[e]);
    v[e] = act ? gn_silu(t) : t;
  }
}

// Where a normalization takes its groups' statistics from: coefficients that a
// launch before it has written, or (JOIN) the statistics' chunks, which each
// workgroup joins itself.
struct GnFrom {
  const float* coef;
  const double2* part;
  int chunks;
  int64_t rows_per;
  int groups;
  float eps;
  const float* weight;
  const float* bias;
};

// (mean, rstd) of a sample's groups into stat_s, from its chunks' pairs.
template <int T>
__device__ __forceinline__ void gn_join_chunks(const GnFrom& f, int64_t sample, int64_t length, int cg, float2* stat_s) {
  const double2* part = f.part + sample * f.chunks * f.groups;
  const int P = gn_lanes(f.groups, T), p = (int)threadIdx.x % P;
  for (int g0 = 0; g0 < f.groups; g0 += T / P) {
    const int g = g0 + (int)threadIdx.x / P;
    if (g >= f.groups) continue;  // lane groups of P leave together
    const double ref = part[g].x;
    double sn = 0.0, sd = 0.0, s2 = 0.0;
    for (int i = p; i < f.chunks; i += P) {
      const double2 q = part[i * f.groups + g];
      const double w = (double)min(f.rows_per, length - i * f.rows_per) * cg, d = q.x - ref;
      sn += w;
      sd += w * d;
      s2 += q.y + w * d * d;
    }
    double n, mean, m2;
    gn_join_lanes(P, ref, sn, sd, s2, n, mean, m2);
    if (p == 0) stat_s[g] = gn_stat(mean, m2, n, f.eps);
  }
  __syncthreads();
}

// A vector's coefficients.
template <int V, bool JOIN>
__device__ __forceinline__ void gn_coefs(const GnFrom& f, int64_t sample, int C, int cg, int ch, const float2* stat_s,
                                         float (&mean)[V], float (&a)[V], float (&b)[V]) {
  if constexpr (JOIN) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 st = stat_s[(ch + e) / cg];
      mean[e] = st.x;
      a[e] = f.weight != nullptr ? st.y * f.weight[ch + e] : st.y;
      b[e] = f.bias != nullptr ? f.bias[ch + e] : 0.0f;
    }
  } else {
    const float* cf = f.coef + sample * 3 * C + ch;
    gn_load_coef<V>(cf, mean);
    gn_load_coef<V>(cf + C, a);
    gn_load_coef<V>(cf + 2 * C, b);
  }
}

// Rows [r0, r0 + rows_per) of a sample, one channel vector per thread as in
// k_gn_partial; the workgroups run through the rows from the end, so that
// what the statistics read last is still in the memory-side cache.
template <typename TI, typename TO, int V, bool JOIN>
__global__ __launch_bounds__(kGnThreads) void k_gn_apply(const TI* x, int64_t length, int C, int chunks,
                                                         int64_t rows_per, GnFrom from, int act, TO* y) {
  extern __shared__ float2 pair_s[];  // JOIN: one (mean, rstd) per group
  const unsigned blk = gridDim.x - 1 - blockIdx.x;
  const int64_t sample = blk / (unsigned)chunks;
  const int64_t r0 = (blk % (unsigned)chunks) * rows_per;
  const int rows = (int)min(rows_per, length - r0);
  const int64_t base = (sample * length + r0) * C;
  const int cv = C / V, rpar = cv >= kGnThreads ? 1 : kGnThreads / cv;
  const int pr = rpar > 1 ? (int)threadIdx.x / cv : 0;
  const int cg = JOIN ? C / from.groups : 1;
  if constexpr (JOIN) gn_join_chunks<kGnThreads>(from, sample, length, cg, pair_s);
  if (pr >= rpar) return;
  for (int c = (int)threadIdx.x - pr * cv; c < cv; c += kGnThreads) {
    float mean[V], a[V], b[V];
    gn_coefs<V, JOIN>(from, sample, C, cg, c * V, pair_s, mean, a, b);
    const int64_t o = base + (int64_t)pr * C + c * V, step = (int64_t)rpar * C;
    const int cnt = pr < rows ? (rows - pr + rpar - 1) / rpar : 0;
    // four rows are loaded before the first is stored (y may be x)
    for (int i = 0; i < cnt; i += 4) {
      GnRaw<TI, V> q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < cnt) q[u].load(x + o + (i + u) * step);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < cnt) {
          float v[V];
          q[u].get(v);
          gn_normalize<V>(v, mean, a, b, act);
          gn_store<TO, V, true>(y + o + (i + u) * step, v);
        }
    }
  }
}

// A slab: `width` channels (whole groups and vectors) of one sample, one
// workgroup.  Thread t owns channel vector t % cv of rows t / cv, + rpar, ...
// (cv vectors a slab row).  ROWS > 0: the thread's at most ROWS vectors stay in
// registers, and the slab is normalized and written from them.  ROWS 0: the
// slab is streamed and its channels' coefficients are written.
template <typename TI, typename TO, int V, bool MERGE, int T, int ROWS>
__global__ __launch_bounds__(T) void k_gn_slab(const TI* x, int64_t length, int C, int cg, int width,
                                                            int slabs, float eps, const float* __restrict__ weight,
                                                            const float* __restrict__ bias, int act, TO* y,
                                                            float* __restrict__ coef) {
  extern __shared__ float2 pair_s[];  // [rpar][width or cv], then one (mean, rstd) per group of the slab
  // neighbouring slabs on one XCD at a time: they share the rows' cache lines
  int lo, hi;
  xcd_range((int)gridDim.x, blockIdx.x & 7, lo, hi);
  const unsigned id = (unsigned)lo + (blockIdx.x >> 3);
  const int64_t sample = id / (unsigned)slabs;
  const int c0 = (int)(id % (unsigned)slabs) * width, w = min(width, C - c0);
  const int cv = w / V, rpar = T / cv, groups = w / cg, rows = (int)length;
  const int pr = (int)threadIdx.x / cv, c = (int)threadIdx.x - pr * cv;
  float2* const stat_s = pair_s + rpar * (MERGE ? cv : w);
  auto slot_rows = [&](int r) { return r < rows ? (rows - r + rpar - 1) / rpar : 0; };
  const int cnt = pr < rpar ? slot_rows(pr) : 0;
  const int64_t o = (sample * length + pr) * C + c0 + c * V, step = (int64_t)rpar * C;
  constexpr int KEEP = ROWS > 0 ? ROWS : 1;
  GnRaw<TI, V> keep[KEEP];
  GnSums<V> t;
  if constexpr (ROWS > 0) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (i < cnt) keep[i].load(x + o + i * step);
    if (cnt > 0) t.start(keep, cnt);
  } else {
    gn_stream<TI, V>(x + o, step, cnt, t);
  }
  gn_put<MERGE>(pair_s, t, x + o, step, cnt, gn_least(eps), pr, c, cv);
  __syncthreads();
  const int P = gn_lanes(groups, T);
  for (int g0 = 0; g0 < groups; g0 += T / P) {
    const int g = g0 + (int)threadIdx.x / P;
    if (g >= groups) continue;  // lane groups of P leave together
    double n, mean, m2;
    gn_join_group<MERGE, V>(pair_s, g, cg, cv, min(rpar, rows), (int)threadIdx.x % P, P, slot_rows, n, mean, m2);
    if (threadIdx.x % P == 0) stat_s[g] = gn_stat(mean, m2, n, eps);
  }
  __syncthreads();
  if constexpr (ROWS == 0) {
    for (int ch = threadIdx.x; ch < w; ch += T) {
      const float2 st = stat_s[ch / cg];
      gn_write_coef(coef + sample * 3 * C, C, c0 + ch, st, weight, bias);
    }
  } else {
    if (cnt == 0) return;
    float mean[V], a[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 st = stat_s[(c * V + (MERGE ? 0 : e)) / cg];
      const int ch = c0 + c * V + e;
      mean[e] = st.x;
      a[e] = weight != nullptr ? st.y * weight[ch] : st.y;
      b[e] = bias != nullptr ? bias[ch] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (i < cnt) {
        float v[V];
        keep[i].get(v);
        gn_normalize<V>(v, mean, a, b, act);
        gn_store<TO, V>(y + o + i * step, v);
      }
  }
}

// Rotates and codes one 8-channel chunk (of block b; in: within the channels) of
// a row held by 16 lanes, and stores it.
__device__ __forceinline__ void gn_code_chunk(float (&y)[8], bool in, int lane, int hb, float c_b,
                                              uint8_t* __restrict__ codes, float* __restrict__ scale, int64_t row,
                                              int b, int chunk, int kb, int64_t total_rows) {
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = in ? y[e] : 0.0f;
  if (hb > 1) {
    const float sc = fwht8(y, lane, hb) * c_b;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = y[e] * sc;
  }
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, fabsf(y[e]));
  float s, inv;
  fp8_scales(row16_max(m), s, inv);
  // lanes past the channels (whole Hadamard blocks) hold rotated zeros of either sign
  *reinterpret_cast<uint2*>(codes + row * ((int64_t)kb * kFp8Block) + b * kFp8Block + 8 * chunk) =
      fp8_encode8(y, in ? inv : 0.0f);
  if ((lane & 15) == 0) scale[(int64_t)b * total_rows + row] = s;
}

// The normalization to FP8 codes: a wave owns one block of 128 channels of four
// rows at a time, a lane one 8-channel chunk (the one the rotation's lane
// numbering gives it), whose coefficients it keeps over the rows of its chunk.
// The loads of kGnRows row groups are in flight together.  (32 channels a lane,
// as in the quantizer, take 96 registers of coefficients: 20.1 us for 13 x 1350
// x 512, this form 11 to 12.)  That is 2.4 TB/s of the rows and codes: with 16
// rows a workgroup, a lane loads 96 bytes of coefficients for 64 of x.
template <typename TI, int HB, bool JOIN>
__global__ __launch_bounds__(kGnCodeThreads) void k_gn_apply_fp8(const TI* __restrict__ x, int64_t length, int C, int chunks,
                                                      int64_t rows_per, GnFrom from, int act, float c_b, int kb,
                                                      int64_t total_rows, uint8_t* __restrict__ codes,
                                                      float* __restrict__ scale) {
  extern __shared__ float2 pair_s[];  // JOIN: one (mean, rstd) per group
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15;
  const int kgroups = (kb + 3) >> 2;
  const unsigned blk = gridDim.x - 1 - blockIdx.x;
  const int b = (int)(blk % (unsigned)kgroups) * 4 + wave;
  const unsigned rest = blk / (unsigned)kgroups;
  const int64_t sample = rest / (unsigned)chunks;
  const int64_t r0 = (rest % (unsigned)chunks) * rows_per;
  const int rows = (int)min(rows_per, length - r0);
  const int cg = JOIN ? C / from.groups : 1;
  if constexpr (JOIN) gn_join_chunks<kGnCodeThreads>(from, sample, length, cg, pair_s);
  if (b >= kb) return;
  constexpr int NL = HB >= 16 ? HB / 8 : 1;
  const int chunk = (l16 & ~(NL - 1)) + fwht_chunk(lane, HB);
  const int ch = b * kFp8Block + 8 * chunk;
  const bool in = ch < C;  // C is a multiple of 8
  const int64_t row0 = sample * length + r0;
  const TI* p = x + row0 * C + (in ? ch : 0);
  float mean[8], a[8], bs[8];
  gn_coefs<8, JOIN>(from, sample, C, cg, in ? ch : 0, pair_s, mean, a, bs);
  for (int r = lane >> 4; r < rows; r += 4 * kGnRows) {  // 16 lanes stay together
    GnRaw<TI, 8> q[kGnRows];
#pragma unroll
    for (int u = 0; u < kGnRows; ++u)
      if (r + 4 * u < rows) q[u].load(p + (int64_t)(r + 4 * u) * C);
#pragma unroll
    for (int u = 0; u < kGnRows; ++u)
      if (r + 4 * u < rows) {
        float y[8];
        q[u].get(y);
        gn_normalize<8>(y, mean, a, bs, act);
        gn_code_chunk(y, in, lane, HB, c_b, codes, scale, row0 + r + 4 * u, b, chunk, kb, total_rows);
      }
  }
}

// Short samples to FP8 codes in one launch: a workgroup codes 16 rows, and works
// out the whole sample's statistics by itself first (so do the sample's other
// workgroups: a short sample's rows come from L2, and a launch, its workspace
// and its wait cost more).
template <typename TI, int V, bool MERGE>
__global__ __launch_bounds__(kGnThreads) void k_gn_short_fp8(const TI* __restrict__ x, int length, int C, int groups,
                                                             int chunks, float eps, const float* __restrict__ weight,
                                                             const float* __restrict__ bias, int act, int hb,
                                                             float c_b, int kb, int64_t total_rows,
                                                             uint8_t* __restrict__ codes, float* __restrict__ scale) {
  extern __shared__ float2 pair_s[];  // [rpar][C or cv], then one (mean, rstd) per group
  const int64_t sample = blockIdx.x / (unsigned)chunks;
  const int r0 = (int)(blockIdx.x % (unsigned)chunks) * 16;
  const int cv = C / V, rpar = kGnThreads / cv, cg = C / groups;
  const TI* xs = x + sample * length * C;
  float2* const stat_s = pair_s + ((rpar * (MERGE ? cv : C) + 1) & ~1);
  auto slot_rows = [&](int r) { return r < length ? (length - r + rpar - 1) / rpar : 0; };
  {
    const int pr = (int)threadIdx.x / cv, c = (int)threadIdx.x - pr * cv;
    GnSums<V> t;
    if (pr < rpar) {
      const TI* p = xs + (int64_t)pr * C + c * V;
      const int64_t step = (int64_t)rpar * C;
      const int cnt = slot_rows(pr);
      gn_stream<TI, V>(p, step, cnt, t);
      gn_put<MERGE>(pair_s, t, p, step, cnt, gn_least(eps), pr, c, cv);
    }
  }
  __syncthreads();
  const int P = gn_lanes(groups, kGnThreads);
  for (int g0 = 0; g0 < groups; g0 += kGnThreads / P) {
    const int g = g0 + (int)threadIdx.x / P;
    if (g >= groups) continue;  // lane groups of P leave together
    double n, mean, m2;
    gn_join_group<MERGE, V>(pair_s, g, cg, cv, min(rpar, length), (int)threadIdx.x % P, P, slot_rows, n, mean, m2);
    if (threadIdx.x % P == 0) stat_s[g] = gn_stat(mean, m2, n, eps);
  }
  __syncthreads();
  float* const coef_s = reinterpret_cast<float*>(stat_s + groups + (groups & 1));  // [3][C]
  for (int ch = threadIdx.x; ch < C; ch += kGnThreads) {
    const float2 st = stat_s[ch / cg];
    gn_write_coef(coef_s, C, ch, st, weight, bias);
  }
  // a wave codes four rows of a block of 128 channels at a time, as
  // k_gn_apply_fp8; the next four are loaded meanwhile
  const int lane = threadIdx.x & 63, l16 = lane & 15, nl = fwht_lanes(hb);
  const int chunk = (l16 & ~(nl - 1)) + fwht_chunk(lane, hb);
  constexpr int kWaves = kGnThreads / 64;
  auto load = [&](int u, GnRaw<TI, 8>& q) {
    const int row = r0 + 4 * (u & 3) + (lane >> 4), ch = (u >> 2) * kFp8Block + 8 * chunk;
    if (u < 4 * kb && row < length && ch < C) q.load(xs + (int64_t)row * C + ch);
  };
  GnRaw<TI, 8> next;
  int u = (int)threadIdx.x >> 6;
  load(u, next);
  __syncthreads();
  for (; u < 4 * kb; u += kWaves) {
    const GnRaw<TI, 8> q = next;
    load(u + kWaves, next);
    const int b = u >> 2, row = r0 + 4 * (u & 3) + (lane >> 4);
    if (row >= length) continue;  // 16 lanes stay together
    const int ch = b * kFp8Block + 8 * chunk;
    const bool in = ch < C;
    float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
      float mean[8], a[8], bs[8];
      gn_load_coef<8>(coef_s + ch, mean);
      gn_load_coef<8>(coef_s + C + ch, a);
      gn_load_coef<8>(coef_s + 2 * C + ch, bs);
      q.get(y);
      gn_normalize<8>(y, mean, a, bs, act);
    }
    gn_code_chunk(y, in, lane, hb, c_b, codes, scale, sample * length + row, b, chunk, kb, total_rows);
  }
}

// Enough for either input type: nothing when the slabs are kept (not the FP8
// form), else the coefficients, and the chunks' pairs unless the statistics are
// a slab's.
size_t group_norm_ws_bytes(int64_t n, int64_t length, int64_t C, int64_t groups, bool fp8) {
  size_t most = 0;
  for (const bool f32 : {false, true}) {
    const GnPlan p = gn_plan(n, length, C, groups, f32);
    if (fp8 ? p.brief : p.keep) continue;
    const size_t b = gn_coef_bytes(n, C) + (p.slab ? 0 : gn_align((size_t)(n * p.chunks * groups) * sizeof(double2)));
    if (b > most) most = b;
  }
  return most;
}

// Calls f with the vector length and the merge flag as constants.
template <typename TI, typename F>
static hipError_t gn_dispatch(const GnPlan& p, F f) {
  using std::integral_constant;
  if constexpr (sizeof(TI) == 2) {
    if (p.vec == 8)
      return p.merge ? f(integral_constant<int, 8>{}, std::true_type{}) : f(integral_constant<int, 8>{}, std::false_type{});
  }
  if (p.vec == 4)
    return p.merge ? f(integral_constant<int, 4>{}, std::true_type{}) : f(integral_constant<int, 4>{}, std::false_type{});
  return f(integral_constant<int, 1>{}, std::true_type{});  // one channel is in one group
}

template <typename TI, typename TO, int T, int ROWS>
static hipError_t gn_launch_slab(const GroupNormArgs& g, const GnPlan& p, void* y, float* coef, hipStream_t s) {
  return gn_dispatch<TI>(p, [&](auto v, auto merge) {
    constexpr int V = decltype(v)::value;
    constexpr bool MERGE = decltype(merge)::value;
    const int64_t cg = g.C / g.groups;
    // row slots x vectors are at most one per thread, in a narrower last slab too
    const size_t lds = ((size_t)T * (MERGE ? 1 : V) + (size_t)(p.width / cg)) * sizeof(float2);
    const hipError_t e = set_dynamic_lds_once<&k_gn_slab<TI, TO, V, MERGE, T, ROWS>>(kGnSlabLds);
    if (e != hipSuccess) return e;
    k_gn_slab<TI, TO, V, MERGE, T, ROWS><<<to_dim3(p.slab_grid), dim3(T), lds, s>>>(
        static_cast<const TI*>(g.x), g.length, (int)g.C, (int)cg, (int)p.width, (int)p.slabs, g.eps, g.weight, g.bias,
        g.act, static_cast<TO*>(y), coef);
    return hipGetLastError();
  });
}

// The statistics into ws: the coefficients of every sample and channel, or
// (p.join) the chunks' pairs.
template <typename TI>
static hipError_t gn_statistics(const GroupNormArgs& g, const GnPlan& p, void* ws, GnFrom& from, hipStream_t s) {
  float* coef = static_cast<float*>(ws);
  double2* part = reinterpret_cast<double2*>(static_cast<uint8_t*>(ws) + gn_coef_bytes(g.n, g.C));
  from = GnFrom{coef, part, (int)p.chunks, p.rows_per, (int)g.groups, g.eps, g.weight, g.bias};
  if (p.slab)
    return p.threads == 256 ? gn_launch_slab<TI, TI, 256, 0>(g, p, nullptr, coef, s)
                            : gn_launch_slab<TI, TI, kGnSlabThreads, 0>(g, p, nullptr, coef, s);
  const hipError_t e = gn_dispatch<TI>(p, [&](auto v, auto merge) {
    constexpr int V = decltype(v)::value;
    constexpr bool MERGE = decltype(merge)::value;
    const size_t lds = (size_t)(gn_rpar(g.C, V) * g.C) * sizeof(float2) / (MERGE ? V : 1);
    k_gn_partial<TI, V, MERGE><<<to_dim3(p.partial_grid), dim3(kGnThreads), lds, s>>>(
        static_cast<const TI*>(g.x), g.length, (int)g.C, (int)g.groups, (int)p.chunks, p.rows_per,
        gn_least(g.eps), part);
    return hipGetLastError();
  });
  if (e != hipSuccess || p.join) return e;
  k_gn_final<<<to_dim3(p.final_grid), dim3(kGnFinalThreads), 0, s>>>(
      part, g.n * g.groups, g.length, (int)(g.C / g.groups), (int)g.groups, (int)p.chunks, p.rows_per, g.eps, g.weight,
      g.bias, coef);
  return hipGetLastError();
}

template <typename TI, typename TO>
static hipError_t group_norm_t(const GroupNormArgs& g, void* y, void* ws, hipStream_t s) {
  const GnPlan p = gn_plan(g.n, g.length, g.C, g.groups, g.x_f32);
  if (p.keep) {
    if (p.rows <= 4) return gn_launch_slab<TI, TO, 256, 4>(g, p, y, nullptr, s);
    if (p.rows <= 8) return gn_launch_slab<TI, TO, 256, 8>(g, p, y, nullptr, s);
    return gn_launch_slab<TI, TO, 256, 16>(g, p, y, nullptr, s);
  }
  GnFrom from;
  const hipError_t e = gn_statistics<TI>(g, p, ws, from, s);
  if (e != hipSuccess) return e;
  return gn_dispatch<TI>(p, [&](auto v, auto) {
    constexpr int V = decltype(v)::value;
    const auto launch = [&](auto kernel, size_t lds) {
      kernel<<<to_dim3(p.apply_grid), dim3(kGnThreads), lds, s>>>(static_cast<const TI*>(g.x), g.length, (int)g.C,
                                                                  (int)p.apply_chunks, p.apply_rows, from, g.act,
                                                                  static_cast<TO*>(y));
      return hipGetLastError();
    };
    return p.join ? launch(&k_gn_apply<TI, TO, V, true>, (size_t)g.groups * sizeof(float2))
                  : launch(&k_gn_apply<TI, TO, V, false>, 0);
  });
}

// f(arguments, first sample) for every run of samples.
template <typename F>
static hipError_t gn_runs(const GroupNormArgs& g, F f) {
  const int64_t step = gn_run_samples(g.n, g.C);
  for (int64_t n0 = 0; n0 < g.n; n0 += step) {
    GroupNormArgs r = g;
    r.x = static_cast<const uint8_t*>(g.x) + n0 * g.length * g.C * (g.x_f32 ? 4 : 2);
    r.n = std::min(step, g.n - n0);
    const hipError_t e = f(r, n0);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_group_norm(const GroupNormArgs& g, void* y, bool y_f32, void* ws, hipStream_t s) {
  return gn_runs(g, [&](const GroupNormArgs& r, int64_t n0) {
    void* yr = static_cast<uint8_t*>(y) + n0 * g.length * g.C * (y_f32 ? 4 : 2);
    if (r.x_f32) return y_f32 ? group_norm_t<float, float>(r, yr, ws, s) : group_norm_t<float, uint16_t>(r, yr, ws, s);
    return y_f32 ? group_norm_t<uint16_t, float>(r, yr, ws, s) : group_norm_t<uint16_t, uint16_t>(r, yr, ws, s);
  });
}

template <typename TI, int HB>
static hipError_t gn_apply_fp8(const GroupNormArgs& g, const GnPlan& p, const GnFrom& from, uint8_t* codes,
                               float* scale, hipStream_t s) {
  const auto launch = [&](auto kernel, size_t lds) {
    kernel<<<to_dim3(p.code_grid), dim3(kGnCodeThreads), lds, s>>>(
        static_cast<const TI*>(g.x), g.length, (int)g.C, (int)p.code_chunks, p.code_rows, from, g.act,
        hadamard_scale(HB), (int)fp8_blocks(g.C), g.total_rows, codes, scale);
    return hipGetLastError();
  };
  return p.join ? launch(&k_gn_apply_fp8<TI, HB, true>, (size_t)g.groups * sizeof(float2))
                : launch(&k_gn_apply_fp8<TI, HB, false>, 0);
}

template <typename TI>
static hipError_t gn_short_fp8(const GroupNormArgs& g, const GnPlan& p, int hb, uint8_t* codes, float* scale,
                               hipStream_t s) {
  const int64_t chunks = (g.length + kGnBriefRows - 1) / kGnBriefRows;
  return gn_dispatch<TI>(p, [&](auto v, auto merge) {
    constexpr int V = decltype(v)::value;
    constexpr bool MERGE = decltype(merge)::value;
    if constexpr (V == 1 || (V == 4 && sizeof(TI) == 2)) {
      return hipErrorInvalidValue;  // channels are a multiple of 8
    } else {
      // pairs, (mean, rstd) of the groups, coefficients; 16-byte aligned
      const size_t pairs = (size_t)(kGnThreads / (g.C / V)) * (size_t)(MERGE ? g.C / V : g.C);
      const size_t lds = (pairs + (pairs & 1) + (size_t)(g.groups + (g.groups & 1))) * sizeof(float2) + (size_t)g.C * 3 * sizeof(float);
      const hipError_t e = set_dynamic_lds_once<&k_gn_short_fp8<TI, V, MERGE>>(kGnShortLds);
      if (e != hipSuccess) return e;
      k_gn_short_fp8<TI, V, MERGE><<<to_dim3(p.brief_grid), dim3(kGnThreads), lds, s>>>(
          static_cast<const TI*>(g.x), (int)g.length, (int)g.C, (int)g.groups, (int)chunks, g.eps, g.weight, g.bias,
          g.act, hb, hadamard_scale(hb), (int)fp8_blocks(g.C), g.total_rows, codes, scale);
      return hipGetLastError();
    }
  });
}

template <typename TI>
static hipError_t group_norm_fp8_t(const GroupNormArgs& g, int hb, uint8_t* codes, float* scale, void* ws,
                                   hipStream_t s) {
  const GnPlan p = gn_plan(g.n, g.length, g.C, g.groups, g.x_f32);
  if (p.brief) return gn_short_fp8<TI>(g, p, hb, codes, scale, s);
  GnFrom from;
  const hipError_t e = gn_statistics<TI>(g, p, ws, from, s);
  if (e != hipSuccess) return e;
  switch (hb) {
    case 1: return gn_apply_fp8<TI, 1>(g, p, from, codes, scale, s);
    case 2: return gn_apply_fp8<TI, 2>(g, p, from, codes, scale, s);
    case 4: return gn_apply_fp8<TI, 4>(g, p, from, codes, scale, s);
    case 8: return gn_apply_fp8<TI, 8>(g, p, from, codes, scale, s);
    case 16: return gn_apply_fp8<TI, 16>(g, p, from, codes, scale, s);
    case 32: return gn_apply_fp8<TI, 32>(g, p, from, codes, scale, s);
    case 64: return gn_apply_fp8<TI, 64>(g, p, from, codes, scale, s);
    case 128: return gn_apply_fp8<TI, 128>(g, p, from, codes, scale, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_group_norm_fp8(const GroupNormArgs& g, int hb, uint8_t* codes, float* scale, void* ws,
                                 hipStream_t s) {
  return gn_runs(g, [&](const GroupNormArgs& r, int64_t n0) {
    const int64_t row0 = n0 * g.length;
    uint8_t* cr = codes + row0 * fp8_blocks(g.C) * kFp8Block;
    return r.x_f32 ? group_norm_fp8_t<float>(r, hb, cr, scale + row0, ws, s)
                   : group_norm_fp8_t<uint16_t>(r, hb, cr, scale + row0, ws, s);
  });
}

}  // namespace hdq
