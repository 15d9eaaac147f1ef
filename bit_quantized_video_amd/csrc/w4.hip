// w4.hip -- linear layer of few tokens with 4-bit weights in groups (gfx950).
//
//   y[m, n] = sum over groups g of s[n, g] sum_{k in g} (u[n, k] - z[n, g]) x[m, k],
// u the codes 0 .. 15, z the group's zero point (8 without).  Bound by HBM: half
// a byte a weight, each read once.  The matrix instruction takes 16 rows x 32
// columns of weights and 32 columns of 16 tokens at a time; fewer tokens leave
// its other columns unused, at no cost beside the loads.  A code becomes bf16
// in one operation a pair: nibble u in bits 6..3 of a bf16 16.0 is 16 + u,
// exact, so the product is sum (16 + u) x - (16 + z) sum x, and sum x comes from a
// second product with ones; without zero points from one with -24, in whose
// registers the codes' product goes on.  Sums are float32, and a wanted (u - z) x is
// the difference of a (16 + u) x and a (16 + z) x: the error is a float32 sum's
// over terms (32 + u + z) |s x|.
// Measured: one token 512 -> 345600 with zero points 21.5 us, 4.5 TB/s of codes and
// scales; 12288 -> 12288 17.5 us, 4.4 TB/s; 1920 -> 5760 4.2 us, 1.3 TB/s (an empty
// launch is 1.5, the loads' latency another 1 to 1.5).
#include "hdq_device.h"
#include "hdq_internal.h"
#include "w4.h"

#include <type_traits>

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
  int wn, wk, per;  // k_w4: waves along rows and K, tiles of rows of a wave
  int step, part;   // its waves, in tokens of as many blocks and blocks
  int split;      // workgroups along K; above 1 each writes float32 sums to y + its number * slice
  int64_t slice;
};

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));

// Codes to bf16 16 + u: eight columns of a word, which is kept rotated left by 3
// bits, so that the first pair lies in place.  The constants are kept in vector
// registers: as literals they make two operations of each and-or.
__device__ __forceinline__ v8bf decode(uint32_t w) {
  uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
  asm("" : "+v"(mask), "+v"(sixteen));
  v4u r;
  r.x = (w & mask) | sixteen;
  r.y = ((w >> 4) & mask) | sixteen;
  r.z = ((w >> 8) & mask) | sixteen;
  r.w = (__builtin_rotateright32(w, 12) & mask) | sixteen;
  return __builtin_bit_cast(v8bf, r);
}

// Scales (bf16) and zero points (bytes) of a lane's row, l % 16, in COUNT groups.
template <int COUNT, bool ZERO>
struct Groups {
  uint16_t scale[COUNT];
  uint8_t zero[ZERO ? COUNT : 1];
  // from scalar bases on (buffers aligned to 16 bytes)
  __device__ __forceinline__ void load(const uint16_t* s, const uint8_t* z, uint32_t at) {
    __builtin_memcpy(scale, __builtin_assume_aligned(s + at, COUNT < 8 ? 2 * COUNT : 16), 2 * COUNT);
    if (ZERO) __builtin_memcpy(zero, __builtin_assume_aligned(z + at, COUNT), COUNT);
  }
};

// y += the tile's product; x(m, s): tokens 16 m .. + 15, columns 32 s .. + 31.  Of
// the lane's four results of an instruction, tokens 4 quad + r, the first R are
// wanted.  The tile's groups begin at group `at` of those loaded.
template <int MT, int NT, int R, int GROUPS, int COUNT, bool ZERO, typename X>
__device__ __forceinline__ void multiply(const v4u (&codes)[NT], const Groups<COUNT, ZERO> (&of)[NT], int at, const X& x,
                                         float (&y)[NT][MT][R]) {
  constexpr int STEPS = 4 / GROUPS;
  // ones, or without zero points the -24 itself, whose product the codes' then begins with
  constexpr uint32_t kSum = ZERO ? 0x3f803f80u : 0xc1c0c1c0u;
  const v8bf ones = __builtin_bit_cast(v8bf, v4u{kSum, kSum, kSum, kSum});
  const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < GROUPS; ++q) {
    v4f d[NT][MT], sum[MT];
    v8bf a[STEPS][MT];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        a[s][m] = x(m, q * STEPS + s);
        sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[s][m], ones, s == 0 ? none : sum[m], 0, 0, 0);
      }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const v8bf b = decode(codes[i][q * STEPS + s]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          d[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[s][m], b, s > 0 ? d[i][m] : ZERO ? none : sum[m], 0, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float sc = __uint_as_float((uint32_t)of[i].scale[at + q] << 16);
      const float off = ZERO ? 16.0f + (float)of[i].zero[ZERO ? at + q : 0] : 0.0f;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) y[i][m][r] = fmaf(sc, ZERO ? fmaf(-off, sum[m][r], d[i][m][r]) : d[i][m][r], y[i][m][r]);
    }
    // one group's products at a time: with all of a tile's the compiler runs out of registers
    if (MT > 1) __builtin_amdgcn_sched_barrier(0);
  }
}

// An output: token m, row n.
template <bool F32>
__device__ __forceinline__ void store(const W4Args& g, void* y, int64_t m, int64_t n, float v) {
  if (m >= g.M || n >= g.N) return;
  if (F32)
    static_cast<float*>(y)[m * g.N + n] = v;
  else
    static_cast<uint16_t*>(y)[m * g.N + n] = (uint16_t)pack_bf16x2(v, 0.0f);
}

// Up to 16 tokens whose columns fit LDS.  The workgroup keeps the tokens there
// (a row's pitch is 16 bytes past a multiple of 256: a fragment's 16 rows fall on
// all banks), and its waves stream weights in blocks of four tiles, 512
// columns of 16 rows, whose scales are one load; the next block is in flight.
//   wk = 1: a wave takes `per` tiles of rows, one after the other;
//   wk > 1: wk waves share a tile of rows, each taking every wk-th block of K,
//           and their sums meet in LDS, in order.
// Token 4 r + q is row 4 q + r of the product, so that R results a lane hold up
// to 4 R tokens (R = 4: at most 8 waves, more than 8 tokens' 28 tiles have no more blocks).
template <int R, int GROUPS, bool ZERO, bool F32>
__global__ __launch_bounds__(R == 4 ? 512 : 1024) void k_w4(const W4Args g) {
  extern __shared__ __align__(16) uint8_t s_lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / g.wk, wk = wave - wn * g.wk;
  const int col = lane & 15, quad = lane >> 4;
  const int tiles_k = (int)g.tiles_k, blocks = (tiles_k + 3) >> 2, pitch = tiles_k * 256 + 16;
  const int64_t tn0 = ((int64_t)blockIdx.x * g.wn + wn) * g.per;
  const int rows_here = (int)max((int64_t)0, min((int64_t)g.per, g.tiles_n - tn0));

  struct Block {
    v4u codes[4][1];
    Groups<4 * GROUPS, ZERO> of[1];
  };
  auto load = [&](Block& t, int64_t tn, int b) {
    const int64_t tile = tn * tiles_k + 4 * b, group = (tn * blocks + b) * (64 * GROUPS);
    t.of[0].load(g.scale + group, ZERO ? g.zero + group : nullptr, col * (4 * GROUPS));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * b + j < tiles_k) t.codes[j][0] = reinterpret_cast<const v4u*>(g.codes + (tile + j) * 1024)[lane];
  };
  // the wave's blocks: b = wk, wk + g.wk, ... of row tile tn, then of the next
  int64_t tn = tn0;
  int b = wk;
  int count = rows_here * ((blocks - wk + g.wk - 1) / g.wk);
  int64_t next_tn = tn0;
  int next_b = wk;
  auto advance = [&](int64_t& t, int& k) {
    k += g.wk;
    if (k >= blocks) k = wk, ++t;
  };
  Block ring[2];
  if (count > 0) load(ring[0], next_tn, next_b);

  // the tokens, zeros past the last column: 64 pieces of a token a wave at a time, four such loads in flight
  const int pieces = tiles_k * 16, filled = (int)(g.K / 8), tokens = (int)g.M;
  int m = 0, part = wave;
  while (part >= blocks) part -= blocks, ++m;
  while (m < tokens) {
    v4u v[4];
    int to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      to[j] = -1;
      if (m < tokens) {
        const int i = part * 64 + lane;
        if (i < pieces) to[j] = m * pitch + i * 16;
        v[j] = v4u{0u, 0u, 0u, 0u};
        if (i < filled) v[j] = *reinterpret_cast<const v4u*>(g.x + m * g.K + i * 8);
      }
      m += g.step;
      part += g.part;
      if (part >= blocks) part -= blocks, ++m;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (to[j] >= 0) *reinterpret_cast<v4u*>(s_lds + to[j]) = v[j];
  }
  __syncthreads();
  // rows of tokens that are not there repeat the first's, and are not stored
  const int token = (col & 3) * 4 + (col >> 2);
  const uint8_t* xr = s_lds + (token < g.M ? token : 0) * pitch + quad * 16;

  float y[1][1][R] = {};
  auto work = [&](const Block& t) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * b + j < tiles_k)
        multiply<1, 1, R, GROUPS>(t.codes[j], t.of, j * GROUPS, [&](int, int s) {
          return *reinterpret_cast<const v8bf*>(xr + (4 * b + j) * 256 + s * 64);
        }, y);
    const int64_t done = tn;
    advance(tn, b);
    if (g.wk == 1 && tn != done) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        store<F32>(g, g.y, 4 * r + quad, done * 16 + col, y[0][0][r]);
        y[0][0][r] = 0.0f;
      }
    }
  };
  for (; count > 0; count -= 2) {
    if (count > 1) advance(next_tn, next_b), load(ring[1], next_tn, next_b);
    work(ring[0]);
    if (count > 1) {
      if (count > 2) advance(next_tn, next_b), load(ring[0], next_tn, next_b);
      work(ring[1]);
    }
  }
  if (g.wk == 1) return;
  __syncthreads();  // the tokens are done with
  float* sums = reinterpret_cast<float*>(s_lds);  // [wn][wk][R][64]
#pragma unroll
  for (int r = 0; r < R; ++r) sums[(wave * R + r) * 64 + lane] = y[0][0][r];
  __syncthreads();
  if (wk != 0 || rows_here == 0) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float v = y[0][0][r];
    for (int k = 1; k < g.wk; ++k) v += sums[((wave + k) * R + r) * 64 + lane];
    store<F32>(g, g.y, 4 * r + quad, tn0 * 16 + col, v);
  }
}

// Few rows.  The workgroup has one tile of them, so it wants a fragment of the
// tokens once and LDS would serve no second reader; with 4 / MT tiles of K for
// each wave (16 fragments of the tokens, 64 registers) all its loads are in
// flight at once.  One launch where k_w4_shared takes two.  13 x 4096 -> 1921 in
// groups of 32 6.7 us (k_w4_shared 5.4 + 2.5), 16 x 1920 -> 1920 4.7 (k_w4 6.8).
// Bound by the tokens' way from L2 to the CU: 4096 -> 1921 takes 4.8 us with 1 token,
// 5.2 with 4, 6.0 with 8, 7.2 with 16, so 0.16 us and 8 KB a token, 50 bytes a ns and
// CU; a workgroup alone (16 rows) 3.5 with 1 token and 5.7 with 13, 256 of them 7.2.
template <int MT, int GROUPS, bool ZERO, bool F32>
__global__ __launch_bounds__(1024) void k_w4_direct(const W4Args g) {
  constexpr int TILES = 4 / MT;  // of K, a wave's
  extern __shared__ __align__(16) float s_sums[];  // [waves][MT][4][64]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int tiles_k = (int)g.tiles_k, k0 = wave * TILES;
  const int64_t tn = blockIdx.x;
  const int64_t group = tn * ((tiles_k + 3) >> 2) * (64 * GROUPS) + (k0 >> 2) * (64 * GROUPS) + (k0 & 3) * GROUPS;
  const uint8_t* codes = g.codes + (tn * tiles_k + k0) * 1024;
  // rows of tokens that are not there repeat the first's, and are not stored; columns past the last read zeros.
  // All of an offset is the lane's and the instruction's: a scalar one may lie past the end of a single short
  // token, and the range check takes it off the size.
  const uint32_t bytes = (uint32_t)(g.M * g.K * 2), k_bytes = (uint32_t)(g.K * 2), lane0 = k0 * 256 + quad * 16;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x, bytes);
  uint32_t from[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) from[m] = (16 * m + col < g.M ? 16 * m + col : 0) * k_bytes + lane0;
  v4u w[TILES][1];
  Groups<TILES * GROUPS, ZERO> of[1];
  uint4 x[TILES * 4][MT];
  of[0].load(g.scale + group, ZERO ? g.zero + group : nullptr, col * (4 * GROUPS));
#pragma unroll
  for (int j = 0; j < TILES; ++j)
    if (k0 + j < tiles_k) w[j][0] = reinterpret_cast<const v4u*>(codes + j * 1024)[lane];
#pragma unroll
  for (int i = 0; i < TILES * 4; ++i) {
    const bool in = lane0 + i * 64 < k_bytes;
#pragma unroll
    for (int m = 0; m < MT; ++m) x[i][m] = buf_load16(xr, (in ? from[m] : bytes) + i * 64, 0);
  }
  float y[1][MT][4] = {};
#pragma unroll
  for (int j = 0; j < TILES; ++j)
    if (k0 + j < tiles_k)
      multiply<MT, 1, 4, GROUPS>(w[j], of, j * GROUPS, [&](int m, int s) { return __builtin_bit_cast(v8bf, x[4 * j + s][m]); }, y);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) s_sums[((wave * MT + m) * 4 + r) * 64 + lane] = y[0][m][r];
  __syncthreads();
  for (int r = wave; r < 4 * MT; r += g.wk) {
    float v = s_sums[r * 64 + lane];
    for (int k = 1; k < g.wk; ++k) v += s_sums[(k * MT * 4 + r) * 64 + lane];
    store<F32>(g, g.y, 16 * (r >> 2) + 4 * quad + (r & 3), tn * 16 + col, v);
  }
}

// More tokens, or longer ones.  A workgroup of eight waves takes 16 MT MW tokens
// x 128 rows, 128 columns a stage; a wave multiplies MT tiles of tokens and NT
// of rows, MW waves sharing the rows.  The tokens lie in LDS in rows of 16
// pieces of 16 bytes, piece p of row r at p ^ (r % 16), so that a fragment's 16
// rows fall on all banks.  Loads run two stages ahead in registers (memory
// takes longer than a stage), none of them under a condition: the waits then
// count the ones that may still be in flight.
//
// 64 x 12288 -> 4096: 15.5 to 16.3 us and 4 for the sums (16.5 to 17.2 a call in a row
// of them, whose second launch overlaps the next call's first), 12 stages of 0.9 us and
// about 5 to begin and end.  A stage's parts are 650 cycles of vector
// instructions, 770 of matrix ones and 640 of LDS a SIMD or CU, of about 2000:
// what is left is waiting between them.  SIMD: waves a SIMD that the
// registers leave room for.  Four (128 registers, a few of them spilled) are
// faster for 64 tokens without zero points where a CU has a second workgroup to run
// (2000 x 1920 -> 5760 95 -> 80, 64 x 1024 -> 65536 18.8 -> 17.8) and slower where not
// (64 x 12288 -> 4096 15.9 -> 16.9); with zero points too much spills (64 x 1920 ->
// 1920 9.5 -> 13.5).  Loads at the top of a stage
// gain with one tile of tokens a wave (2 x 32768 -> 8192 37 -> 31) and cost
// registers with two (64 x 1024 -> 65536 17.4 -> 20).  Not kept: two halves of K
// in a workgroup of 16 waves (16.9 -> 16.2, shorter ones 5 to 10% slower), weights
// four or six stages ahead (16.5 -> 16.8, 17.4), stages of 256 columns, DMA into
// LDS (17).
template <int MW, int MT, int NT, int SIMD, int GROUPS, bool ZERO, bool F32>
__global__ __launch_bounds__(512, SIMD) void k_w4_shared(const W4Args g) {
  static_assert(NT * (8 / MW) == 8, "128 rows a workgroup");
  constexpr int TILES = MT * MW;            // of 16 tokens
  constexpr int PIECES = (TILES + 1) / 2;   // of the tokens a thread brings
  __shared__ __align__(16) uint8_t s_x[2][TILES * 4096];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4, wm = wave % MW;
  const int64_t tn0 = (int64_t)blockIdx.x * 8 + wave / MW * NT, m0 = (int64_t)blockIdx.y * (16 * TILES);
  const int each = (int)((g.tiles_k + g.split - 1) / g.split);
  const int k0 = (int)blockIdx.z * each, n = min(each, (int)g.tiles_k - k0);
  // The tiles of K go round from one that neighbours on the XCD do not start
  // with: rows of tokens a multiple of 4 KB apart, and tiles of weights, put
  // all that one tile reads on one or a few of L2's 16 channels.
  const unsigned id = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
  const int turn = (int)(((id >> 3) - (unsigned)k0) & 15u) % n;
  // scalar bases; the lane's part of an address is the same in every stage
  const uint8_t* codes[NT];
  const uint16_t* scale[NT];
  const uint8_t* zero[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t tile = tn0 + i < g.tiles_n ? tn0 + i : g.tiles_n - 1;  // past the end: the last again
    const int64_t block = tile * ((g.tiles_k + 3) >> 2);
    codes[i] = g.codes + tile * g.tiles_k * 1024;
    scale[i] = g.scale + block * (64 * GROUPS);
    zero[i] = ZERO ? g.zero + block * (64 * GROUPS) : nullptr;
  }
  // the workgroup's tokens: the thread's rows are tid / 16 + 32 j; pieces past the last token or column read zeros
  const int64_t here = g.M - m0 < 16 * TILES ? g.M - m0 : 16 * TILES;
  const uint32_t bytes = (uint32_t)(here * g.K * 2), k_bytes = (uint32_t)(g.K * 2);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + m0 * g.K, bytes);
  const int row = tid >> 4, piece = tid & 15;
  uint32_t from[PIECES];
#pragma unroll
  for (int j = 0; j < PIECES; ++j) from[j] = row + 32 * j < here ? (row + 32 * j) * k_bytes + piece * 16 : bytes;
  const int last = (int)g.tiles_k - 1;
  const bool past = (uint32_t)last * 256 + piece * 16 >= k_bytes;  // of the last tile
  struct Stage {
    v4u codes[NT];
    Groups<GROUPS, ZERO> of[NT];
    uint4 x[PIECES];
  };
  auto load = [&](Stage& t, int i_k) {
    i_k = min(i_k, n - 1) + turn;  // past the end: the last again
    const int kt = k0 + (i_k < n ? i_k : i_k - n);
    const int64_t at = (int64_t)(kt >> 2) * (64 * GROUPS) + (kt & 3) * GROUPS;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      t.codes[i] = reinterpret_cast<const v4u*>(codes[i] + (int64_t)kt * 1024)[lane];
      t.of[i].load(scale[i] + at, ZERO ? zero[i] + at : nullptr, col * (4 * GROUPS));
    }
#pragma unroll
    for (int j = 0; j < PIECES; ++j) t.x[j] = buf_load16(xr, past && kt == last ? bytes : from[j], kt * 256);
  };
  auto place = [&](const Stage& t, int kt) {
#pragma unroll
    for (int j = 0; j < PIECES; ++j)
      if (TILES % 2 == 0 || row < 16)
        *reinterpret_cast<uint4*>(&s_x[kt & 1][(row + 32 * j) * 256 + ((piece ^ (row & 15)) * 16)]) = t.x[j];
  };
  float y[NT][MT][4] = {};
  Stage w[3];
  load(w[0], 0);
  load(w[1], 1);
  place(w[0], 0);
  auto stage = [&](auto slot, int kt) {
    constexpr int H = decltype(slot)::value;
    lds_only_barrier();  // the stage's tokens are there, and the other half is read
    load(w[(H + 2) % 3], kt + 2);
    if (MT == 1) __builtin_amdgcn_sched_barrier(0);  // first: two whole stages to arrive in
    const uint8_t* xs = s_x[kt & 1] + wm * (MT * 4096) + col * 256;
    multiply<MT, NT, 4, GROUPS>(w[H].codes, w[H].of, 0, [&](int m, int s) {
      return *reinterpret_cast<const v8bf*>(xs + m * 4096 + (((4 * s + quad) ^ col) * 16));
    }, y);
    place(w[(H + 1) % 3], kt + 1);
  };
  int kt = 0;
  for (; kt + 2 < n; kt += 3) {
    stage(std::integral_constant<int, 0>(), kt);
    stage(std::integral_constant<int, 1>(), kt + 1);
    stage(std::integral_constant<int, 2>(), kt + 2);
  }
  if (kt < n) stage(std::integral_constant<int, 0>(), kt);
  if (kt + 1 < n) stage(std::integral_constant<int, 1>(), kt + 1);
  constexpr int kOut = F32 ? 4 : 2;
  const int64_t pitch = g.N * kOut, first = m0 + wm * (MT * 16) + quad * 4;
  char* out = static_cast<char*>(g.y) + (g.split > 1 ? blockIdx.z * g.slice * 4 : 0) + first * pitch + (tn0 * 16 + col) * kOut;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      char* p = out + (m * 16 + r) * pitch;
      if (first + m * 16 + r >= g.M) continue;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if ((tn0 + i) * 16 + col < g.N) {
          if (F32)
            reinterpret_cast<float*>(p)[i * 16] = y[i][m][r];
          else
            reinterpret_cast<uint16_t*>(p)[i * 16] = (uint16_t)pack_bf16x2(y[i][m][r], 0.0f);
        }
    }
}

// Sums of the splits, in order: 4 outputs a thread.
template <bool F32>
__global__ __launch_bounds__(256) void k_w4_join(const float* __restrict__ sums, int split, int64_t slice, int64_t count,
                                                 void* __restrict__ y) {
  const int64_t i = ((int64_t)wide_block() * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < split; k += 8) {  // eight loads in flight
    v4f part[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      part[u] = k + u < split ? *reinterpret_cast<const v4f*>(sums + (k + u) * slice + i) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < 8; ++u) v += part[u];
  }
  const v2u w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  if (i + 4 <= count) {
    if (F32)
      __builtin_memcpy(static_cast<float*>(y) + i, &v, 16);
    else
      __builtin_memcpy(static_cast<uint16_t*>(y) + i, &w, 8);
    return;
  }
  for (int r = 0; r < 3; ++r)
    if (i + r < count) {
      if (F32)
        static_cast<float*>(y)[i + r] = v[r];
      else
        static_cast<uint16_t*>(y)[i + r] = (uint16_t)(w[r >> 1] >> (16 * (r & 1)));
    }
}

// ---- weights ----------------------------------------------------------------

// Position of column e of eight in a packed word.
__device__ __forceinline__ int nibble(int e) { return (e >> 1) + 4 * (e & 1); }

// Codes in rows (bytes [N, K / 2], even columns in the low nibbles; scales and
// zero points [N, K / group]) to tiles: a lane's 16 bytes each.  Done once for a
// layer: 512 -> 345600 54 us, 3.5 TB/s; 12288 -> 4096 18.
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
      w[s] = __builtin_rotateleft32(w[s], 3);
    }
  }
  reinterpret_cast<uint4*>(out.codes)[tile * 64 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
  const int groups = 128 / group;
  // the row tile's last wave also clears the rest of its block of four tiles
  const int64_t end = tk + 1 == tiles_k ? (tiles_k + 3) / 4 * 4 : tk + 1;
  for (int64_t k = tk; k < end; ++k) {
    if (lane >= 16 * groups) break;
    const int64_t n = lane / groups, r = tn * 16 + n, kg = k * groups + lane % groups, kgs = K / group;
    const int64_t at = w4_group_at(tn, n, kg, tiles_k, groups);
    const bool in = r < N && kg < kgs;
    out.scale[at] = in ? scale[r * kgs + kg] : (uint16_t)0;
    if (out.zero != nullptr) out.zero[at] = in ? zero[r * kgs + kg] : (uint8_t)0;
  }
}

// bf16 weights to tiles, a thread for each group of a row:
//   without zero points  s = bf16(max|w| / 7), u = clamp(rne(w / s), -8, 7) + 8;
//   with                 s = bf16((max - min) / 15) (0 among the values),
//                        z = rne(-min / s), u = clamp(rne(w / s) + z, 0, 15).
// A group below 2^-100 gets s = 0; one with a NaN or an infinity s = NaN.
// Done once for a layer, and simple: neighbouring lanes read a group apart, twice.
// 12288 -> 12288 in groups of 32 190 us, 2.1 TB/s; 512 -> 345600 in groups of 64 755 us
// and 12288 -> 4096 in groups of 128 240, 0.6 and 0.5 TB/s.
__global__ __launch_bounds__(256) void k_w4_quantize(const uint16_t* __restrict__ src, int64_t N, int64_t K, int group,
                                                     int64_t tiles_n, int64_t tiles_k, W4Out out) {
  const int groups = 128 / group;
  const int64_t kgs = (tiles_k + 3) / 4 * 4 * groups, id = (int64_t)wide_block() * 256 + threadIdx.x;
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
  const int64_t at = w4_group_at(row >> 4, n, kg, tiles_k, groups);
  out.scale[at] = finite ? (s > 0.0f ? (uint16_t)bits : (uint16_t)0) : (uint16_t)0x7fc0;
  if (zp) out.zero[at] = in ? (uint8_t)z : (uint8_t)0;
  if (kg >= tiles_k * groups) return;
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
    reinterpret_cast<uint32_t*>(out.codes)[(tile * 64 + ((k >> 3) & 3) * 16 + n) * 4 + (k >> 5)] = __builtin_rotateleft32(w, 3);
  }
}

template <int GROUPS, bool ZERO, bool F32>
void run(const W4Args& a, const W4Plan& p, hipStream_t s) {
  const dim3 grid((unsigned)p.grid_x, (unsigned)p.grid_y, (unsigned)p.split), block((unsigned)(64 * p.wn * p.wk));
  if (p.per > 0 && a.M <= 4)
    k_w4<1, GROUPS, ZERO, F32><<<grid, block, p.lds, s>>>(a);
  else if (p.per > 0 && a.M <= 8)
    k_w4<2, GROUPS, ZERO, F32><<<grid, block, p.lds, s>>>(a);
  else if (p.per > 0)
    k_w4<4, GROUPS, ZERO, F32><<<grid, block, p.lds, s>>>(a);
  else if (p.direct && p.mt == 1)
    k_w4_direct<1, GROUPS, ZERO, F32><<<grid, block, p.lds, s>>>(a);
  else if (p.direct && p.mt == 2)
    k_w4_direct<2, GROUPS, ZERO, F32><<<grid, block, p.lds, s>>>(a);
  else if (p.direct)
    k_w4_direct<4, GROUPS, ZERO, F32><<<grid, block, p.lds, s>>>(a);
  else if (p.mt == 4 && !ZERO && p.grid_x * p.grid_y * p.split > kW4Groups)
    k_w4_shared<2, 2, 2, ZERO ? 2 : 4, GROUPS, ZERO, F32><<<grid, block, 0, s>>>(a);
  else if (p.mt == 4)
    k_w4_shared<2, 2, 2, 2, GROUPS, ZERO, F32><<<grid, block, 0, s>>>(a);
  else if (p.mt == 2)
    k_w4_shared<2, 1, 2, 2, GROUPS, ZERO, F32><<<grid, block, 0, s>>>(a);
  else
    k_w4_shared<1, 1, 1, 2, GROUPS, ZERO, F32><<<grid, block, 0, s>>>(a);
}

template <bool F32>
void run_group(const W4Args& a, const W4Plan& p, int group, hipStream_t s) {
  const bool z = a.zero != nullptr;
  switch (group) {
    case 32: return z ? run<4, true, F32>(a, p, s) : run<4, false, F32>(a, p, s);
    case 64: return z ? run<2, true, F32>(a, p, s) : run<2, false, F32>(a, p, s);
    default: return z ? run<1, true, F32>(a, p, s) : run<1, false, F32>(a, p, s);
  }
}

}  // namespace

hipError_t launch_w4(const uint16_t* x, int64_t M, const W4Weights& w, void* y, bool f32, void* ws, hipStream_t s) {
  const W4Plan p = plan_w4(M, w.N, w.K);
  const bool join = p.split > 1;
  const int64_t slice = w4_slice(M, w.N), count = M * w.N;
  const W4Args a{x, w.codes, w.scale, w.zero, join ? ws : y, M, w.N, w.K, w4_tiles_n(w.N), w4_tiles_k(w.K),
                 p.wn, p.wk, p.per, p.step, p.part, p.split, slice};
  f32 || join ? run_group<true>(a, p, w.group, s) : run_group<false>(a, p, w.group, s);
  if (join) {
    const dim3 grid = wide_grid((count + 1023) / 1024);
    if (f32)
      k_w4_join<true><<<grid, dim3(256), 0, s>>>(static_cast<const float*>(ws), p.split, slice, count, y);
    else
      k_w4_join<false><<<grid, dim3(256), 0, s>>>(static_cast<const float*>(ws), p.split, slice, count, y);
  }
  return hipGetLastError();
}

hipError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scale, const uint8_t* zero, int64_t N, int64_t K,
                          int group, const W4Out& out, hipStream_t s) {
  const int64_t tiles = w4_tiles_n(N) * w4_tiles_k(K);
  k_w4_pack<<<wide_grid((tiles + 3) / 4), dim3(256), 0, s>>>(codes, scale, zero, N, K, group, w4_tiles_k(K), tiles, out);
  return hipGetLastError();
}

hipError_t launch_w4_quantize(const uint16_t* w, int64_t N, int64_t K, int group, const W4Out& out, hipStream_t s) {
  const int64_t tn = w4_tiles_n(N), tk = w4_tiles_k(K), threads = tn * 16 * ((tk + 3) / 4 * 4) * (128 / group);
  k_w4_quantize<<<wide_grid((threads + 255) / 256), dim3(256), 0, s>>>(w, N, K, group, tn, tk, out);
  return hipGetLastError();
}

}  // namespace hdq
