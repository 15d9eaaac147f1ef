// gemm_fp8.hip -- FP8 block-128 linear layers on gfx950.
//
// Operands, product forms and accuracy: gemm_fp8_tile.h.
#include "gemm_fp8_pipe.h"

namespace hdq {

// At most 16 tokens (single-token serving): no LDS staging of the weights and no
// barrier in the K loop.  A workgroup owns 16 features; its WAVES waves take the
// blocks of K in turn (wave w: w, w + WAVES, ...), each reading its weight
// fragments from global memory straight into registers one block ahead, and
// the partial tiles are added over LDS in a fixed order.  Bound by the weights'
// bytes, and for small layers by the launch: one token, 3072 -> 12288 8.4 us (4.5
// TB/s), 12288 -> 3072 9.4, 1920 -> 5760 4.5 from codes and 5.5 from bf16.
//
// HB > 0: the activations come as bf16 and the workgroup quantizes them itself
// (rotation block HB), into LDS, while its first weights are on their way: the
// same codes as k_fp8_quant_rows', without a launch and a workspace.  One pass
// of its threads has to do, M x kb <= 16 WAVES row blocks.
template <int OUT, int WAVES, int HB>
__global__ __launch_bounds__(64 * WAVES) void k_fp8_few(const uint8_t* __restrict__ xc, const float* __restrict__ xs,
                                                        const uint16_t* __restrict__ xb, int K, float c_b,
                                                        const uint8_t* __restrict__ wc, const float* __restrict__ ws,
                                                        void* __restrict__ Y, int M, int N, int kb) {
  constexpr bool FAST = OUT == kOutBf16;
  constexpr int XBLOCKS = HB > 0 ? 16 * WAVES : 1;
  __shared__ v4f part[WAVES / 2][64];
  __shared__ __attribute__((aligned(16))) uint8_t xcodes[XBLOCKS * kFp8Block];
  __shared__ float xscale[XBLOCKS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int n0 = (int)wide_block() * 16;
  if (n0 >= N) return;
  const int64_t ld = (int64_t)kb * kFp8Block;
  // rows past the end repeat the last one; their results are not stored
  const int m = min(r16, M - 1);
  const uint8_t* xp = HB > 0 ? nullptr : xc + m * ld + 16 * q;
  const uint8_t* wp = wc + (int64_t)min(n0 + r16, N - 1) * ld + 16 * q;
  // the tile's features lie in one block row of the weights' scales
  const float* wsp = ws + (int64_t)(n0 / kFp8Block) * kb;

  struct Block {
    Fp8Frag x, w;
    float s;
  };
  auto load_w = [&](Block& b, int k) {
    const int64_t o = (int64_t)k * kFp8Block;
    b.w = load_frag(wp + o, wp + o + 64);
    b.s = wsp[k];
  };
  auto load_x = [&](Block& b, int k) {
    if constexpr (HB > 0) {
      const uint8_t* p = xcodes + (m * kb + k) * kFp8Block + 16 * q;
      b.x = load_frag(p, p + 64);
      b.s *= xscale[m * kb + k];
    } else {
      const int64_t o = (int64_t)k * kFp8Block;
      b.x = load_frag(xp + o, xp + o + 64);
      b.s *= xs[(int64_t)k * M + m];
    }
  };
  v4f acc = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto compute = [&](const Block& b) {
    Fp8Operand<FAST> w, x;
    w.set(b.w);
    x.set(b.x);
    add_scaled(acc, block_product(w, x), b.s);
  };
  Block b0, b1;
  int k = wave;
  if (k < kb) load_w(b0, k);
  if constexpr (HB > 0) {
    const int rb = threadIdx.x >> 2, part4 = threadIdx.x & 3;  // a quad per row block
    if (rb < M * kb) {
      const int row = rb / kb, b = rb - row * kb;
      float y[32];
      load_row32(reinterpret_cast<const uint4*>(xb + (int64_t)row * K), b * 16 + part4 * 4, K >> 3, y);
      rotate32<HB>(y, lane, c_b);
      float s, inv;
      fp8_scales(quad_max(absmax32(y)), s, inv);
      uint4 out[2];
      fp8_encode32(y, b * kFp8Block + part4 * 32 < K ? inv : 0.0f, out);
      uint4* dst = reinterpret_cast<uint4*>(xcodes + rb * kFp8Block + part4 * 32);
      dst[0] = out[0];
      dst[1] = out[1];
      if (part4 == 0) xscale[rb] = s;
    }
    __syncthreads();
  }
  if (k < kb) load_x(b0, k);
  while (k < kb) {
    if (k + WAVES < kb) {
      load_w(b1, k + WAVES);
      load_x(b1, k + WAVES);
    }
    compute(b0);
    k += WAVES;
    if (k >= kb) break;
    if (k + WAVES < kb) {
      load_w(b0, k + WAVES);
      load_x(b0, k + WAVES);
    }
    compute(b1);
    k += WAVES;
  }
  // halving sum over the waves: wave w adds wave w + h
#pragma unroll
  for (int h = WAVES / 2; h >= 1; h >>= 1) {
    if (wave >= h && wave < 2 * h) part[wave - h][lane] = acc;
    __syncthreads();
    if (wave < h) acc += part[wave][lane];
    __syncthreads();
  }
  if (wave == 0 && r16 < M) store_out4<OUT>(Y, r16, n0 + 4 * q, N, acc);
}

constexpr int kFewWaves = 8;

template <int OUT, int HB>
static hipError_t launch_few(const uint8_t* xc, const float* xs, const uint16_t* xb, int64_t K, const uint8_t* wc,
                             const float* ws, void* y, int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  k_fp8_few<OUT, kFewWaves, HB><<<wide_grid((N + 15) / 16), dim3(64 * kFewWaves), 0, s>>>(
      xc, xs, xb, (int)K, HB > 0 ? hadamard_scale(HB) : 1.0f, wc, ws, y, (int)M, (int)N, (int)kb);
  return hipGetLastError();
}

bool gemm_fp8_quantizes(int64_t M, int64_t kb) { return M <= 16 && M * kb <= 16 * kFewWaves; }

template <int OUT>
static hipError_t launch_few_bf16(const uint16_t* x, int64_t K, int hb, const uint8_t* wc, const float* ws, void* y,
                                  int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  switch (hb) {
    case 1: return launch_few<OUT, 1>(nullptr, nullptr, x, K, wc, ws, y, M, N, kb, s);
    case 2: return launch_few<OUT, 2>(nullptr, nullptr, x, K, wc, ws, y, M, N, kb, s);
    case 4: return launch_few<OUT, 4>(nullptr, nullptr, x, K, wc, ws, y, M, N, kb, s);
    case 8: return launch_few<OUT, 8>(nullptr, nullptr, x, K, wc, ws, y, M, N, kb, s);
    case 16: return launch_few<OUT, 16>(nullptr, nullptr, x, K, wc, ws, y, M, N, kb, s);
    case 32: return launch_few<OUT, 32>(nullptr, nullptr, x, K, wc, ws, y, M, N, kb, s);
    case 64: return launch_few<OUT, 64>(nullptr, nullptr, x, K, wc, ws, y, M, N, kb, s);
    case 128: return launch_few<OUT, 128>(nullptr, nullptr, x, K, wc, ws, y, M, N, kb, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_gemm_fp8_bf16(const uint16_t* x, int64_t K, int hb, const uint8_t* wc, const float* ws, void* y,
                                int out_dtype, int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  if (!gemm_fp8_quantizes(M, kb)) return hipErrorNotSupported;
  return out_dtype == kOutBf16 ? launch_few_bf16<kOutBf16>(x, K, hb, wc, ws, y, M, N, kb, s)
                               : launch_few_bf16<kOutF32>(x, K, hb, wc, ws, y, M, N, kb, s);
}

// Middle sizes: one tile of 32 WM_T x 32 WN_T per workgroup, KW groups of 2 x 2
// waves that take the blocks of K in turn, and STAGES LDS buffers of KW blocks
// filled by LDS-DMA STAGES - 1 stages ahead: with few workgroups a stage's
// arithmetic is much shorter than its loads' latency.  PROD: waves of their own
// issue the loads (a wave is held up while it issues; 5-15% faster with one
// group).  The groups' partial tiles are added over LDS in a fixed order.  Bound
// by the operands' way into LDS: 226 x 4096 -> 1920 takes 8.2 to 9.3 us (direct
// loads without LDS 25.5), in which each of its 240 workgroups brings 478 KB, 24 to
// 28 bytes per clock and CU, more than the large tiles reach; a fifth of that
// are the loads past its last stage.  1350 x 1920 -> 1024: 10.0.
template <int WM_T, int WN_T, int KW, int STAGES, bool PROD>
struct Fp8Deep {
  static constexpr int BM = 32 * WM_T, BN = 32 * WN_T, THREADS = 256 * KW * (PROD ? 2 : 1);
  static constexpr int BLOCK = (BM + BN) * kFp8Block + 1024;  // a block's codes and 256 scale slots
  static constexpr int STAGE = KW * BLOCK, LDS = STAGES * STAGE;
  static constexpr int LOADS = (BM + BN) / 32 + 1;            // LDS-DMA instructions per wave and stage
  static_assert(BM <= 256 && LDS <= 160 * 1024 && LOADS * (STAGES - 2) < 64, "tile shape");
  static_assert((KW - 1) * BM * BN * 4 <= LDS, "the groups' partial tiles fit");
};

template <int OUT, int WM_T, int WN_T, int KW, int STAGES, bool PROD>
__global__ __launch_bounds__(256 * KW * (PROD ? 2 : 1)) void k_fp8_deep(const uint8_t* __restrict__ xc, const float* __restrict__ xs,
                                                       const uint8_t* __restrict__ wc, const float* __restrict__ ws,
                                                       void* __restrict__ Y, int64_t M, int N, int kb) {
  using Tile = Fp8Deep<WM_T, WN_T, KW, STAGES, PROD>;
  constexpr bool FAST = OUT == kOutBf16;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = (wave >> 2) % KW, wq = wave & 3, wm = wq & 1, wn = wq >> 1;
  const int r16 = lane & 15, q = lane >> 4;
  int tm, tn;
  xcd_tile((int)((M + Tile::BM - 1) / Tile::BM), (N + Tile::BN - 1) / Tile::BN, tm, tn);
  const int64_t m0 = (int64_t)tm * Tile::BM;
  const int n0 = tn * Tile::BN, ld = kb * kFp8Block;
  const uint32_t mrows = (uint32_t)min((int64_t)Tile::BM, M - m0);
  const __amdgpu_buffer_rsrc_t xres = make_rsrc(xc + m0 * ld, mrows * (uint32_t)ld);
  const __amdgpu_buffer_rsrc_t wres = make_rsrc(wc + (int64_t)n0 * ld, (uint32_t)min(Tile::BN, N - n0) * (uint32_t)ld);
  const int stages = (kb + KW - 1) / KW;

  // A group's four waves load its block: instruction p of wave wq fills rows
  // 32 p + 8 wq + (lane >> 3), slot lane & 7.  Blocks past the last one read
  // other rows' bytes or zeros, and are not computed.
  const int drow = 8 * wq + (lane >> 3);
  const uint32_t dvoff = (uint32_t)(drow * ld + 16 * ((lane & 7) ^ (drow & 7)));
  auto issue = [&](int buf, int stage) {
    const int k = stage * KW + kw;
    uint8_t* base = smem + buf * Tile::STAGE + kw * Tile::BLOCK;
#pragma unroll
    for (int p = 0; p < Tile::BM / 32; ++p) lds_dma16(xres, base + 4096 * p + 1024 * wq, dvoff, k * kFp8Block + p * 32 * ld);
#pragma unroll
    for (int p = 0; p < Tile::BN / 32; ++p)
      lds_dma16(wres, base + Tile::BM * kFp8Block + 4096 * p + 1024 * wq, dvoff, k * kFp8Block + p * 32 * ld);
    const __amdgpu_buffer_rsrc_t sres = make_rsrc(xs + (int64_t)min(k, kb - 1) * M + m0, mrows * 4u);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        sres, (__attribute__((address_space(3))) void*)(base + (Tile::BM + Tile::BN) * kFp8Block + 256 * wq), 4,
        4 * (64 * wq + lane), 0, 0, 0);
  };

  v4f acc[WM_T][WN_T];
#pragma unroll
  for (int i = 0; i < WM_T; ++i)
#pragma unroll
    for (int j = 0; j < WN_T; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  // scalar loads, which do not wait for the DMA loads in flight
  typedef const __attribute__((address_space(4))) float* ConstFloats;
  const int nb = min((n0 + wn * 16 * WN_T) / kFp8Block, (N + kFp8Block - 1) / kFp8Block - 1);
  const ConstFloats wsp = (ConstFloats)(uintptr_t)ws + (int64_t)nb * kb;

  auto frag = [&](const uint8_t* rows, int r) {
    return load_frag(rows + r * 128 + 16 * (q ^ (r & 7)), rows + r * 128 + 16 * ((q + 4) ^ (r & 7)));
  };
  auto compute = [&](int buf, float sw) {
    const uint8_t* lx = smem + buf * Tile::STAGE + kw * Tile::BLOCK;
    const uint8_t* lw = lx + Tile::BM * kFp8Block;
    const float* ls = reinterpret_cast<const float*>(lw + Tile::BN * kFp8Block) + wm * 16 * WM_T + r16;
    Fp8Frag xf[WM_T], wf[WN_T];
    float sx[WM_T];
#pragma unroll
    for (int j = 0; j < WN_T; ++j) wf[j] = frag(lw, wn * 16 * WN_T + 16 * j + r16);
#pragma unroll
    for (int i = 0; i < WM_T; ++i) {
      xf[i] = frag(lx, wm * 16 * WM_T + 16 * i + r16);
      sx[i] = ls[16 * i];
    }
    __builtin_amdgcn_sched_barrier(0);
    // fragment i's products run while fragment i - 1's are scaled and added
    Fp8Operand<FAST> w[WN_T];
    v4f p[2][WN_T];
#pragma unroll
    for (int i = 0; i <= WM_T; ++i) {
      Fp8Operand<FAST> x;
      if (i < WM_T) x.set(xf[i]);
#pragma unroll
      for (int j = 0; j < WN_T; ++j) {
        if (i == 0) w[j].set(wf[j]);
        if (i < WM_T) p[i & 1][j] = block_product(w[j], x);
        if (i > 0) add_scaled(acc[i - 1][j], p[(i - 1) & 1][j], sx[i - 1] * sw);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // Stage g lives in buffer g % STAGES.  At its end at most the STAGES - 2
  // stages after the next one are in flight (loads land in order), so after the
  // barrier the next stage is in LDS and this one's buffer is free.
  const bool loads = !PROD || wave >= 4 * KW, computes = !PROD || wave < 4 * KW;
  if (loads) {
#pragma unroll
    for (int g = 0; g < STAGES - 1; ++g) issue(g, g);
    wait_vmem<Tile::LOADS*(STAGES - 2)>();
  }
  float sw = wsp[min(kw, kb - 1)];
  lds_only_barrier();
  for (int g0 = 0; g0 < stages; g0 += STAGES) {
#pragma unroll
    for (int u = 0; u < STAGES; ++u) {
      const int g = g0 + u;
      if (g < stages) {
        // past the end these loads are of no use, but keep the count of loads in flight
        if (loads) issue((u + STAGES - 1) % STAGES, g + STAGES - 1);
        if (computes && g * KW + kw < kb) compute(u, sw);
        sw = wsp[min((g + 1) * KW + kw, kb - 1)];
        if (loads) wait_vmem<Tile::LOADS*(STAGES - 2)>();
        lds_only_barrier();
      }
    }
  }
  if (PROD && !computes && KW == 1) {
    wait_vmem<0>();
    return;
  }
  if constexpr (KW > 1) {
    // the loads past the end have to land before their buffers are written
    wait_vmem<0>();
    lds_only_barrier();
    v4f* part = reinterpret_cast<v4f*>(smem);
    if (computes && kw > 0) {
#pragma unroll
      for (int i = 0; i < WM_T; ++i)
#pragma unroll
        for (int j = 0; j < WN_T; ++j) part[(((kw - 1) * 4 + wq) * WM_T * WN_T + i * WN_T + j) * 64 + lane] = acc[i][j];
    }
    lds_only_barrier();
    if (!computes || kw > 0) return;
#pragma unroll
    for (int g = 1; g < KW; ++g)
#pragma unroll
      for (int i = 0; i < WM_T; ++i)
#pragma unroll
        for (int j = 0; j < WN_T; ++j) acc[i][j] += part[(((g - 1) * 4 + wq) * WM_T * WN_T + i * WN_T + j) * 64 + lane];
  } else {
    wait_vmem<0>();
  }
#pragma unroll
  for (int i = 0; i < WM_T; ++i) {
    const int64_t m = m0 + wm * 16 * WM_T + 16 * i + r16;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < WN_T; ++j) store_out4<OUT>(Y, m, n0 + wn * 16 * WN_T + 16 * j + 4 * q, N, acc[i][j]);
  }
}

template <int OUT, int WM_T, int WN_T, int KW, int STAGES, bool PROD>
static hipError_t launch_deep(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws, void* y,
                              int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  using Tile = Fp8Deep<WM_T, WN_T, KW, STAGES, PROD>;
  const int64_t tiles = ((M + Tile::BM - 1) / Tile::BM) * ((N + Tile::BN - 1) / Tile::BN);
  if (tiles > 0x7fffffff) return hipErrorInvalidValue;
  const hipError_t e = set_dynamic_lds_once<&k_fp8_deep<OUT, WM_T, WN_T, KW, STAGES, PROD>>(Tile::LDS);
  if (e != hipSuccess) return e;
  k_fp8_deep<OUT, WM_T, WN_T, KW, STAGES, PROD>
      <<<dim3((unsigned)tiles), dim3(Tile::THREADS), Tile::LDS, s>>>(xc, xs, wc, ws, y, M, (int)N, (int)kb);
  return hipGetLastError();
}

template <int OUT, int WM_T, int WN_T>
__global__ __launch_bounds__(kPipeThreads, 2) void k_fp8_pipe(const uint8_t* __restrict__ xc, const float* __restrict__ xs,
                                                              const uint8_t* __restrict__ wc,
                                                              const float* __restrict__ ws, void* __restrict__ Y,
                                                              int64_t M, int N, int kb) {
  gemm_fp8_pipe_body<OUT, WM_T, WN_T>(xc, xs, wc, ws, Y, M, N, kb);
}

constexpr int64_t kPipeSlots = 256;  // workgroups that run at a time, one per CU
template <int OUT, int WM_T, int WN_T>
static hipError_t launch_pipe(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws, void* y,
                              int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  using Tile = Fp8Tile<WM_T, WN_T>;
  const int64_t tiles = ((M + Tile::BM - 1) / Tile::BM) * ((N + Tile::BN - 1) / Tile::BN);
  if (tiles > 0x7fffffff) return hipErrorInvalidValue;
  const hipError_t e = set_dynamic_lds_once<&k_fp8_pipe<OUT, WM_T, WN_T>>(Tile::LDS);
  if (e != hipSuccess) return e;
  // as few workgroups as keep the number of rounds, a multiple of 8 (XCDs)
  const int64_t rounds = (tiles + kPipeSlots - 1) / kPipeSlots;
  const int64_t grid = tiles <= kPipeSlots ? tiles : ((tiles + rounds - 1) / rounds + 7) / 8 * 8;
  k_fp8_pipe<OUT, WM_T, WN_T>
      <<<dim3((unsigned)grid), dim3(kPipeThreads), Tile::LDS, s>>>(xc, xs, wc, ws, y, M, (int)N, (int)kb);
  return hipGetLastError();
}

// Which kernel: by how many tiles of each size there are for the 256 CUs.
// Measured on both sides of each border, each pair on one card, cards differing by
// up to 10% (us, bf16 output, N x K in brackets):
//  * up to 16 tokens: k_fp8_few 6.0, 32 x 64 tiles 5.8 (16, 5760 x 1920); one
//    token 4.9 / 5.8.
//  * fewer than 192 tiles of 64 x 64: 32 x 64 tiles with four K groups 6.2, 64 x
//    64 tiles 7.2 (64 tokens, 5760 x 1920), 8.8 / 12.0 (226, 1920 x 4096); with
//    256 of them (1024, 1024 x 1024) 8.8 / 5.6.
//  * fewer than 800 tiles of 64 x 64 (fp32 output: 1300): 64 x 64 tiles 15.3, 128
//    x 256 tiles 17.9 (450, 5760 x 1920: 720 tiles), fp32 21.1 / 31.4; with 832 (800,
//    4096 x 512) 10.2 / 8.8, fp32 with 1320 (1350, 3840 x 1024) 23.3 / 21.6.
//  * 128 x 256 tiles or 256 x 256 ones: by rounds of 256 tiles, a 128 x 256 round
//    priced at 5 / 8 of the other.  1 round and 1 (1350, 5760 x 1920) 19.9 / 27.1,
//    3 and 2 (4050, 5760 x 1920) 53.7 / 53.3, fp32 94 / 102; 2 and 1 (3000, 4096 x 1024)
//    21.8 / 19.9, fp32 37.9 / 34.4; 13 and 7 (17776, 5760 x 1920) 231 / 208.
template <int OUT>
static hipError_t launch_fp8_out(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws, void* y,
                                 int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  const auto tiles = [&](int64_t m, int64_t n) { return ((M + m - 1) / m) * ((N + n - 1) / n); };
  const auto rounds = [&](int64_t m, int64_t n) { return (tiles(m, n) + kPipeSlots - 1) / kPipeSlots; };
  if (M <= 16) return launch_few<OUT, 0>(xc, xs, nullptr, 0, wc, ws, y, M, N, kb, s);
  if (tiles(64, 64) < 192) return launch_deep<OUT, 1, 2, 4, 3, false>(xc, xs, wc, ws, y, M, N, kb, s);
  if (tiles(64, 64) < (OUT == kOutBf16 ? 800 : 1300)) return launch_deep<OUT, 2, 2, 1, 4, true>(xc, xs, wc, ws, y, M, N, kb, s);
  if (5 * rounds(128, 256) < 8 * rounds(256, 256)) return launch_pipe<OUT, 4, 4>(xc, xs, wc, ws, y, M, N, kb, s);
  return launch_pipe<OUT, 8, 4>(xc, xs, wc, ws, y, M, N, kb, s);
}

hipError_t launch_gemm_fp8(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws, void* y,
                           int out_dtype, int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  return out_dtype == kOutBf16 ? launch_fp8_out<kOutBf16>(xc, xs, wc, ws, y, M, N, kb, s)
                               : launch_fp8_out<kOutF32>(xc, xs, wc, ws, y, M, N, kb, s);
}

}  // namespace hdq
