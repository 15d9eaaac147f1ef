// gemm_fp8.hip -- FP8 block-128 linear layers on gfx950.
//
// Operands, product forms and accuracy: gemm_fp8_tile.h.
#include "gemm_fp8_tile.h"

namespace hdq {

// Few rows or small layers: no LDS staging, no barrier in the K loop.  A
// workgroup owns MT x 16 tokens by NT x 16 features; its WAVES waves take the
// blocks of K in turn (wave w: w, w + WAVES, ...), each reading its fragments
// from global memory straight into registers one block ahead, and the partial
// tiles are added over LDS in a fixed order.  Bound by the weights' bytes at
// few rows.
template <int OUT, int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_fp8_skinny(const uint8_t* __restrict__ xc,
                                                           const float* __restrict__ xs,
                                                           const uint8_t* __restrict__ wc,
                                                           const float* __restrict__ ws, void* __restrict__ Y,
                                                           int64_t M, int N, int kb, int tiles_n) {
  constexpr bool FAST = OUT == kOutBf16;
  __shared__ v4f part[WAVES > 1 ? WAVES / 2 : 1][MT * NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int tn = (int)(blockIdx.x % (unsigned)tiles_n);
  const int64_t m0 = (int64_t)(blockIdx.x / (unsigned)tiles_n) * (16 * MT);
  const int n0 = tn * (16 * NT);
  const int64_t ld = (int64_t)kb * kFp8Block;
  // rows past the end repeat the last one; their results are not stored
  const uint8_t* xp[MT];
  const float* xsp[MT];
  const uint8_t* wp[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = min(m0 + 16 * i + r16, M - 1);
    xp[i] = xc + m * ld + 16 * q;
    xsp[i] = xs + m;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) wp[j] = wc + (int64_t)min(n0 + 16 * j + r16, N - 1) * ld + 16 * q;
  // the tile's features lie in one block row of the weights' scales
  const float* wsp = ws + (int64_t)(n0 / kFp8Block) * kb;

  struct Block {
    Fp8Frag x[MT], w[NT];
    float s[MT];
  };
  auto load = [&](Block& b, int k) {
    const int64_t o = (int64_t)k * kFp8Block;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      b.w[j].lo = *reinterpret_cast<const v4i*>(wp[j] + o);
      b.w[j].hi = *reinterpret_cast<const v4i*>(wp[j] + o + 64);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      b.x[i].lo = *reinterpret_cast<const v4i*>(xp[i] + o);
      b.x[i].hi = *reinterpret_cast<const v4i*>(xp[i] + o + 64);
      b.s[i] = xsp[i][(int64_t)k * M] * wsp[k];
    }
  };
  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto compute = [&](const Block& b) {
    Fp8Operand<FAST> w[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) w[j].set(b.w[j]);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      Fp8Operand<FAST> x;
      x.set(b.x[i]);
      v4f p[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) p[j] = block_product(w[j], x);
#pragma unroll
      for (int j = 0; j < NT; ++j) add_scaled(acc[i][j], p[j], b.s[i]);
    }
  };
  Block b0, b1;
  int k = wave;
  if (k < kb) load(b0, k);
  while (k < kb) {
    if (k + WAVES < kb) load(b1, k + WAVES);
    compute(b0);
    k += WAVES;
    if (k >= kb) break;
    if (k + WAVES < kb) load(b0, k + WAVES);
    compute(b1);
    k += WAVES;
  }
  // halving sum over the waves: wave w adds wave w + h
#pragma unroll
  for (int h = WAVES / 2; h >= 1; h >>= 1) {
    if (wave >= h && wave < 2 * h) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) part[wave - h][i * NT + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave < h) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] += part[wave][i * NT + j][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = m0 + 16 * i + r16;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < NT; ++j) store_out4<OUT>(Y, m, n0 + 16 * j + 4 * q, N, acc[i][j]);
  }
}

template <int OUT, int MT, int NT, int WAVES>
static hipError_t launch_skinny(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws, void* y,
                                int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  const int64_t tiles_n = (N + 16 * NT - 1) / (16 * NT), tiles_m = (M + 16 * MT - 1) / (16 * MT);
  if (tiles_n * tiles_m > 0x7fffffff) return hipErrorInvalidValue;
  k_fp8_skinny<OUT, MT, NT, WAVES><<<dim3((unsigned)(tiles_m * tiles_n)), dim3(64 * WAVES), 0, s>>>(
      xc, xs, wc, ws, y, M, (int)N, (int)kb, (int)tiles_n);
  return hipGetLastError();
}

template <int OUT>
static hipError_t launch_fp8_out(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws, void* y,
                                 int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  if (M <= 16) return launch_skinny<OUT, 1, 1, 8>(xc, xs, wc, ws, y, M, N, kb, s);
  return launch_skinny<OUT, 4, 4, 4>(xc, xs, wc, ws, y, M, N, kb, s);
}

hipError_t launch_gemm_fp8(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws, void* y,
                           int out_dtype, int64_t M, int64_t N, int64_t kb, hipStream_t s) {
  return out_dtype == kOutBf16 ? launch_fp8_out<kOutBf16>(xc, xs, wc, ws, y, M, N, kb, s)
                               : launch_fp8_out<kOutF32>(xc, xs, wc, ws, y, M, N, kb, s);
}

}  // namespace hdq
