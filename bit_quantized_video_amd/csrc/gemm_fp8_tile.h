// gemm_fp8_tile.h -- what the FP8 block-128 GEMM kernels share: fragments,
// block products and output stores.
//
// y[m, n] = sum_b sx[b, m] sw[n / 128, b] sum_{k in block b} cx[m, k] cw[n, k]
//
// The A operand of every product is a 16-row slice of W, the B operand a
// 16-row slice of X, so a lane of the 16 x 16 result holds token m = lane % 16
// and features n = 4 (lane / 16) + 0..3: one activation scale per lane and
// slice, and four consecutive outputs.  A fragment is 16 rows x 128 k: lane l
// holds row l % 16, bytes 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q + 15 of
// the block, q = l / 16 (any order of k is right as long as both operands
// share it).
//
// Two product forms, chosen by the output type:
//  * FAST (bf16 output): v_mfma_scale_f32_16x16x128_f8f6f4 with unit scales, a
//    whole block in one instruction, whose result is then scaled and added by
//    four FMAs.  The hardware aligns the 128 products to the largest one with
//    at least 14 fraction bits: 1.3e-5 of the result in the 2-norm on Gaussian
//    codes (measured), far below the 1.7e-3 of rounding to bf16.  One output in
//    a hundred then rounds to the other neighbour than from a float32 sum.
//  * exact products (fp32 output): the codes converted to bf16 (exactly), four
//    v_mfma_f32_16x16x32_bf16 with float32 sums, at half the matrix rate: 4e-8
//    of the result in the 2-norm for one block, 6e-8 for 15, 1e-7 for 96
//    (measured; storing it in float32 costs 2.5e-8 of that).
#pragma once

#include "fp8_device.h"
#include "hdq_internal.h"

namespace hdq {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// A fragment from its two 16-byte pieces.
typedef v8i Fp8Frag;
__device__ __forceinline__ Fp8Frag load_frag(const uint8_t* lo, const uint8_t* hi) {
  return __builtin_shufflevector(*reinterpret_cast<const v4i*>(lo), *reinterpret_cast<const v4i*>(hi), 0, 1, 2, 3, 4,
                                 5, 6, 7);
}

// Eight E4M3 codes (two words) to bf16, exact.
__device__ __forceinline__ v8bf codes_to_bf16(int w0, int w1) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A fragment in the form its product takes.
template <bool FAST>
struct Fp8Operand;
template <>
struct Fp8Operand<true> {
  v8i v;
  __device__ __forceinline__ void set(const Fp8Frag& f) { v = f; }
};
template <>
struct Fp8Operand<false> {
  v8bf v[4];
  __device__ __forceinline__ void set(const Fp8Frag& f) {
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = codes_to_bf16(f[2 * t], f[2 * t + 1]);
  }
};

// One block's 16 x 16 product.  A caller reads the scaled instruction's result in
// the basic block it is issued in (no branch between, unrolled loops only): where
// the reader began the joining block, the compiler left too few wait states and
// wrong values were read.
__device__ __forceinline__ v4f block_product(const Fp8Operand<true>& w, const Fp8Operand<true>& x) {
  constexpr int kUnitScale = 0x7f7f7f7f;  // E8M0 2^0 in every byte
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, kUnitScale,
                                                           0, kUnitScale);
}
__device__ __forceinline__ v4f block_product(const Fp8Operand<false>& w, const Fp8Operand<false>& x) {
  v4f p = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int t = 0; t < 4; ++t) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[t], x.v[t], p, 0, 0, 0);
  return p;
}

__device__ __forceinline__ void add_scaled(v4f& acc, const v4f& p, float s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(p[e], s, acc[e]);
}

// Vectors at any element's address: with N no multiple of the vector, rows begin
// anywhere, and gfx950's global stores take unaligned addresses (element-wise
// stores made 10877 x 224 -> 2997 68 us instead of 33).
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef int i32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Stores y[m, n .. n + 3] (n a multiple of 4; columns past N are left out).
template <int OUT>
__device__ __forceinline__ void store_out4(void* __restrict__ Y, int64_t m, int n, int N, const v4f& v) {
  const int64_t off = m * N + n;
  if constexpr (OUT == kOutBf16) {
    uint16_t* y = static_cast<uint16_t*>(Y) + off;
    const uint32_t a = pack_bf16x2(v[0], v[1]), b = pack_bf16x2(v[2], v[3]);
    if (n + 4 <= N) {
      *reinterpret_cast<u32x2_a2*>(y) = u32x2_a2{a, b};
    } else {
      const uint16_t h[4] = {(uint16_t)a, (uint16_t)(a >> 16), (uint16_t)b, (uint16_t)(b >> 16)};
      for (int e = 0; e < 4 && n + e < N; ++e) y[e] = h[e];
    }
  } else {
    float* y = static_cast<float*>(Y) + off;
    if (n + 4 <= N) {
      *reinterpret_cast<f32x4_a4*>(y) = v;
    } else {
      for (int e = 0; e < 4 && n + e < N; ++e) y[e] = v[e];
    }
  }
}

}  // namespace hdq
