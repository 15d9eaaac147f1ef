// fp8_quant.hip -- block-Hadamard rotation fused with FP8 block-128
// quantization (gfx950).
//
// Per block of 128 (of a row, or 128 x 128): a = max|y|, s = a / 448,
// code = E4M3(y * (448 / a)).  Bound by HBM: 2 bytes read and 1 + 4/128
// written per element (rows), 2 and 1 (blocks); one pass over the data, since
// a block's maximum is known within a quad of lanes or a workgroup.  Measured:
// rows 17776 x 12288, rotated by 128, 135 us (4.9 TB/s, what a large copy
// reaches); 226 x 1000 3.3 to 3.8 us (the launch); blocks 5760 x 1920 7.7 us.
#include "fp8_device.h"
#include "hdq_internal.h"

namespace hdq {

// Rows: a wave owns 16 rows x one block of 128 (lane l: row l / 4, 32
// elements of the block's quarter l % 4): it reads 16 runs of 256 bytes and
// writes 16 runs of 128, and its 16 scales are one 64-byte store of the
// [block, row] layout.  The four waves of a workgroup take neighbouring
// blocks of the same rows.
template <int HB>
__global__ __launch_bounds__(256) void k_fp8_quant_rows(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                        int kb, float c_b, uint8_t* __restrict__ codes,
                                                        float* __restrict__ scale) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int kgroups = (kb + 3) >> 2;
  const unsigned blk = wide_block();
  const int b = (int)(blk % (unsigned)kgroups) * 4 + wave;
  const int64_t row = (int64_t)(blk / (unsigned)kgroups) * 16 + (lane >> 2);
  if (b >= kb || row >= rows) return;  // whole quads leave together
  float y[32];
  const int part = lane & 3;
  load_row32(reinterpret_cast<const uint4*>(x + row * cols), b * 16 + part * 4, cols >> 3, y);
  rotate32<HB>(y, lane, c_b);
  float s, inv;
  fp8_scales(quad_max(absmax32(y)), s, inv);
  uint4 out[2];
  // lanes past the row (whole Hadamard blocks) hold rotated zeros of either sign
  fp8_encode32(y, b * kFp8Block + part * 32 < cols ? inv : 0.0f, out);
  uint4* dst = reinterpret_cast<uint4*>(codes + row * ((int64_t)kb * kFp8Block) + b * kFp8Block + part * 32);
  dst[0] = out[0];
  dst[1] = out[1];
  if (part == 0) scale[(int64_t)b * rows + row] = s;
}

// Blocks: a workgroup of 512 threads holds one 128 x 128 block in registers
// (thread t: row t / 4, quarter t % 4).
template <int HB>
__global__ __launch_bounds__(512) void k_fp8_quant_blocks(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                          int kb, float c_b, uint8_t* __restrict__ codes,
                                                          float* __restrict__ scale) {
  __shared__ float red[8];
  const int tid = threadIdx.x, lane = tid & 63, part = tid & 3;
  const unsigned blk = wide_block();
  const int b = (int)(blk % (unsigned)kb);
  const int64_t rb = blk / (unsigned)kb, row = rb * kFp8Block + (tid >> 2);
  if (rb * kFp8Block >= rows) return;
  float y[32];
  // rows past the end hold zeros (their quads take part in the maximum)
  const bool in = row < rows;
  load_row32(reinterpret_cast<const uint4*>(x + (in ? row : 0) * cols), b * 16 + part * 4, in ? cols >> 3 : 0, y);
  rotate32<HB>(y, lane, c_b);
  float a = quad_max(absmax32(y));
#pragma unroll
  for (int o = 4; o < 64; o <<= 1) a = __builtin_elementwise_maximum(a, __shfl_xor(a, o));
  if (lane == 0) red[tid >> 6] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) a = __builtin_elementwise_maximum(a, red[w]);
  float s, inv;
  fp8_scales(a, s, inv);
  if (tid == 0) scale[rb * kb + b] = s;
  if (!in) return;
  uint4 out[2];
  // lanes past the row (whole Hadamard blocks) hold rotated zeros of either sign
  fp8_encode32(y, b * kFp8Block + part * 32 < cols ? inv : 0.0f, out);
  uint4* dst = reinterpret_cast<uint4*>(codes + row * ((int64_t)kb * kFp8Block) + b * kFp8Block + part * 32);
  dst[0] = out[0];
  dst[1] = out[1];
}

template <int HB>
static hipError_t launch_fp8_quant_hb(const uint16_t* x, int64_t rows, int64_t cols, int layout, uint8_t* codes,
                                      float* scale, hipStream_t s) {
  const int64_t kb = fp8_blocks(cols);
  const float c_b = hadamard_scale(HB);
  if (layout == kFp8Rows) {
    const int64_t grid = (rows + 15) / 16 * ((kb + 3) / 4);
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    k_fp8_quant_rows<HB><<<wide_grid(grid), dim3(256), 0, s>>>(x, rows, (int)cols, (int)kb, c_b, codes, scale);
  } else {
    const int64_t grid = fp8_blocks(rows) * kb;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    k_fp8_quant_blocks<HB><<<wide_grid(grid), dim3(512), 0, s>>>(x, rows, (int)cols, (int)kb, c_b, codes, scale);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_quant(const uint16_t* x, int64_t rows, int64_t cols, int hb, int layout, uint8_t* codes,
                            float* scale, hipStream_t s) {
  switch (hb) {
    case 1: return launch_fp8_quant_hb<1>(x, rows, cols, layout, codes, scale, s);
    case 2: return launch_fp8_quant_hb<2>(x, rows, cols, layout, codes, scale, s);
    case 4: return launch_fp8_quant_hb<4>(x, rows, cols, layout, codes, scale, s);
    case 8: return launch_fp8_quant_hb<8>(x, rows, cols, layout, codes, scale, s);
    case 16: return launch_fp8_quant_hb<16>(x, rows, cols, layout, codes, scale, s);
    case 32: return launch_fp8_quant_hb<32>(x, rows, cols, layout, codes, scale, s);
    case 64: return launch_fp8_quant_hb<64>(x, rows, cols, layout, codes, scale, s);
    case 128: return launch_fp8_quant_hb<128>(x, rows, cols, layout, codes, scale, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace hdq
