// w4.h -- launchers of the 4-bit group-scaled weights (w4.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "w4_plan.h"

namespace hdq {

struct W4Weights {
  const uint8_t* codes;
  const uint16_t* scale;
  const uint8_t* zero;  // null: 8
  int64_t N, K;
  int group;
};
struct W4Out {
  uint8_t* codes;
  uint16_t* scale;
  uint8_t* zero;  // null: without zero points
};

// y [M, N] (float32 or bf16) from bf16 x [M, K]; ws: w4_workspace bytes.
hipError_t launch_w4(const uint16_t* x, int64_t M, const W4Weights& w, void* y, bool f32, void* ws, hipStream_t s);
hipError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scale, const uint8_t* zero, int64_t N, int64_t K,
                          int group, const W4Out& out, hipStream_t s);
hipError_t launch_w4_quantize(const uint16_t* w, int64_t N, int64_t K, int group, const W4Out& out, hipStream_t s);

}  // namespace hdq
