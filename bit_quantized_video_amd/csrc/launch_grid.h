// launch_grid.h -- grids of many workgroups, in host code without HIP types.
#pragma once

#include <stdint.h>

namespace hdq {

struct Grid {
  int64_t x, y;
};

// A grid of `blocks` workgroups (at most 2^31) of up to 512 threads: HIP takes fewer
// than 2^32 threads along x, so past 2^22 workgroups they are laid out in
// rows.  The last row may pass `blocks`.
constexpr int64_t kWideRow = 1 << 22;
inline Grid wide(int64_t blocks) {
  return blocks <= kWideRow ? Grid{blocks, 1} : Grid{kWideRow, (blocks + kWideRow - 1) / kWideRow};
}

}  // namespace hdq
