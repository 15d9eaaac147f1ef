// heads16_f32.hip -- k_heads16 for float32 heads (a file of its own: they compile side by side).
#include "heads16.h"

namespace hdq {

void run_heads16_f32(const HeadArgs& g, bool cache, dim3 grid, hipStream_t s) {
  cache ? run16<true, -1, true>(g, grid, s) : run16<true, -1, false>(g, grid, s);
}

}  // namespace hdq
