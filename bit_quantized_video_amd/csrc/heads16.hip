// heads16.hip -- k_heads16 for bf16 heads to floats (a file of its own: they compile side by side).
#include "heads16.h"

namespace hdq {

void run_heads16(const HeadArgs& g, dim3 grid, hipStream_t s) {
  g.dim == 64 ? run16<false, 2, false>(g, grid, s) : g.dim == 128 ? run16<false, 3, false>(g, grid, s) : run16<false, -1, false>(g, grid, s);
}

}  // namespace hdq
