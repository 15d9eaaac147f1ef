// heads16_cache.hip -- k_heads16 for bf16 heads, keys and values to the cache (a file of its own: they compile side by side).
#include "heads16.h"

namespace hdq {

void run_heads16_cache(const HeadArgs& g, dim3 grid, hipStream_t s) {
  g.dim == 64 ? run16<false, 2, true>(g, grid, s) : g.dim == 128 ? run16<false, 3, true>(g, grid, s) : run16<false, -1, true>(g, grid, s);
}

}  // namespace hdq
