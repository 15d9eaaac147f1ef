// heads16_cache.hip -- k_heads16 for bf16 heads of other sizes, keys and values to the cache (a file of its own: they compile side by side).
#include "heads16.h"

namespace hdq {

void run_heads16_cache(const HeadArgs& g, dim3 grid, hipStream_t s) { run16<false, -1, true>(g, grid, s); }

}  // namespace hdq
