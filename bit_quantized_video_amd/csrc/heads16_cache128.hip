// heads16_cache128.hip -- k_heads16 for bf16 heads of 128, keys and values to the cache (a file of its own: they compile side by side).
#include "heads16.h"

namespace hdq {

void run_heads16_cache128(const HeadArgs& g, dim3 grid, hipStream_t s) { run16<false, 3, true>(g, grid, s); }

}  // namespace hdq
