// heads16_cache64.hip -- k_heads16 for bf16 heads of 64, keys and values to the cache (a file of its own: they compile side by side).
#include "heads16.h"

namespace hdq {

void run_heads16_cache64(const HeadArgs& g, dim3 grid, hipStream_t s) { run16<false, 2, true>(g, grid, s); }

}  // namespace hdq
