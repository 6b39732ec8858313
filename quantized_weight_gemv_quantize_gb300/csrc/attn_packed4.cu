// Attention over a packed cache of 4-bit codes, bf16 queries and results.
#include "attn_packed.cuh"

namespace qg {
const void* attn_packed4_kernel_ptr(int dim, int rows, PackedLaunch* launch) { return pick_packed<4, false>(dim, rows, launch); }
}  // namespace qg
