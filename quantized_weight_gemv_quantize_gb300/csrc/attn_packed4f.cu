// Attention over a packed cache of 4-bit codes, f16 queries and results.
#include "attn_packed.cuh"

namespace qg {
const void* attn_packed4f_kernel_ptr(int dim, int rows, PackedLaunch* launch) { return pick_packed<4, true>(dim, rows, launch); }
}  // namespace qg
