// Attention over a packed cache of 8-bit codes, f16 queries and results.
#include "attn_packed.cuh"

namespace qg {
const void* attn_packed8f_kernel_ptr(int dim, int rows, PackedLaunch* launch) { return pick_packed<8, true>(dim, rows, launch); }
}  // namespace qg
