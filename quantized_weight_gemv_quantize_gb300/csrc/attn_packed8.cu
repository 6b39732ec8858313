// Attention over a packed cache of 8-bit codes, bf16 queries and results.
#include "attn_packed.cuh"

namespace qg {
const void* attn_packed8_kernel_ptr(int dim, int rows, PackedLaunch* launch) { return pick_packed<8, false>(dim, rows, launch); }
}  // namespace qg
