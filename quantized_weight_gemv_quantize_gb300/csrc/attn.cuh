// What the attention kernels share: a row tile's sequence and range of keys, and the joining of its parts.
//
// The rows of a sequence and key/value head are its (new token, query head of the group) pairs, token-major:
// row r is token r / group, head kv_head * group + r % group.  All of them read the same keys, so a tile of rows is one
// operand of the matrix products whatever the group size is.
#pragma once
#include "common.cuh"
#include "internal.h"
#include "step.h"

namespace qg {

constexpr float NEG_INF = -__builtin_huge_valf();

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool BF>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    uint32_t r;  // the first operand goes to the upper half
    if constexpr (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// One row tile of the launch: which rows, which keys, which of its parts.
struct Tile {
    int seq, kv_head, part, parts;  // parts: how many the tile has (its own count, at most the grid's)
    int row0, rows;                 // first row, and rows in the tile
    int q0;                         // first new token of the sequence in q
    int first_pos;                  // position of the sequence's new token 0
    int k0, k1;                     // keys of this part
    int kv_len;                     // keys that may be read
    long long index;                // number of (seq, kv_head, row tile) in the grid
};

// False: nothing to do for this block (past the sequence's rows or the tile's parts).  LAST_FIRST: the row tiles with the
// most keys (the last ones, under a causal mask) of all sequences and heads come first, so that the grid ends with short ones.
template <int ROWS, bool LAST_FIRST>
__device__ __forceinline__ bool find_tile(const AttnArgs& a, long long block, Tile* t) {
    t->part = static_cast<int>(block % a.parts);
    t->index = block / a.parts;
    const int pairs = a.kv_heads * a.seqs;
    const int rt = static_cast<int>(LAST_FIRST ? a.row_tiles - 1 - t->index / pairs : t->index % a.row_tiles);
    const int sh = static_cast<int>(LAST_FIRST ? t->index % pairs : t->index / a.row_tiles);
    t->kv_head = static_cast<int>(sh % a.kv_heads);
    t->seq = static_cast<int>(sh / a.kv_heads);
    // the values on the device are held to the bounds that the launch was shaped for
    const int q0 = max(0, min(a.q_start[t->seq], a.tokens));
    const int n = max(0, min(a.q_start[t->seq + 1], a.tokens) - q0);
    const int len = max(0, a.kv_len[t->seq]);
    t->q0 = q0;
    t->first_pos = len - n;
    const long long table = a.pages_stride * a.page_size;
    const int usable = static_cast<int>(min(static_cast<long long>(min(len, a.max_kv)), table));
    t->kv_len = usable;
    t->row0 = rt * ROWS;
    t->rows = min(ROWS, min(n, a.max_q) * a.group - t->row0);
    if (t->rows <= 0) return false;
    const int pos_lo = t->first_pos + t->row0 / a.group;
    const int pos_hi = t->first_pos + (t->row0 + t->rows - 1) / a.group;
    int lo = 0, hi = usable;
    if (a.window > 0) lo = max(0, pos_lo - a.window + 1);
    if (a.causal) hi = min(hi, pos_hi + 1);
    if (LAST_FIRST) lo = lo / 128 * 128;  // the 128-row kernel's key tiles start at multiples of their size
    hi = max(hi, lo);
    t->parts = max(1, (hi - lo + a.chunk - 1) / a.chunk);
    if (t->part >= t->parts) return false;
    t->k0 = lo + t->part * a.chunk;
    t->k1 = min(hi, t->k0 + a.chunk);
    return true;
}

// Positions of the keys that row `r` of the tile sees: first_key(r) <= t <= last_key(r).
__device__ __forceinline__ int row_pos(const AttnArgs& a, const Tile& t, int r) {
    return t.first_pos + (t.row0 + r) / a.group;
}

__device__ __forceinline__ long long out_at(const AttnArgs& a, const Tile& t, int r, long long token_stride,
                                            long long head_stride) {
    const int row = t.row0 + r;
    return (t.q0 + row / a.group) * token_stride + (t.kv_head * a.group + row % a.group) * head_stride;
}

__device__ __forceinline__ void put_lse(const AttnArgs& a, const Tile& t, int r, float m2, float l) {
    if (!a.lse) return;
    const int row = t.row0 + r;
    const long long at = static_cast<long long>(t.q0 + row / a.group) * a.heads + t.kv_head * a.group + row % a.group;
    a.lse[at] = l > 0.f ? (m2 + log2f(l)) * 0.693147180559945309f : NEG_INF;
}

// Record of row r of a part: m (base 2), l, then dim unnormalised sums.
__device__ __forceinline__ float* part_row(const AttnArgs& a, const Tile& t, int part, int r) {
    return a.part + ((t.index * a.parts + part) * a.rows_part + r) * static_cast<long long>(a.dim + 2);
}

// Called by every thread of the block after its part's records are written.  The block that arrives last joins the parts
// in their order (so the result does not depend on which one that is) and puts the counter back to zero.
template <bool BF>
__device__ __forceinline__ void join_parts(const AttnArgs& a, const Tile& t) {
    __shared__ unsigned last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.count + t.index, 1u) == static_cast<unsigned>(t.parts - 1);
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (threadIdx.x == 0) a.count[t.index] = 0;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    for (int r = warp; r < t.rows; r += warps) {
        float m = NEG_INF;
        for (int p = 0; p < t.parts; ++p) m = fmaxf(m, __ldcg(part_row(a, t, p, r)));
        const float base = m == NEG_INF ? 0.f : m;
        float l = 0.f;
        for (int p = 0; p < t.parts; ++p) {
            const float* rec = part_row(a, t, p, r);
            l += exp2_approx(__ldcg(rec) - base) * __ldcg(rec + 1);
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const long long at = out_at(a, t, r, a.out_token, a.out_head);
        for (int d = 2 * lane; d < a.dim; d += 64) {
            float x = 0.f, y = 0.f;
            for (int p = 0; p < t.parts; ++p) {
                const float* rec = part_row(a, t, p, r);
                const float w = exp2_approx(__ldcg(rec) - base);
                const float2 v = __ldcg(reinterpret_cast<const float2*>(rec + 2 + d));
                x += w * v.x, y += w * v.y;
            }
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at + d) = pack16<BF>(x * inv, y * inv);
        }
        if (lane == 0) put_lse(a, t, r, m, l);
    }
}

}  // namespace qg
