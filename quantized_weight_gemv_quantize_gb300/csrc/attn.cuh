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

// The probabilities meet the values in 16 bits.  bf16 has fp32's exponents; f16 keeps its 11 bits only down to 2^-14 and nothing below 2^-25,
// so that what many keys far below the largest add up to would be lost.  There p is taken 2^lift times as large, as far as f16
// reaches: 11 bits down to 2^-29 (e^-20) of the largest in the 16-row kernel and 2^-21 (e^-14.5) in the 128-row one, something down to 2^-40
// and 2^-32.  The sums l and o carry the same factor, and m, the maximum in use, is the largest score less the lift.
// (A lift of 12 in the 128-row kernel leaves its maximum 2^3 to lag by, which costs up to a quarter of its speed: 2000 f16 tokens over 24000,
// scores of standard deviation 3: 589 -> 682 us, two prompts 352 -> 436.)
template <bool BF>
struct Lift {
    static constexpr float ROWS = BF ? 0.f : 15.f;  // p <= 1: p 2^15 <= 32768
    static constexpr float LAG = 8.f;               // the 128-row kernel's maximum may lag by 2^LAG ...
    static constexpr float TILES = BF ? 0.f : 7.f;  // ... so that p <= 2^LAG, and p 2^TILES <= 32768
};

// x / d for d with shift = log2(d), or -1 where d is no power of two (both the same for the whole launch).
__device__ __forceinline__ int div_by(int x, int d, int shift) { return shift >= 0 ? x >> shift : x / d; }

// Rows of one key/value head, and the keys of them that a block takes.
struct Tile {
    int seq, kv_head, part, parts;  // parts: how many the row tile's keys are cut into
    int row0, rows;                 // first row, and rows in the tile
    int q0;                         // first new token of the sequence in q
    int first_pos;                  // position of the sequence's new token 0
    int first;                      // the first key that a row of the tile sees: those of its key tile before it are as if missing
    int k0, k1;                     // keys of this part
    long long index;                // number of the row tile, for the records of its parts
};

// A sequence, with the values on the device held to the bounds that the launch was shaped for.
struct Seq {
    int q0, n, first_pos, usable;  // first token in q, new tokens, position of the first of them, keys that may be read
};
__device__ __forceinline__ Seq find_seq(const AttnArgs& a, int b) {
    Seq s;
    s.q0 = max(0, min(a.q_start[b], a.tokens));
    const int n = max(0, min(a.q_start[b + 1], a.tokens) - s.q0), len = max(0, a.kv_len[b]);
    s.first_pos = len - n;
    s.n = min(n, a.max_q);
    s.usable = min(len, a.max_kv);
    return s;
}

// The first key that a token at position `pos` sees (any window: no difference leaves 32 bits).
__device__ __forceinline__ int first_key(const AttnArgs& a, int pos) {
    return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}

// The keys that some row of [row0, row0 + rows) sees, from a multiple of `step` on; returns the first one seen.  Where there are
// none, hi = lo: nothing before that first one, and nothing beyond the keys that may be read, is then in the range.
__device__ __forceinline__ int find_keys(const AttnArgs& a, const Seq& s, int row0, int rows, int step, int* lo, int* hi) {
    const int first = first_key(a, s.first_pos + div_by(row0, a.group, a.group_shift));
    *lo = first / step * step;
    *hi = a.causal ? min(s.usable, s.first_pos + div_by(row0 + rows - 1, a.group, a.group_shift) + 1) : s.usable;
    if (*hi <= first) *hi = *lo;
    return first;
}

// Position of row `r` of the tile: it sees the keys from first_key to (under a causal mask) its own position.
__device__ __forceinline__ int row_pos(const AttnArgs& a, const Tile& t, int r) {
    return t.first_pos + div_by(t.row0 + r, a.group, a.group_shift);
}

__device__ __forceinline__ long long out_at(const AttnArgs& a, const Tile& t, int r, long long token_stride,
                                            long long head_stride) {
    const int row = t.row0 + r, token = div_by(row, a.group, a.group_shift);
    return (t.q0 + token) * token_stride + (t.kv_head * a.group + row - token * a.group) * head_stride;
}

__device__ __forceinline__ void put_lse(const AttnArgs& a, const Tile& t, int r, float m2, float l) {
    if (!a.lse) return;
    // (l is 0 where the row sees nothing; NaN, of a query that is no number, goes on as NaN)
    a.lse[out_at(a, t, r, a.heads, 1)] = l == 0.f ? NEG_INF : (m2 + log2f(l)) * 0.693147180559945309f;
}

// Elements d .. d + 3 of a row of the result from its unnormalised sums; with d = 0 its log-sum-exp.
template <bool BF>
__device__ __forceinline__ void put_row4(const AttnArgs& a, const Tile& t, int r, int d, float4 x, float m, float l) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out_at(a, t, r, a.out_token, a.out_head) + d) =
        make_uint2(pack16<BF>(x.x * inv, x.y * inv), pack16<BF>(x.z * inv, x.w * inv));
    if (d == 0) put_lse(a, t, r, m, l);
}

// A part's record of a row: the maximum in use (base 2) and the sum in part_stat[at], dim unnormalised sums of values in
// part_sum[at * dim ..].  A warp joins the parts of one row (at most 32, of heads of up to 128), always in the same order, and writes the
// result; rec(p): the record of part p.  Lane l takes elements 4 l .. 4 l + 3.  The first loads depend on nothing but rec, so that all are
// on their way at once.
template <bool BF, class Rec>
__device__ __forceinline__ void join_row(const AttnArgs& a, const Tile& t, int r, Rec rec) {
    const int lane = threadIdx.x % 32, d = 4 * lane;
    const float2 s = lane < t.parts ? __ldcg(a.part_stat + rec(lane)) : make_float2(NEG_INF, 0.f);  // a lane a part
    float m = s.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float w = exp2_approx(s.x - (m == NEG_INF ? 0.f : m));
    float l = w * s.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int p = 0; p < t.parts; ++p) {
        const float f = __shfl_sync(0xffffffffu, w, p);
        const float4 v = d < a.dim ? __ldcg(reinterpret_cast<const float4*>(a.part_sum + rec(p) * a.dim + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
        acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
    }
    if (d < a.dim) put_row4<BF>(a, t, r, d, acc, m, l);
}

}  // namespace qg
