// Attention of a few rows (decode, drafted tokens) over a packed cache: the codes go into the matrix instructions as they are.
//
// With k = d_g c + m_g in block g of 32 elements, and likewise for v,
//     <q, k> = sum_g d_g <q_g, c_g> + sum_g m_g sum(q_g),    out_g = sum_t (p_t d_tg) c_t + sum_t p_t m_tg.
// Keys are the rows of the products (16 a step), queries the columns (8, or twice 8): S^T = K Q^T and O^T = V^T P^T.  A code is taken as an f16
// without a conversion: its bits in the low places of a half are the subnormal c 2^-24 (or c 2^-20, four places higher), which the tensor cores
// take exactly, so that one AND makes two operands; 2^24 comes off the fp32 sums, and the 2^4 between the halves of a byte is taken into q (for
// keys) and off at the end (for values).  ldmatrix, and its transposing form for the values, puts a byte's neighbours where an operand wants
// them; which element of a head stands in which place of the sum does not matter, and q is laid out alike.
// The steps d of keys are applied to the fp32 sums of their block, those of values to p (a product in f16); the bases are one more product: with the
// block sums of q, in two f16 pieces (22 bits), and with p.
//
// q is taken in f16, times a power of two of its row that brings its largest element to [2^9, 2^10): elements down to 2^-19 of that keep 11
// bits (a bf16 q all its 8), smaller ones are off by 2^-30 of it.  p is taken as f16 times 2^LIFT and rounded, and its product with a
// step is rounded once more: each by 2^-12 of itself at most, where the product is above 2^-14.  That is 2^-24 d of the largest probability, below
// which bits are lost, for steps of a tenth and more below 2^-21.  The running maximum may lag by 2^LAG, so that it rarely
// moves; a step above 2 counts in the maximum with its own size, so that no product leaves f16.
//
// The rest is as in the 16-bit cache's kernel of few rows: a warp has its own pieces of keys, its own ring of copies, maximum and sum; no barrier in
// the loop; the warps, then a row tile's parts over the blocks, are joined in a fixed order.  A piece is two copies by tensor map, one a page where
// pages are shorter, keys' and values' rows as they lie, steps and bases with them.
#pragma once
#include "attn_rows.cuh"

namespace qg {

template <int DP, int BITS, int NT>
struct PackedShape {
    static constexpr int CODES = DP * BITS / 8;                    // bytes of a row's codes
    static constexpr int PITCH = (CODES + DP / 8 + 15) / 16 * 16;  // bytes of a row (16 bytes times an odd number for heads of 64 and 128:
                                                                   // eight rows' pieces then lie in different banks)
    static constexpr int KEYS = DP <= 128 && 64 * PITCH <= 5120 ? 32 : 16;  // keys of a piece
    static constexpr int STAGE = 2 * KEYS * PITCH;
    static constexpr bool HEAVY = NT == 2 || DP == 256;  // sums that leave room for fewer warps
    static constexpr int WARPS = HEAVY ? 4 : 8, BLOCKS = HEAVY ? 3 : 2;
    static constexpr int FIT = (HEAVY ? 74 : 111) * 1024 / (WARPS * STAGE), STAGES = FIT > 4 ? 4 : FIT;
    static constexpr int ROWS = 8 * NT;
    static constexpr int LINE = DP + 8;  // floats of a row while the warps are joined (in the ring)
    static constexpr unsigned SMEM = WARPS * STAGES * STAGE;
    static_assert(STAGES >= 2 && WARPS * ROWS * (LINE + 2) * 4 <= SMEM, "");
};

constexpr float PACKED_LIFT = 10.f, PACKED_LAG = 4.f;  // p 2^LIFT d <= 2^(LIFT + LAG + 1) where d <= 2

__device__ __forceinline__ void ldsm2(uint32_t& r0, uint32_t& r1, uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm2t(uint32_t& r0, uint32_t& r1, uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
// The bits of `mask` in x as they stand (an AND that is not taken apart or joined with a shift).
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t y;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(y) : "r"(at) : "memory");
    return y;
}
__device__ __forceinline__ float half_at(uint32_t w, int i) { return h2f(i ? w >> 16 : w & 0xFFFFu); }

__device__ __forceinline__ void tma_rows(uint32_t dst, const unsigned long long* map, int token, int page, int head, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(0), "r"(token), "r"(page), "r"(head), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void copy_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(bar)
                 : "memory");
}

// What a warp keeps over the row tiles of its block.
struct Copies {
    uint32_t bars;   // its barriers, one a slot of its ring
    unsigned fills;  // pieces copied so far: piece n is in slot n % STAGES, in phase n / STAGES
    bool broken;     // a copy did not come: no more are asked for
};

// One row tile's part: into the result, or into its record.  Called by the whole block.  WHOLE: heads of DP elements.
template <int DP, int BITS, int NT, bool WHOLE>
__device__ __forceinline__ void attend_packed(const AttnPackedArgs& pa, const Tile& t, long long record, uint8_t* smem, Copies& cp) {
    using S = PackedShape<DP, BITS, NT>;
    const AttnArgs& a = pa.a;
    constexpr int G = DP / 32;             // blocks of a head
    constexpr int CH = S::CODES / 16;      // 16-byte chunks of a row's codes: a block each, or half a block
    constexpr int KT = S::KEYS / 16;
    constexpr uint32_t LO = BITS == 4 ? 0x000F000Fu : 0x00FF00FFu, HI = BITS == 4 ? 0x00F000F0u : 0x00FF00FFu;
    constexpr int HS = BITS == 4 ? 0 : 8;  // 8-bit codes: the odd bytes are moved down
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g8 = lane / 4, t4 = lane % 4;
    const int gd = WHOLE ? G : a.dim / 32;
    const int pitch = WHOLE ? S::PITCH : pa.pitch;
    const int codes = WHOLE ? S::CODES : a.dim * BITS / 8;
    const uint32_t ring = smem_addr(smem) + warp * S::STAGES * S::STAGE;
    const int* table = a.pages + t.seq * a.pages_stride;
    const int pieces = (t.k1 - t.k0 + S::KEYS - 1) / S::KEYS;
    int mine = pieces > warp && !cp.broken ? (pieces - warp + S::WARPS - 1) / S::WARPS : 0;
    auto key_of = [&](int i) { return t.k0 + (warp + i * S::WARPS) * S::KEYS; };

    // ---- copies.  With tensor maps a piece is S::KEYS / box boxes, each on one page; lane n holds page and token of box 32 * batch + n of
    // this warp's, read a batch ahead.  Without, every lane looks its key up and copies its rows.
    const int box = pa.box, nb = box ? S::KEYS / box : 1, nb_shift = box ? __ffs(nb) - 1 : 0;
    struct Where {
        int page, token;  // page -1: no such keys
    };
    auto look_up = [&](int key, int n) {  // keys key .. key + n - 1, on one page
        const int nth = div_by(key, a.page_size, a.page_shift);
        Where w = {-1, key - nth * a.page_size};
        if (key < t.k1 && key + n > t.first) {
            w.page = table[nth];
            if (w.page < 0 || w.page >= a.num_pages) atomicOr(a.err, ERR_BAD_INDEX), w.page = -1;
        }
        return w;
    };
    auto box_at = [&](int n) { return look_up(key_of(n >> nb_shift) + (n & (nb - 1)) * box, box); };
    Where batch = {-1, 0}, ahead = {-1, 0};
    if (box) batch = box_at(lane), ahead = box_at(32 + lane);
    // Asks for piece i; returns which of its keys will be there, one bit each.
    auto issue = [&](int i) -> unsigned {
        const unsigned n = cp.fills + i;
        const int slot = n % S::STAGES;
        const uint32_t bar = cp.bars + slot * 8, kdst = ring + slot * S::STAGE, vdst = kdst + S::KEYS * S::PITCH;
        const int key0 = key_of(i);
        unsigned live = 0;
        if (box) {
            if (i && (i << nb_shift) % 32 == 0) batch = ahead, ahead = box_at((i << nb_shift) + 32 + lane);
            const unsigned ones = box == 32 ? 0xffffffffu : (1u << box) - 1u;
            unsigned there = 0;
            for (int b = 0; b < nb; ++b) {
                const int page = __shfl_sync(0xffffffffu, batch.page, ((i << nb_shift) + b) % 32);
                if (page >= 0) there |= 1u << b, live |= ones << (b * box);
            }
            if (lane == 0) mbar_arrive_expect_tx(bar, 2u * __popc(live) * pitch);
            for (int b = 0; b < nb; ++b) {
                const int page = __shfl_sync(0xffffffffu, batch.page, ((i << nb_shift) + b) % 32);
                const int token = __shfl_sync(0xffffffffu, batch.token, ((i << nb_shift) + b) % 32);
                if (lane == 0 && there >> b & 1u) {
                    tma_rows(kdst + b * box * pitch, pa.k_map, token, page, t.kv_head, bar);
                    tma_rows(vdst + b * box * pitch, pa.v_map, token, page, t.kv_head, bar);
                }
            }
            // (a box reaches over the ends of the range: the keys beyond them are not used)
            const int left = t.k1 - key0;
            if (left < S::KEYS) live &= left <= 0 ? 0u : (1u << left) - 1u;
            if (key0 < t.first) live &= t.first - key0 >= 32 ? 0u : 0xffffffffu << (t.first - key0);
        } else {
            Where w = {-1, 0};
            if (lane < S::KEYS) w = look_up(key0 + lane, 1);
            live = __ballot_sync(0xffffffffu, w.page >= 0);
            if (lane == 0) mbar_arrive_expect_tx(bar, 2u * __popc(live) * pitch);
            __syncwarp();
            if (w.page >= 0) {
                copy_row(kdst + lane * pitch, pa.k + w.page * a.k_page + w.token * a.k_token + t.kv_head * a.k_head, pitch, bar);
                copy_row(vdst + lane * pitch, pa.v + w.page * a.v_page + w.token * a.v_token + t.kv_head * a.v_head, pitch, bar);
            }
        }
        return live;
    };
    unsigned live_ring[S::STAGES] = {};  // which keys of a piece on its way are there, the next first
#pragma unroll
    for (int i = 0; i < S::STAGES; ++i)
        if (i < mine) live_ring[i] = issue(i);

    // ---- queries: column g8 (+ 8) of the products.  A lane holds, of every block, the elements whose codes it meets: 4 bits, elements 8 t4 ..
    // 8 t4 + 7 of the block; 8 bits, 4 t4 .. 4 t4 + 3 of either half.
    uint32_t qb[NT][G][4], mb[NT][G > 4 ? 2 : 1][2];
    float unit[NT][2];  // of the columns 2 t4, 2 t4 + 1 that this lane's sums belong to: scale log2(e) over the row's power of two
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = g8 + 8 * nt;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + out_at(a, t, min(r, t.rows - 1), a.q_token, a.q_head);
        float q[G][8];
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < G; ++s) {
            uint32_t w[4] = {};
            if (r < t.rows && (WHOLE || s < gd)) {
                if constexpr (BITS == 4) {
                    const uint4 u = *reinterpret_cast<const uint4*>(src + 32 * s + 8 * t4);
                    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(src + 32 * s + 4 * t4), v = *reinterpret_cast<const uint2*>(src + 32 * s + 16 + 4 * t4);
                    w[0] = u.x, w[1] = u.y, w[2] = v.x, w[3] = v.y;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t h = w[j / 2] >> (16 * (j % 2)) & 0xFFFFu;
                q[s][j] = pa.bf16 ? __uint_as_float(h << 16) : h2f(h);
                top = fmaxf(top, fabsf(q[s][j]));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the power of two that brings the largest element to [2^9, 2^10); 2^126 is the last one that fp32 has with its inverse
        const int e = top > 0.f ? min(126, 136 - static_cast<int>(__float_as_uint(top) >> 23)) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23), down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * a.scale_log2;
        unit[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t4);
        unit[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
#pragma unroll
        for (int c = 0; c < (G > 4 ? 2 : 1); ++c) mb[nt][c][0] = mb[nt][c][1] = 0u;
#pragma unroll
        for (int s = 0; s < G; ++s) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q[s][j] = __half2float(__float2half_rn(q[s][j] * up));
                sum += q[s][j];
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if constexpr (BITS == 4) {
                qb[nt][s][0] = pack16<false>(q[s][0], q[s][4]);
                qb[nt][s][1] = pack16<false>(q[s][1] * 0.0625f, q[s][5] * 0.0625f);
                qb[nt][s][2] = pack16<false>(q[s][2], q[s][6]);
                qb[nt][s][3] = pack16<false>(q[s][3] * 0.0625f, q[s][7] * 0.0625f);
            } else {
                qb[nt][s][0] = pack16<false>(q[s][0], q[s][2]);
                qb[nt][s][1] = pack16<false>(q[s][1], q[s][3]);
                qb[nt][s][2] = pack16<false>(q[s][4], q[s][6]);
                qb[nt][s][3] = pack16<false>(q[s][5], q[s][7]);
            }
            // the half of a row's steps and bases that block s's base is, where this lane holds it
            const uint32_t first = pack16<false>(sum, 0.f) & 0xFFFFu, rest = pack16<false>(sum - h2f(first), 0.f) & 0xFFFFu;
            const int at = gd + s - 2 * t4;  // 0, 1: first chunk; 8, 9: second
#pragma unroll
            for (int c = 0; c < (G > 4 ? 2 : 1); ++c)
                if ((WHOLE || s < gd) && (at == 8 * c || at == 8 * c + 1)) {
                    mb[nt][c][0] |= first << (16 * (at & 1));
                    mb[nt][c][1] |= rest << (16 * (at & 1));
                }
        }
    }
    // keys that the rows of this lane's two columns see: lo <= key <= hi; all rows see low .. high
    int lo[NT][2], hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int pos = row_pos(a, t, 8 * nt + 2 * t4 + j);
            hi[nt][j] = a.causal ? min(t.k1 - 1, pos) : t.k1 - 1;
            lo[nt][j] = first_key(a, pos);
        }
    const int high = a.causal ? min(t.k1 - 1, row_pos(a, t, 0)) : t.k1 - 1, low = first_key(a, row_pos(a, t, t.rows - 1));

    float o[NT][CH * (BITS == 4 ? 2 : 1)][4], ob[NT][4];  // sums of codes; of the steps and bases (row h: half h of a row's)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (auto& x : o[nt]) x[0] = x[1] = x[2] = x[3] = 0.f;
        ob[nt][0] = ob[nt][1] = ob[nt][2] = ob[nt][3] = 0.f;
    }
    float m[NT][2], base[NT][2], l[NT][2];  // running maximum; what the exponent is taken against (the maximum less LIFT)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) m[nt][j] = NEG_INF, base[nt][j] = 0.f, l[nt][j] = 0.f;

    // this lane's addresses within a piece, for the loads of eight rows' chunks
    const int row8 = lane & 7, sel = lane >> 3;
    const uint32_t k_at = CH >= 4 ? row8 * pitch + sel * 16 : (row8 + (sel >> 1) * 8) * pitch + (sel & 1) * 16;  // chunks of eight keys
    const uint32_t v_at = (row8 + (sel & 1) * 8) * pitch + (sel >> 1) * 16;                                      // of sixteen
    const uint32_t scale_at = (lane & 15) * pitch + codes + (G > 4 ? (lane >> 4) * 16 : 0);
    const uint32_t keep_k0 = 2 * t4 < 2 * gd ? 0xffffffffu : 0u;          // halves beyond a row's steps and bases are anything
    const uint32_t keep_k1 = 8 + 2 * t4 < 2 * gd ? 0xffffffffu : 0u;
    const uint32_t steps = g8 < gd ? 0x80008000u : 0u;                     // rows of the turned steps and bases that are steps

    for (int i = 0; i < mine; ++i) {
        const unsigned n = cp.fills + i;
        const int slot = n % S::STAGES;
        if (!mbar_wait_bounded(cp.bars + slot * 8, n / S::STAGES & 1u)) {
            if (lane == 0) atomicOr(a.err, ERR_WAIT_TIMEOUT);
            // the copies that are still on their way are waited for too; nothing more is asked for
            for (int j = i + 1; j < min(mine, i + S::STAGES); ++j)
                (void)mbar_wait_bounded(cp.bars + (cp.fills + j) % S::STAGES * 8, (cp.fills + j) / S::STAGES & 1u);
            cp.broken = true;
            break;
        }
        const unsigned live = live_ring[0];
        const uint32_t kbase = ring + slot * S::STAGE, vbase = kbase + S::KEYS * S::PITCH;
        const int key0 = key_of(i);
        constexpr unsigned ALL = S::KEYS == 32 ? 0xffffffffu : 0xffffu;
        if (live != ALL) {
            // what is not there may be anything, but has to be a number where it meets p = 0: the steps and bases of its values
            if (lane < S::KEYS && !(live >> lane & 1u)) {
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vbase + lane * pitch + codes), "r"(0) : "memory");
                if constexpr (G > 4)
                    if (pitch - codes > 16) asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vbase + lane * pitch + codes + 16), "r"(0) : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (before a copy writes there again)
            __syncwarp();
        }
        // ---- scores, base 2
        float s[KT][NT][4];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            const uint32_t at = kbase + kt * 16 * pitch;
            uint32_t k[CH][2];  // words of the chunks of key g8 and of key g8 + 8
            if constexpr (CH >= 4) {
#pragma unroll
                for (int c = 0; c < CH; c += 4)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t r[4];
                        ldsm4(r, at + k_at + h * 8 * pitch + c * 16);
                        k[c][h] = r[0], k[c + 1][h] = r[1], k[c + 2][h] = r[2], k[c + 3][h] = r[3];
                    }
            } else {
                uint32_t r[4];
                ldsm4(r, at + k_at);
                k[0][0] = r[0], k[1][0] = r[1], k[0][1] = r[2], k[1][1] = r[3];
            }
            uint32_t w[G > 4 ? 4 : 2];  // steps and bases of key g8, g8 + 8 (twice)
            if constexpr (G > 4) ldsm4(w, at + scale_at);
            else ldsm2(w[0], w[1], at + scale_at);
            float d[2][G];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < G; j += 2) {
                    const uint32_t u = lds32(at + (g8 + 8 * h) * pitch + codes + 2 * j);
                    d[h][j] = half_at(u, 0), d[h][j + 1] = half_at(u, 1);
                }
            if (!WHOLE || G == 2) w[0] &= keep_k0, w[1] &= keep_k0;
            if constexpr (G > 4)
                if (!WHOLE) w[2] &= keep_k1, w[3] &= keep_k1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float sum[4] = {}, bias[4] = {};
#pragma unroll
                for (int c = 0; c < G; ++c) {
                    if (!WHOLE && c >= gd) break;
                    float x[4] = {};
                    if constexpr (BITS == 4) {
                        const uint32_t a0[4] = {k[c][0] & LO, k[c][1] & LO, k[c][0] & HI, k[c][1] & HI};
                        const uint32_t u0 = k[c][0] >> 8, u1 = k[c][1] >> 8;
                        const uint32_t a1[4] = {u0 & LO, u1 & LO, u0 & HI, u1 & HI};
                        mma16816<false>(x, a0, qb[nt][c][0], qb[nt][c][1]);
                        mma16816<false>(x, a1, qb[nt][c][2], qb[nt][c][3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t k0 = k[2 * c + e][0], k1 = k[2 * c + e][1];
                            const uint32_t a0[4] = {k0 & LO, k1 & LO, k0 >> HS & HI, k1 >> HS & HI};
                            mma16816<false>(x, a0, qb[nt][c][2 * e], qb[nt][c][2 * e + 1]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[e] += d[e >> 1][c] * x[e];
                }
                const uint32_t b0[4] = {w[0], w[1], w[0], w[1]};
                if (!WHOLE || G <= 4) mma16816<false>(bias, b0, mb[nt][0][0], mb[nt][0][1]);
                if constexpr (G > 4) {
                    const uint32_t b1[4] = {w[2], w[3], w[2], w[3]};
                    mma16816<false>(bias, b1, mb[nt][1][0], mb[nt][1][1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[kt][nt][e] = unit[nt][e & 1] * (sum[e] * 16777216.f + bias[e]);
            }
        }
        if (live != ALL || key0 < low || key0 + S::KEYS - 1 > high) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = kt * 16 + g8 + 8 * (e >> 1), j = e & 1;
                        const bool sees = (live >> c & 1u) && key0 + c >= lo[nt][j] && key0 + c <= hi[nt][j];
                        if (!sees) s[kt][nt][e] = NEG_INF;
                    }
        }
        // ---- steps and bases of the values, turned: this lane has half g8 (and g8 + 8) of keys 2 t4, 2 t4 + 1 and of those 8 on
        uint32_t w[KT][G > 4 ? 4 : 2];
        unsigned large = 0;  // a step above 2 (bits above 0x4000) carries into a half's top bit
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            const uint32_t at = vbase + kt * 16 * pitch + scale_at;
            if constexpr (G > 4) ldsm4t(w[kt], at);
            else ldsm2t(w[kt][0], w[kt][1], at);
            large |= (w[kt][0] + 0x3FFF3FFFu) | (w[kt][1] + 0x3FFF3FFFu);
        }
        // ---- the running maximum, where it has to move
        bool moves = (large & steps) != 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float top = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
                if constexpr (KT == 2) top = fmaxf(top, fmaxf(s[KT - 1][nt][j], s[KT - 1][nt][j + 2]));
                moves |= top > m[nt][j] + PACKED_LAG;
            }
        if (__any_sync(0xffffffffu, moves)) {
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) top[nt][0] = m[nt][0], top[nt][1] = m[nt][1];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float d = 2.f;
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        if (!WHOLE && j >= gd) break;
                        const uint32_t u = lds32(vbase + (kt * 16 + g8 + 8 * h) * pitch + codes + j / 2 * 4);
                        d = fmaxf(d, half_at(u, j & 1));
                    }
                    const float e = log2f(d) - 1.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) top[nt][j] = fmaxf(top[nt][j], s[kt][nt][j + 2 * h] + e);
                }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float keep[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float& x = top[nt][j];
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    keep[j] = x == NEG_INF ? 1.f : exp2_approx(m[nt][j] - x);
                    m[nt][j] = x;
                    base[nt][j] = x == NEG_INF ? 0.f : x - PACKED_LIFT;
                    l[nt][j] *= keep[j];
                }
#pragma unroll
                for (auto& x : o[nt]) x[0] *= keep[0], x[1] *= keep[1], x[2] *= keep[0], x[3] *= keep[1];
                ob[nt][0] *= keep[0], ob[nt][1] *= keep[1], ob[nt][2] *= keep[0], ob[nt][3] *= keep[1];
            }
        }
        // ---- values
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            const uint32_t at = vbase + kt * 16 * pitch;
            uint32_t p[NT][2];  // column g8's p of keys 2 t4, 2 t4 + 1 and of those 8 on
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = exp2_approx(s[kt][nt][e] - base[nt][e & 1]);
                l[nt][0] += x[0] + x[2], l[nt][1] += x[1] + x[3];
                p[nt][0] = turn8x8(pack16<false>(x[0], x[1]));
                p[nt][1] = turn8x8(pack16<false>(x[2], x[3]));
                uint32_t b[4] = {w[kt][0], 0u, w[kt][1], 0u};
                if constexpr (G > 4) b[1] = w[kt][2], b[3] = w[kt][3];
                mma16816<false>(ob[nt], b, p[nt][0], p[nt][1]);
            }
#pragma unroll
            for (int c2 = 0; c2 < CH; c2 += 2) {
                uint32_t v[4];  // chunks c2 and c2 + 1, keys 0 .. 7 and 8 .. 15 of each
                ldsm4t(v, at + v_at + c2 * 16);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = c2 + e, blk = BITS == 4 ? c : c / 2;
                    if (!WHOLE && blk >= gd) break;
                    uint32_t d0, d1;
                    d0 = __shfl_sync(0xffffffffu, w[kt][0], 4 * blk + t4);
                    d1 = __shfl_sync(0xffffffffu, w[kt][1], 4 * blk + t4);
                    const uint32_t v0 = v[2 * e], v1 = v[2 * e + 1];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t p0 = mul2(p[nt][0], d0), p1 = mul2(p[nt][1], d1);
                        if constexpr (BITS == 4) {
                            const uint32_t a0[4] = {v0 & LO, v0 & HI, v1 & LO, v1 & HI};
                            const uint32_t u0 = v0 >> 8, u1 = v1 >> 8;
                            const uint32_t a1[4] = {u0 & LO, u0 & HI, u1 & LO, u1 & HI};
                            mma16816<false>(o[nt][2 * c], a0, p0, p1);
                            mma16816<false>(o[nt][2 * c + 1], a1, p0, p1);
                        } else {
                            const uint32_t a0[4] = {v0 & LO, v0 >> HS & HI, v1 & LO, v1 >> HS & HI};
                            mma16816<false>(o[nt][c], a0, p0, p1);
                        }
                    }
                }
            }
        }
        __syncwarp();  // every lane has read the piece
#pragma unroll
        for (int j = 0; j + 1 < S::STAGES; ++j) live_ring[j] = live_ring[j + 1];
        live_ring[S::STAGES - 1] = i + S::STAGES < mine ? issue(i + S::STAGES) : 0u;
    }
    cp.fills += mine;

    // ---- join the warps, in the (now idle) ring
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);        // [WARPS][ROWS][LINE]
    float* stat = acc + S::WARPS * S::ROWS * S::LINE;   // [WARPS][ROWS][2]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        if (8 * nt >= t.rows) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int x = 4; x < 32; x *= 2) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], x);
            const int row = warp * S::ROWS + 8 * nt + 2 * t4 + j;
            if (g8 == 0) stat[row * 2] = m[nt][j] == NEG_INF ? NEG_INF : base[nt][j], stat[row * 2 + 1] = l[nt][j];
            float* line = acc + row * S::LINE;
#pragma unroll
            for (int b = 0; b < G; ++b) {
                if (!WHOLE && b >= gd) break;
                const int h = gd + b;  // the half that block b's base is: what it adds lies with the lanes of row h % 8
                const float lower = __shfl_sync(0xffffffffu, ob[nt][j], 4 * (h & 7) + t4), upper = __shfl_sync(0xffffffffu, ob[nt][j + 2], 4 * (h & 7) + t4);
                const float add = h < 8 ? lower : upper;
                constexpr float U = 16777216.f, U4 = 1048576.f;  // 2^24, and 2^20 for a byte's upper half
                if constexpr (BITS == 4) {
                    const auto& x = o[nt][2 * b];
                    const auto& y = o[nt][2 * b + 1];
                    *reinterpret_cast<float4*>(line + 32 * b + 4 * g8) =
                        make_float4(x[j] * U + add, x[j + 2] * U4 + add, y[j] * U + add, y[j + 2] * U4 + add);
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const auto& x = o[nt][2 * b + e];
                        *reinterpret_cast<float2*>(line + 32 * b + 16 * e + 2 * g8) = make_float2(x[j] * U + add, x[j + 2] * U + add);
                    }
                }
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < t.rows * (DP / 4); i += S::WARPS * 32) {
        const int r = i / (DP / 4), d = i % (DP / 4) * 4;
        if (d >= a.dim) continue;
        float mm = NEG_INF;
#pragma unroll
        for (int w = 0; w < S::WARPS; ++w) mm = fmaxf(mm, stat[(w * S::ROWS + r) * 2]);
        const float from = mm == NEG_INF ? 0.f : mm;
        float ll = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < S::WARPS; ++w) {
            const float f = exp2_approx(stat[(w * S::ROWS + r) * 2] - from);
            const float4 v = *reinterpret_cast<const float4*>(acc + (w * S::ROWS + r) * S::LINE + d);
            ll += f * stat[(w * S::ROWS + r) * 2 + 1];
            x.x += f * v.x, x.y += f * v.y, x.z += f * v.z, x.w += f * v.w;
        }
        if (t.parts > 1) {
            __stcg(reinterpret_cast<float4*>(a.part_sum + (record + r) * a.dim + d), x);
            if (d == 0) __stcg(a.part_stat + record + r, make_float2(mm, ll));
        } else if (pa.bf16) {
            put_row4<true>(a, t, r, d, x, mm, ll);
        } else {
            put_row4<false>(a, t, r, d, x, mm, ll);
        }
    }
    // (the ring is written by copies again: what was written and read here comes before them)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int DP, int BITS, int NT, bool WHOLE>
__global__ void __launch_bounds__(PackedShape<DP, BITS, NT>::WARPS * 32, PackedShape<DP, BITS, NT>::BLOCKS)
    attn_packed_kernel(const __grid_constant__ AttnPackedArgs pa) {
    using S = PackedShape<DP, BITS, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ unsigned long long bars[S::WARPS * S::STAGES];
    __shared__ unsigned last;
    if (threadIdx.x < S::WARPS * S::STAGES) mbar_init(smem_addr(bars + threadIdx.x), 1);
    fence_mbar_init();
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    Copies cp = {smem_addr(bars + threadIdx.x / 32 * S::STAGES), 0u, false};
    divide_rows<S::ROWS, 32>(
        pa.a, &last, [&](const Tile& t, long long record) { attend_packed<DP, BITS, NT, WHOLE>(pa, t, record, smem, cp); },
        [&](const Tile& t) {
            constexpr int THREADS = S::WARPS * 32, AT_ONCE = THREADS / (DP / 4), ITEMS = (S::ROWS + AT_ONCE - 1) / AT_ONCE;
            if (pa.bf16) join_rows<DP, THREADS, true, ITEMS>(pa.a, t);
            else join_rows<DP, THREADS, false, ITEMS>(pa.a, t);
        });
}

template <int BITS, int DP, int NT, bool WHOLE>
static const void* packed_kernel(PackedLaunch* launch) {
    using S = PackedShape<DP, BITS, NT>;
    *launch = {S::SMEM, S::WARPS * 32u, S::BLOCKS, S::ROWS, S::KEYS};
    return (const void*)attn_packed_kernel<DP, BITS, NT, WHOLE>;
}

// Heads of up to 128 have kernels for up to 8 and up to 16 rows; those of 64, 128 and 256 kernels of their own.
template <int BITS>
const void* pick_packed(int dim, int rows, PackedLaunch* launch) {
    if (dim > 128) return dim == 256 ? packed_kernel<BITS, 256, 1, true>(launch) : packed_kernel<BITS, 256, 1, false>(launch);
    if (dim == 128) return rows <= 8 ? packed_kernel<BITS, 128, 1, true>(launch) : packed_kernel<BITS, 128, 2, true>(launch);
    if (dim == 64) return rows <= 8 ? packed_kernel<BITS, 64, 1, true>(launch) : packed_kernel<BITS, 64, 2, true>(launch);
    if (dim > 64) return rows <= 8 ? packed_kernel<BITS, 128, 1, false>(launch) : packed_kernel<BITS, 128, 2, false>(launch);
    return rows <= 8 ? packed_kernel<BITS, 64, 1, false>(launch) : packed_kernel<BITS, 64, 2, false>(launch);
}

}  // namespace qg
