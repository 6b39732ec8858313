// Attention of a few rows (decode, drafted tokens) over a packed cache: the codes go into the matrix instructions as they are.
//
// With k = d_g c + m_g in block g of 32 elements, and likewise for v,
//     <q, k> = sum_g d_g <q_g, c_g> + sum_g m_g sum(q_g),    out_g = sum_t (p_t d_tg) c_t + sum_t p_t m_tg.
// Keys are the rows of the products (16 a step), queries the columns (8, or twice 8): S^T = K Q^T and O^T = V^T P^T.  A code is taken as an f16
// without a conversion: its bits in the low places of a half are the subnormal c 2^-24 (or c 2^-20, four places higher), which the tensor cores
// take exactly, so that one AND makes two operands (a step's sum is cut 2^-23 below the largest product's nominal exponent, which a subnormal has as 2^-14: with 17
// addends at most 17 2^-13 of the step's largest p d, or q d, is lost, 1/16 of it four places higher); 2^24 comes off the fp32 sums, and the 2^4 between the halves of a byte is taken into q (for
// keys) and off at the end (for values).  ldmatrix, and its transposing form for the values, puts a byte's neighbours where an operand wants
// them; which element of a head stands in which place of the sum does not matter, and q is laid out alike.
// The steps d of keys are applied to the fp32 sums of their block, those of values to p (a product in f16); the bases are one more product: with the
// block sums of q, in two f16 pieces (22 bits), and with p.
//
// q is taken in f16, times a power of two of its row that brings its largest element to [2^9, 2^10): elements down to 2^-19 of that keep 11
// bits (a bf16 q all its 8), smaller ones are off by 2^-30 of it.  p is taken in f16, 2^LIFT p rounded; for f16 results its rest too, so that its
// product with a step is rounded once, to 11 bits.  What that rounding leaves is multiplied by codes about Z, the middle one, in place of codes from 0: sum (p d)(c - Z)
// + sum p (m + Z d), where (p d) stands for the rounded product in both of its sums (one product with ones a block) and the last sum is
// small.  Bits are lost where p d is below 2^-24 of what stands for a p of 2^-LIFT.  The running maximum may lag by 2^LAG, so that it rarely
// moves; a step above 2 counts in the maximum with its own size, so that no product leaves f16.
//
// The division over one wave of blocks and the joining are those of the 16-bit cache's kernel of few rows: a warp has its own pieces of keys, maximum
// and sum; the warps of a head, then a row tile's parts over the blocks, are joined in a fixed order.  The copies are the block's: a ring of rounds, each
// one or two pieces of 16 keys of every warp, rows as they lie, steps and bases with them; by tensor map, or where pages are no multiple of 16 tokens by
// plain copies of a token's rows or of a run of tokens (pages of 24: 195 and 143 us for the 48 sequences' 99 below).
// The warps take turns to issue a round.  Where the ring has 5 or 6 slots (heads of 64 in 4 bits, and more than 8 rows but for heads of 128 in 8 bits) a slot is filled
// again two rounds after it was read, and nobody waits for the slowest warp; where 2 or 3 (up to 8 rows of heads of 128 and 256, among others) the issuing
// warp waits for the round just before.  Rounds of half the size, with twice the slots, were slower there too (113 us for 99 below).
// The warps of a block take 1 to 4 key/value heads side by side, the same keys of each: a row is 80 bytes for heads of 128 in 4 bits, so that where
// a token's heads lie together a head alone fetched 2.6 times its bytes from memory (1166 MB for 442).
//
// Bound by memory in the loop (5.8 TB/s of codes, of 6.8 that a copy reaches; 297 instructions a warp for 16 keys of a head, issue slots 42% taken),
// and by what comes before and after it: lengths and division 2 to 4 us, the first keys 4, joining 3 to 7.  Measured over several GPUs with 32 heads of 128 over 8 (us; bytes at a
// copy's rate in brackets): 4 bits, one sequence of 777 10.3 to 12.2 (0.15), one of 100003 41 (19), 48 sequences of up to 16384 99 (67); 8 bits, f16, up
// to 5 drafts of 16 sequences over 4000 (16 heads) 31 to 35 (9), a window of 1024 over 33 sequences 25 to 29 (12).  Steps on the way, the 48 sequences: a ring
// of asynchronous 16-byte copies a warp, one head a block 200; heads side by side 130; the block's ring of whole lines 104; queries asked for before the copies 99.  Slower
// were a copy a row (151 to 170), a ring a warp (121 to 145), a warp that only copies (116), rounds of one piece (113), even shares (107).
#pragma once
#include "attn_rows.cuh"

namespace qg {

template <int DP, int BITS, int NT>
struct PackedShape {
    static constexpr int CODES = DP * BITS / 8;                    // bytes of a row's codes
    static constexpr int PITCH = (CODES + DP / 8 + 15) / 16 * 16;  // bytes of a row (16 bytes times an odd number for heads of 64 and 128:
                                                                   // eight rows' pieces then lie in different banks)
    static constexpr int WARPS = 4, BLOCKS = NT == 2 || DP == 256 ? 2 : 3;  // 255 or 168 registers a thread
    static constexpr int SIDE = WARPS * 16 * PITCH + 256;  // 16 keys, or values, of every warp, and room to keep rows of several heads apart
    static constexpr int ROOM = (BLOCKS == 2 ? 111 : 74) * 1024;
    static constexpr int KT = 4 * SIDE <= ROOM / 2 ? 2 : 1;  // a round is KT times 16 keys of every warp
    static constexpr int STAGE = KT * 2 * SIDE;
    static constexpr int FIT = ROOM / STAGE, STAGES = FIT > 6 ? 6 : FIT;
    static constexpr int BACK = STAGES > 3 ? 2 : 1;      // a slot is filled again so many rounds after it was read
    static constexpr int ROWS = 8 * NT;
    static constexpr int LINE = DP + 8;  // floats of a row while the warps are joined (in the ring)
    static constexpr unsigned SMEM = STAGES * STAGE;
    static_assert(STAGES >= 2 && WARPS * ROWS * (LINE + 2) * 4 <= SMEM, "");
};

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// (by the threads with one != 0, without a branch)
__device__ __forceinline__ void mbar_arrive(uint32_t bar, uint32_t one) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar), "r"(one) : "memory");
}
// 16 tokens of one page and of some heads.
__device__ __forceinline__ void tma_box(uint32_t dst, const unsigned long long* map, int x, int y, int page, int head, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(page), "r"(head), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void copy_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(bar)
                 : "memory");
}

constexpr float PACKED_LIFT = 10.f, PACKED_LAG = 4.f;  // p 2^LIFT d <= 2^(LIFT + LAG + 1) where d <= 2

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
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t y;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
    return y;
}
// The product alone: nothing is added to it.
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// The N (2, 4 or 8) halves at an address, widened.
template <int N>
__device__ __forceinline__ void lds_halves(float (&x)[N], uint32_t at) {
    uint32_t w[N / 2];
    if constexpr (N == 2) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
    else if constexpr (N == 4) asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    else asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        x[2 * j] = f.x, x[2 * j + 1] = f.y;
    }
}

constexpr unsigned PLAIN = 0x10000u;
// The ring of a block's copies.  A round is KT times 16 keys of each warp; its slot and parity run on over the block's row tiles.
template <int STAGES>
struct Ring {
    unsigned long long full[STAGES], empty[STAGES];
    unsigned lives[STAGES * 16]; // which of a box's 16 keys are there, one bit each, and PLAIN where every row sees them all
    int broken;                  // a wait ran out: no more is copied
};

// One row tile's part: into the result, or into its record.  Called by the whole block.  WHOLE: heads of DP elements.  FINE:
// p's rounding is made up for.  plain: 16 bytes of zeros in shared memory, then 16 of ones in f16.
template <int DP, int BITS, int NT, bool WHOLE, bool FINE>
__device__ __forceinline__ void attend_packed(const AttnPackedArgs& pa, const Tile& t, long long record, uint8_t* smem, uint32_t plain,
                                              Ring<PackedShape<DP, BITS, NT>::STAGES>& ring, int& slot, unsigned& parity) {
    using S = PackedShape<DP, BITS, NT>;
    const AttnArgs& a = pa.a;
    constexpr int G = DP / 32;             // blocks of a head
    constexpr int CH = S::CODES / 16;      // 16-byte chunks of a row's codes: a block each, or half a block
    constexpr uint32_t LO = BITS == 4 ? 0x000F000Fu : 0x00FF00FFu, HI = BITS == 4 ? 0x00F000F0u : 0x00FF00FFu;
    constexpr int HS = BITS == 4 ? 0 : 8;  // 8-bit codes: the odd bytes are moved down
    constexpr int KT = S::KT;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g8 = lane / 4, t4 = lane % 4;
    const uint32_t one = lane == 0;
    const int gd = WHOLE ? G : a.dim / 32;
    const int pitch = WHOLE ? S::PITCH : pa.pitch;
    const int codes = WHOLE ? S::CODES : a.dim * BITS / 8;
    const uint32_t store = smem_addr(smem);
    const int* table = a.pages + t.seq * a.pages_stride;
    // this warp's head, and which of the head's warps it is
    const int heads = 1 << pa.hb_shift, warps = S::WARPS >> pa.hb_shift;
    const int hh = warp & (heads - 1), nth_warp = warp >> pa.hb_shift, head = t.kv_head + hh;
    const int per_round = warps * KT * 16;
    const int rounds = ring.broken ? 0 : (t.k1 - t.k0 + per_round - 1) / per_round;
    // keys that every row sees: low .. high
    const int high = a.causal ? min(t.k1 - 1, row_pos(a, t, 0)) : t.k1 - 1, low = first_key(a, row_pos(a, t, t.rows - 1));

    // ---- queries: column g8 (+ 8) of the products.  A lane holds, of every block, the elements whose codes it meets: 4 bits, elements 8 t4 ..
    // 8 t4 + 7 of the block; 8 bits, 4 t4 .. 4 t4 + 3 of either half.  They are asked for before the copies, which would keep them waiting.
    Tile own = t;
    own.kv_head = head;
    uint32_t qw[NT][G][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = g8 + 8 * nt;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + out_at(a, own, min(r, t.rows - 1), a.q_token, a.q_head);
#pragma unroll
        for (int s = 0; s < G; ++s) {
            uint32_t (&w)[4] = qw[nt][s];
            w[0] = w[1] = w[2] = w[3] = 0u;
            if (r < t.rows && (WHOLE || s < gd)) {
                if constexpr (BITS == 4) {
                    const uint4 u = *reinterpret_cast<const uint4*>(src + 32 * s + 8 * t4);
                    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(src + 32 * s + 4 * t4), v = *reinterpret_cast<const uint2*>(src + 32 * s + 16 + 4 * t4);
                    w[0] = u.x, w[1] = u.y, w[2] = v.x, w[3] = v.y;
                }
            }
        }
    }

    // ---- copies.  A slot holds KT times: 16 keys of each warp, then their values, by boxes of 16 keys of all the heads.  Round r is asked for by
    // warp r % WARPS: lane n for box n, the keys 16 n of the round on, which are the (n % KT)th of the heads' (n / KT)th warps.  Its pages are looked
    // up a turn ahead.
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
    // rows are `rp` bytes apart in a box and heads `hp`
    const bool by_rows = pa.copies == COPY_ROWS || pa.copies == COPY_TOKENS, by_map = pa.copies < COPY_TOKENS;
    const int rp = by_rows ? heads * pitch + (heads == S::WARPS ? 16 : 0) : pitch, hp = by_rows ? pitch : 16 * pitch;
    const int box_bytes = by_rows ? 16 * rp : heads * 16 * pitch;
    auto box_key = [&](int r, int n) { return t.k0 + r * per_round + n * 16; };
    auto box_at = [&](int n) { return n % KT * 2 * S::SIDE + n / KT * box_bytes; };
    auto put_live = [&](int to, int n, int key, unsigned live) {
        ring.lives[to * 16 + n] = live | (live == 0xffffu && key >= low && key + 15 <= high ? PLAIN : 0u);
    };
    Where ahead = {-1, 0};
    if (by_map && warp < rounds && lane < warps * KT) ahead = look_up(box_key(warp, lane), 16);
    auto issue = [&](int r, int to) {
        const uint32_t bar = smem_addr(&ring.full[to]), dst = store + to * S::STAGE;
        if (by_map) {
            const int key = box_key(r, lane), left = t.k1 - key, before = t.first - key;
            const bool there = ahead.page >= 0;
            unsigned live = there ? 0xffffu : 0u;
            // (a box reaches over the ends of the range: the keys beyond them are not used)
            if (left < 16) live &= left <= 0 ? 0u : (1u << left) - 1u;
            if (before > 0) live &= before >= 16 ? 0u : 0xffffu << before;
            if (lane < warps * KT) put_live(to, lane, key, live);
            const unsigned boxes = __popc(__ballot_sync(0xffffffffu, there));
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(bar, 2u * boxes * box_bytes);
            __syncwarp();
            if (there) {
                // (map coordinates: COPY_BOXES 0, token, page, head; COPY_ROWS the heads' place in a token's rows, token, page; COPY_HEADS the token's place in
                // a head's rows, head, page)
                const int x = by_rows ? t.kv_head * pitch / 8 : pa.copies == COPY_HEADS ? ahead.token * (pitch / 8) : 0;
                const int y = pa.copies == COPY_HEADS ? t.kv_head : ahead.token, z = pa.copies == COPY_BOXES ? t.kv_head : 0;
                tma_box(dst + box_at(lane), pa.k_map, x, y, ahead.page, z, bar);
                tma_box(dst + S::SIDE + box_at(lane), pa.v_map, x, y, ahead.page, z, bar);
            }
            ahead.page = -1;
            if (r + S::WARPS < rounds && lane < warps * KT) ahead = look_up(box_key(r + S::WARPS, lane), 16);
        } else {
            // 32 keys at a time, the next ones looked up before their copies: of a token's rows, of a page's or of one
            auto key_at = [&](int k) { return k < per_round ? look_up(box_key(r, 0) + k, 1) : Where{-1, 0}; };
            Where next = key_at(lane);
#pragma unroll 1
            for (int k = lane; k - lane < per_round; k += 32) {
                const Where w = next;
                next = key_at(k + 32);
                const unsigned some = __ballot_sync(0xffffffffu, w.page >= 0);
                const int box = (k - lane) / 16 + lane;
                if (lane < 2 && box < warps * KT) put_live(to, box, box_key(r, box), some >> (16 * lane) & 0xffffu);
                if (lane == 0) mbar_expect_tx(bar, 2u * __popc(some) * heads * pitch);
                __syncwarp();
                const bool goes_on = pa.copies == COPY_RUNS && w.token != 0 && (lane & 15) && (some >> (lane - 1) & 1u);
                const unsigned begin = __ballot_sync(0xffffffffu, w.page >= 0 && !goes_on), cut = lane < 31 ? (begin | ~some) >> (lane + 1) : 0u;
                if (!(begin >> lane & 1u)) continue;
                const int n = cut ? __ffs(cut) : 32 - lane;  // keys of the run that begins here
                const uint8_t* kp = pa.k + w.page * a.k_page + w.token * a.k_token + t.kv_head * a.k_head;
                const uint8_t* vp = pa.v + w.page * a.v_page + w.token * a.v_token + t.kv_head * a.v_head;
                const uint32_t at = dst + box_at(k >> 4) + (k & 15) * rp;
                const int bytes = by_rows ? heads * pitch : n * pitch;
#pragma unroll 1
                for (int h = 0; h < (by_rows ? 1 : heads); ++h) {
                    copy_row(at + h * hp, kp + h * a.k_head, bytes, bar);
                    copy_row(at + S::SIDE + h * hp, vp + h * a.v_head, bytes, bar);
                }
            }
            __syncwarp();  // (what is there is written)
            mbar_arrive(bar, one);
        }
    };
    // the first rounds: their slots were read in the row tile before, which ended with a barrier
    {
        int to = slot;
#pragma unroll 1
        for (int r = 0; r < S::STAGES - S::BACK && r < rounds; ++r) {
            if (r % S::WARPS == warp) issue(r, to);
            to = to + 1 == S::STAGES ? 0 : to + 1;
        }
    }

    // ---- the queries as operands
    uint32_t qb[NT][G][4], mb[NT][G > 4 ? 2 : 1][2];
    float unit[NT][2];  // of the columns 2 t4, 2 t4 + 1 that this lane's sums belong to: 2^24 scale log2(e) over the row's power of two
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float q[G][8];
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < G; ++s) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t h = qw[nt][s][j / 2] >> (16 * (j % 2)) & 0xFFFFu;
                q[s][j] = pa.bf16 ? __uint_as_float(h << 16) : h2f(h);
                top = fmaxf(top, fabsf(q[s][j]));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the power of two that brings the largest element to [2^9, 2^10); 2^126 is the last one that fp32 has with its inverse
        const int e = top > 0.f ? min(126, 136 - static_cast<int>(__float_as_uint(top) >> 23)) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        // (finite and above 0, so that no product with an infinity is NaN)
        const float down = fminf(fmaxf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23) * a.scale_log2 * 16777216.f, 1e-37f), 3e38f);
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
    // keys that the rows of this lane's two columns see: lo <= key <= hi
    int lo[NT][2], hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int pos = row_pos(a, t, 8 * nt + 2 * t4 + j);
            hi[nt][j] = a.causal ? min(t.k1 - 1, pos) : t.k1 - 1;
            lo[nt][j] = first_key(a, pos);
        }

    // Sums of codes, and with p alone of the steps and bases (row h: half h of a row's).  Sums of the rounded products p d: rows 8 on of the
    // latter where a row's halves end before them, else in sums of their own.
    float o[NT][CH * (BITS == 4 ? 2 : 1)][4], ob[NT][4], od[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (auto& x : o[nt]) x[0] = x[1] = x[2] = x[3] = 0.f;
        ob[nt][0] = ob[nt][1] = ob[nt][2] = ob[nt][3] = 0.f;
        od[nt][0] = od[nt][1] = od[nt][2] = od[nt][3] = 0.f;
    }
    float m[NT][2], base[NT][2], l[NT][2];  // running maximum; what the exponent is taken against (the maximum less LIFT)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) m[nt][j] = NEG_INF, base[nt][j] = 0.f, l[nt][j] = 0.f;

    // This lane's addresses within a slot, for the loads of eight rows' chunks: two chunks of keys (of values, SIDE on) 0 to 7 and 8 to 15 each;
    const int row8 = lane & 7, sel = lane >> 3;
    const uint32_t mine = store + nth_warp * box_bytes + hh * hp;
    const uint32_t row_at = mine + (row8 + (sel & 1) * 8) * rp + (sel >> 1) * 16;
    // steps and bases as an operand, eight keys and eight halves a quarter: for keys, 0 to 7, 8 to 15, then their second eight halves or the first again;
    const uint32_t ks_at = mine + (lane & 15) * rp + codes + (G > 4 ? (lane >> 4) * 16 : 0);
    // for values (turned), keys 8 to 15 are the third quarter, and the second eight halves, or zeros, the second and the fourth;
    const bool zeros = G <= 4 && (sel & 1);
    const uint32_t vs_at = mine + S::SIDE + (row8 + (sel >> 1) * 8) * rp + codes + (sel & 1) * 16;
    // and the steps of keys g8 and g8 + 8.
    const uint32_t step_at = mine + g8 * rp + codes, step8 = 8 * rp;
    const uint32_t keep_k0 = 2 * t4 < 2 * gd ? 0xffffffffu : 0u;          // halves beyond a row's steps and bases are anything
    const uint32_t keep_k1 = 8 + 2 * t4 < 2 * gd ? 0xffffffffu : 0u;
    const uint32_t steps = g8 < gd ? 0x80008000u : 0u;                     // rows of the turned steps and bases that are steps

    auto wait = [&](const unsigned long long& bar, unsigned phase) {
        if (mbar_try_wait(smem_addr(&bar), phase)) return true;
        if (mbar_wait_bounded(smem_addr(&bar), phase)) return true;
        atomicOr(a.err, ERR_WAIT_TIMEOUT);
        ring.broken = 1;
        return false;
    };
#pragma unroll 1
    for (int i = 0; i < rounds; ++i) {
        const int fresh = i + S::STAGES - S::BACK;
        if (fresh < rounds && (fresh & (S::WARPS - 1)) == warp) {
            // into the slot that was read BACK rounds ago (if one was: else it is free)
            const bool wraps = slot < S::BACK;
            const int to = wraps ? slot + S::STAGES - S::BACK : slot - S::BACK;
            if (i >= S::BACK && !wait(ring.empty[to], parity ^ (wraps ? 1u : 0u))) break;
            issue(fresh, to);
        }
        if (!wait(ring.full[slot], parity)) break;
        unsigned live[KT], all = PLAIN, any = 0;
        if constexpr (KT == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(&ring.lives[slot * 16 + 2 * nth_warp]);
            live[0] = u.x, live[KT - 1] = u.y;
        } else {
            live[0] = ring.lives[slot * 16 + nth_warp];
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) all &= live[kt], any |= live[kt];
        if (any) {
            const uint32_t at = slot * S::STAGE;
            if (!all) {
                // what is not there may be anything, but has to be a number where it meets p = 0: the steps and bases of its values
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
                    if (lane < 16 && !(live[kt] >> lane & 1u)) {
                        const uint32_t to = mine + at + kt * 2 * S::SIDE + S::SIDE + lane * rp + codes;
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(to), "r"(0) : "memory");
                        if (G > 4 && pitch - codes > 16) asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(to + 16), "r"(0) : "memory");
                    }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (before a copy writes there again)
                __syncwarp();
            }
            // ---- scores, in units of `unit`
            float s[KT][NT][4];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const uint32_t from = at + kt * 2 * S::SIDE;
                uint32_t k[CH][2];  // words of the chunks of key g8 and of key g8 + 8
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t r[4];
                    ldsm4(r, row_at + from + c * 16);
                    k[c][0] = r[0], k[c][1] = r[1], k[c + 1][0] = r[2], k[c + 1][1] = r[3];
                }
                uint32_t w[4];  // steps and bases of key g8, g8 + 8; the second eight halves, or the same again
                ldsm4(w, ks_at + from);
                float d[2][G];
                lds_halves(d[0], step_at + from), lds_halves(d[1], step_at + step8 + from);
                if (!WHOLE || G == 2) w[0] &= keep_k0, w[1] &= keep_k0;
                if ((!WHOLE || G == 2) && G <= 4) w[2] &= keep_k0, w[3] &= keep_k0;
                if constexpr (G > 4)
                    if (!WHOLE) w[2] &= keep_k1, w[3] &= keep_k1;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float bias[4];
                    if constexpr (G > 4) {
                        const uint32_t b0[4] = {w[0], w[1], w[0], w[1]};
                        const uint32_t b1[4] = {w[2], w[3], w[2], w[3]};
                        mma_first(bias, b1, mb[nt][1][0], mb[nt][1][1]);
                        if (!WHOLE) mma16816<false>(bias, b0, mb[nt][0][0], mb[nt][0][1]);
                    } else {
                        mma_first(bias, w, mb[nt][0][0], mb[nt][0][1]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[kt][nt][e] = bias[e] * 0x1p-24f;
                }
#pragma unroll
                for (int c = 0; c < G; ++c) {
                    if (!WHOLE && c >= gd) break;
                    uint32_t a0[4], a1[4];
                    if constexpr (BITS == 4) {
                        const uint32_t k0 = k[c][0], k1 = k[c][1], u0 = k0 >> 8, u1 = k1 >> 8;
                        a0[0] = k0 & LO, a0[1] = k1 & LO, a0[2] = k0 & HI, a0[3] = k1 & HI;
                        a1[0] = u0 & LO, a1[1] = u1 & LO, a1[2] = u0 & HI, a1[3] = u1 & HI;
                    } else {
                        const uint32_t k0 = k[2 * c][0], k1 = k[2 * c][1], u0 = k[2 * c + 1][0], u1 = k[2 * c + 1][1];
                        a0[0] = k0 & LO, a0[1] = k1 & LO, a0[2] = k0 >> HS & HI, a0[3] = k1 >> HS & HI;
                        a1[0] = u0 & LO, a1[1] = u1 & LO, a1[2] = u0 >> HS & HI, a1[3] = u1 >> HS & HI;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float x[4];
                        mma_first(x, a0, qb[nt][c][0], qb[nt][c][1]);
                        mma16816<false>(x, a1, qb[nt][c][2], qb[nt][c][3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[kt][nt][e] += d[e >> 1][c] * x[e];
                    }
                }
            }
            if (!all) {
                int key0 = box_key(i, nth_warp * KT);
                asm volatile("" : "+r"(key0));  // (a branch, not predicates: rare)
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = g8 + 8 * (e >> 1), j = e & 1, key = key0 + kt * 16 + c;
                            const bool sees = (live[kt] >> c & 1u) && key >= lo[nt][j] && key <= hi[nt][j];
                            if (!sees) s[kt][nt][e] = NEG_INF;
                        }
                __syncwarp();
            }
            // ---- steps and bases of the values, turned: this lane has half g8 of keys 2 t4, 2 t4 + 1, and half g8 + 8 or zeros, then those of keys 8 on
            uint32_t w[KT][4], large = 0;  // a step above 2 (bits above 0x4000) carries into a half's top bit
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                ldsm4t(w[kt], zeros ? plain : vs_at + at + kt * 2 * S::SIDE);
                large |= (w[kt][0] + 0x3FFF3FFFu) | (w[kt][2] + 0x3FFF3FFFu);
            }
            // ---- the running maximum, where it has to move
            bool moves = (large & steps) != 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
                    if constexpr (KT == 2) top = fmaxf(top, fmaxf(s[KT - 1][nt][j], s[KT - 1][nt][j + 2]));
                    moves |= top * unit[nt][j] > m[nt][j] + PACKED_LAG;
                }
            if (__any_sync(0xffffffffu, moves)) {
                float top[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) top[nt][0] = m[nt][0], top[nt][1] = m[nt][1];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float d[G], most = 2.f;
                        lds_halves(d, step_at + at + kt * 2 * S::SIDE + S::SIDE + h * step8);
#pragma unroll
                        for (int j = 0; j < G; ++j)
                            if (WHOLE || j < gd) most = fmaxf(most, d[j]);
                        const float e = log2f(most) - 1.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j) top[nt][j] = fmaxf(top[nt][j], s[kt][nt][j + 2 * h] * unit[nt][j] + e);
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
#pragma unroll
                    for (int e = 0; e < 4; ++e) ob[nt][e] *= keep[e & 1], od[nt][e] *= keep[e & 1];
                }
            }
            // ---- values
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const uint32_t from = at + kt * 2 * S::SIDE + S::SIDE;
                uint32_t p[NT][2], rest[NT][2];  // column g8's p of keys 2 t4, 2 t4 + 1 and of those 8 on, and what its rounding left
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = exp2_approx(s[kt][nt][e] * unit[nt][e & 1] - base[nt][e & 1]);
                    l[nt][0] += x[0] + x[2], l[nt][1] += x[1] + x[3];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u = pack16<false>(x[2 * h], x[2 * h + 1]);
                        p[nt][h] = turn8x8(u);
                        if constexpr (FINE) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
                            rest[nt][h] = turn8x8(pack16<false>(x[2 * h] - f.x, x[2 * h + 1] - f.y));
                        }
                    }
                    mma16816<false>(ob[nt], w[kt], p[nt][0], p[nt][1]);
                }
                uint32_t pd[NT][2];
#pragma unroll
                for (int c2 = 0; c2 < CH; c2 += 2) {
                    uint32_t v[4];  // chunks c2 and c2 + 1, keys 0 .. 7 and 8 .. 15 of each
                    ldsm4t(v, row_at + from + c2 * 16);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = c2 + e, blk = BITS == 4 ? c : c / 2;
                        if (!WHOLE && blk >= gd) break;
                        if (BITS == 4 || e == 0) {
                            const uint32_t d0 = __shfl_sync(0xffffffffu, w[kt][0], 4 * blk + t4), d1 = __shfl_sync(0xffffffffu, w[kt][2], 4 * blk + t4);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if constexpr (FINE) {
                                    pd[nt][0] = fma2(p[nt][0], d0, mul2(rest[nt][0], d0));
                                    pd[nt][1] = fma2(p[nt][1], d1, mul2(rest[nt][1], d1));
                                    // ones in row blk (8 + blk) of the operand
                                    uint32_t ones[4];
                                    ldsm4(ones, row8 == blk && (sel & 1) == (G > 4 ? 0 : 1) ? plain + 16 : plain);
                                    mma16816<false>(G > 4 ? od[nt] : ob[nt], ones, pd[nt][0], pd[nt][1]);
                                } else {
                                    pd[nt][0] = mul2(p[nt][0], d0), pd[nt][1] = mul2(p[nt][1], d1);
                                }
                            }
                        }
                        const uint32_t v0 = v[2 * e], v1 = v[2 * e + 1];
                        if constexpr (BITS == 4) {
                            const uint32_t u0 = v0 >> 8, u1 = v1 >> 8;
                            const uint32_t a0[4] = {v0 & LO, v0 & HI, v1 & LO, v1 & HI}, a1[4] = {u0 & LO, u0 & HI, u1 & LO, u1 & HI};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816<false>(o[nt][2 * c], a0, pd[nt][0], pd[nt][1]);
                                mma16816<false>(o[nt][2 * c + 1], a1, pd[nt][0], pd[nt][1]);
                            }
                        } else {
                            const uint32_t a0[4] = {v0 & LO, v0 >> HS & HI, v1 & LO, v1 >> HS & HI};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[nt][c], a0, pd[nt][0], pd[nt][1]);
                        }
                    }
                }
            }
        }
        __syncwarp();  // every lane has read the keys and values
        mbar_arrive(smem_addr(&ring.empty[slot]), one);
        if (++slot == S::STAGES) slot = 0, parity ^= 1u;
    }
    if (ring.broken) {
        // (it cannot be in a correct run) what is still on its way is waited for, as far as that goes; no later row tile copies anything
        for (int x = 0; x < S::STAGES; ++x) (void)mbar_wait_bounded(smem_addr(&ring.full[x]), parity);
    }

    // ---- join the warps of each head, in the (now idle) ring
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);        // [WARPS][ROWS][LINE]
    float* stat = acc + S::WARPS * S::ROWS * S::LINE;   // [WARPS][ROWS][2]
    constexpr float U = 16777216.f, U4 = 1048576.f;     // 2^24, and 2^20 for a byte's upper half
    constexpr float Z = BITS == 4 ? 8.f : 128.f;
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
                const int h = gd + b;  // the half that block b's base is: its sum lies with the lanes of row h % 8
                const float lower = __shfl_sync(0xffffffffu, ob[nt][j], 4 * (h & 7) + t4), upper = __shfl_sync(0xffffffffu, ob[nt][j + 2], 4 * (h & 7) + t4);
                float add = G <= 4 || h < 8 ? lower : upper;
                if constexpr (FINE) {
                    const float step = __shfl_sync(0xffffffffu, ob[nt][j], 4 * b + t4);
                    const float rounded = __shfl_sync(0xffffffffu, G > 4 ? od[nt][j] : ob[nt][j + 2], 4 * b + t4);
                    add += Z * (step - rounded);
                }
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
    for (int i = threadIdx.x; i < heads * t.rows * (DP / 4); i += S::WARPS * 32) {
        const int hr = i / (DP / 4), d = i % (DP / 4) * 4, hh = hr / t.rows, r = hr - hh * t.rows;
        if (d >= a.dim) continue;
        float mm = NEG_INF;
        for (int w = hh; w < S::WARPS; w += heads) mm = fmaxf(mm, stat[(w * S::ROWS + r) * 2]);
        const float from = mm == NEG_INF ? 0.f : mm;
        float ll = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = hh; w < S::WARPS; w += heads) {
            const float f = exp2_approx(stat[(w * S::ROWS + r) * 2] - from);
            const float4 v = *reinterpret_cast<const float4*>(acc + (w * S::ROWS + r) * S::LINE + d);
            ll += f * stat[(w * S::ROWS + r) * 2 + 1];
            x.x += f * v.x, x.y += f * v.y, x.z += f * v.z, x.w += f * v.w;
        }
        own.kv_head = t.kv_head + hh;
        if (t.parts > 1) {
            const long long at = (record * S::WARPS + hh) * S::ROWS + r;
            __stcg(reinterpret_cast<float4*>(a.part_sum + at * a.dim + d), x);
            if (d == 0) __stcg(a.part_stat + at, make_float2(mm, ll));
        } else if (pa.bf16) {
            put_row4<true>(a, own, r, d, x, mm, ll);
        } else {
            put_row4<false>(a, own, r, d, x, mm, ll);
        }
    }
    // (the ring is written by copies again: what was written and read here comes before them)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Joins the parts of a row tile that begins in block t.index: four elements of up to four rows a thread, one pass over the parts with the maxima and
// the sums running along.  Eight parts of one row, or four of four, are on their way at once, what is left by twos: more (16, or copies into the ring
// as far ahead as it has room) took longer, since few blocks join and none has this code at hand (one of 100003: 8 42.0 us, 16 44.1; 25000
// 19.5 and 21.1; all of 16 before any is used 51.7).
template <int DP, int BITS, int NT, int ITEMS>
__device__ __forceinline__ void join_packed(const AttnPackedArgs& pa, const Tile& t) {
    using S = PackedShape<DP, BITS, NT>;
    constexpr int AT_ONCE = S::WARPS * 32 / (DP / 4), PARTS = ITEMS == 1 ? 8 : 16 / ITEMS;
    const AttnArgs& a = pa.a;
    const int d = threadIdx.x % (DP / 4) * 4, rows = t.rows << pa.hb_shift;
    if (d >= a.dim) return;
    Tile own = t;
#pragma unroll 1
    for (int first = threadIdx.x / (DP / 4); first < rows; first += AT_ONCE * ITEMS) {
        float m[ITEMS], l[ITEMS];
        float4 x[ITEMS];
        int rec[ITEMS];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            m[k] = NEG_INF, l[k] = 0.f, x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int hr = min(first + k * AT_ONCE, rows - 1), hh = hr / t.rows;  // (rows past the last one read its record)
            rec[k] = static_cast<int>(2 * t.index * S::WARPS + hh) * S::ROWS + hr - hh * t.rows;
        }
        auto take = [&](int p) {
            const int part = (2 * p + (p == 0 ? 1 : 0)) * S::WARPS * S::ROWS;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int at = rec[k] + part;
                const float2 s = __ldcg(a.part_stat + at);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_sum + static_cast<long long>(at) * a.dim + d));
                const float top = fmaxf(m[k], s.x), base = top == NEG_INF ? 0.f : top;
                const float keep = exp2_approx(m[k] - base), w = exp2_approx(s.x - base);
                m[k] = top;
                l[k] = l[k] * keep + w * s.y;
                x[k].x = x[k].x * keep + w * v.x, x[k].y = x[k].y * keep + w * v.y;
                x[k].z = x[k].z * keep + w * v.z, x[k].w = x[k].w * keep + w * v.w;
            }
        };
        int p = 0;
#pragma unroll 1
        for (; p + PARTS <= t.parts; p += PARTS) {
#pragma unroll
            for (int j = 0; j < PARTS; ++j) take(p + j);
        }
#pragma unroll 1
        for (; p + 2 <= t.parts; p += 2) {
#pragma unroll
            for (int j = 0; j < 2; ++j) take(p + j);
        }
#pragma unroll 1
        for (; p < t.parts; ++p) take(p);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int hr = first + k * AT_ONCE, hh = hr / t.rows, r = hr - hh * t.rows;
            if (hr >= rows) break;
            own.kv_head = t.kv_head + hh;
            if (pa.bf16) put_row4<true>(a, own, r, d, x[k], m[k], l[k]);
            else put_row4<false>(a, own, r, d, x[k], m[k], l[k]);
        }
    }
}

template <int DP, int BITS, int NT, bool WHOLE, bool FINE>
__global__ void __launch_bounds__(PackedShape<DP, BITS, NT>::WARPS * 32, PackedShape<DP, BITS, NT>::BLOCKS)
    attn_packed_kernel(const __grid_constant__ AttnPackedArgs pa) {
    using S = PackedShape<DP, BITS, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint4 plain[2];
    __shared__ Ring<S::STAGES> ring;
    __shared__ unsigned last;
    if (threadIdx.x < 8) reinterpret_cast<uint32_t*>(plain)[threadIdx.x] = threadIdx.x < 4 ? 0u : 0x3C003C00u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) mbar_init(smem_addr(&ring.full[i]), 1), mbar_init(smem_addr(&ring.empty[i]), S::WARPS);
        ring.broken = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    fence_copies();
    int slot = 0;
    unsigned parity = 0;
    divide_rows<S::ROWS, 16, true>(
        pa.a, pa.a.kv_heads >> pa.hb_shift, 1 << pa.hb_shift, pa.few, &last, smem,
        [&](const Tile& t, long long record) { attend_packed<DP, BITS, NT, WHOLE, FINE>(pa, t, record, smem, smem_addr(plain), ring, slot, parity); },
        [&](const Tile& t) {
            if ((t.rows << pa.hb_shift) <= S::WARPS * 32 / (DP / 4)) join_packed<DP, BITS, NT, 1>(pa, t);
            else join_packed<DP, BITS, NT, 4>(pa, t);
        });
}

template <int BITS, bool FINE, int DP, int NT, bool WHOLE>
static const void* packed_kernel(PackedLaunch* launch) {
    using S = PackedShape<DP, BITS, NT>;
    *launch = {S::SMEM, S::WARPS * 32u, S::BLOCKS, S::ROWS, S::WARPS};
    return (const void*)attn_packed_kernel<DP, BITS, NT, WHOLE, FINE>;
}

// Heads of up to 128 have kernels for up to 8 and up to 16 rows; those of 64, 128 and 256 kernels of their own.
template <int BITS, bool FINE>
const void* pick_packed(int dim, int rows, PackedLaunch* launch) {
    if (dim > 128) return dim == 256 ? packed_kernel<BITS, FINE, 256, 1, true>(launch) : packed_kernel<BITS, FINE, 256, 1, false>(launch);
    if (dim == 128) return rows <= 8 ? packed_kernel<BITS, FINE, 128, 1, true>(launch) : packed_kernel<BITS, FINE, 128, 2, true>(launch);
    if (dim == 64) return rows <= 8 ? packed_kernel<BITS, FINE, 64, 1, true>(launch) : packed_kernel<BITS, FINE, 64, 2, true>(launch);
    if (dim > 64) return rows <= 8 ? packed_kernel<BITS, FINE, 128, 1, false>(launch) : packed_kernel<BITS, FINE, 128, 2, false>(launch);
    return rows <= 8 ? packed_kernel<BITS, FINE, 64, 1, false>(launch) : packed_kernel<BITS, FINE, 64, 2, false>(launch);
}

}  // namespace qg
