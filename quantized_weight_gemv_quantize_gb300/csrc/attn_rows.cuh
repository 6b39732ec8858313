// What the attention kernels of a few rows share: matrix instructions of a warp, and the division of a batch over one wave of blocks.
#pragma once
#include "attn.cuh"

namespace qg {

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Joins the parts of a row tile that begins in block t.index: four elements of some rows a thread, one pass over the parts with the
// maxima and the sums running along.  Eight loads of each kind on their way at once: rows of one part, or parts of one row.
template <int DP, int THREADS, bool BF, int ITEMS>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const Tile& t) {
    constexpr int ROWS = THREADS / (DP / 4);
    const int r0 = threadIdx.x / (DP / 4), d = threadIdx.x % (DP / 4) * 4;
    if (d >= a.dim || r0 >= t.rows) return;
    float m[ITEMS], l[ITEMS];
    float4 x[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) m[k] = NEG_INF, l[k] = 0.f, x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int rec0 = 2 * static_cast<int>(t.index) * 16 + r0;
#pragma unroll(8 / ITEMS)
    for (int p = 0; p < t.parts; ++p) {
        const int rec = rec0 + p * 32 + (p == 0 ? 16 : 0);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            // (rows past the tile's read its last one's record)
            const int at = rec + min(k * ROWS, t.rows - 1 - r0);
            const float2 s = __ldcg(a.part_stat + at);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_sum + static_cast<long long>(at) * a.dim + d));
            const float top = fmaxf(m[k], s.x), base = top == NEG_INF ? 0.f : top;
            const float keep = exp2_approx(m[k] - base), w = exp2_approx(s.x - base);
            m[k] = top;
            l[k] = l[k] * keep + w * s.y;
            x[k].x = x[k].x * keep + w * v.x, x[k].y = x[k].y * keep + w * v.y;
            x[k].z = x[k].z * keep + w * v.z, x[k].w = x[k].w * keep + w * v.w;
        }
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (r0 + k * ROWS < t.rows) put_row4<BF>(a, t, r0 + k * ROWS, d, x[k], m[k], l[k]);
}

// A block's parts of the batch's row tiles, one after another: attend(t, record) computes one, into the result or into its record, join(t) joins the
// parts of one; both are called by the whole block.  A row tile is ROWS rows of each of `heads` key/value heads, `groups` times those make all of
// them.  Ranges of keys begin at multiples of STEP; less than `few` keys are not worth a block.  `last` and `room`
// (with KEEP KEPT pairs of words, free until attend is called) are in shared memory.
constexpr unsigned KEPT = 1024;
template <int ROWS, int STEP, bool KEEP, class Attend, class Join>
__device__ __forceinline__ void divide_rows(const AttnArgs& a, int groups, int heads, unsigned few, unsigned* last, void* room, Attend&& attend, Join&& join) {
    const unsigned lane = threadIdx.x % 32, me = blockIdx.x, blocks = gridDim.x, seqs = a.seqs, unit = a.unit_shift;
    // A sequence in the division of the work: its row tiles, each as many units of keys (64, over a packed cache 32, or more where 32 bits would not
    // hold the whole) as any of its rows may see, at least one (a row that sees nothing has its zeros written).
    Seq sq = {};
    unsigned sq_units = 1, sq_tiles = 0;
    auto read_seq = [&](unsigned b) {
        sq_units = 1, sq_tiles = 0;
        if (b >= seqs) return;
        sq = find_seq(a, static_cast<int>(b));
        int lo, hi;
        find_keys(a, sq, 0, sq.n * a.group, STEP, &lo, &hi);
        sq_tiles = (sq.n * a.group + ROWS - 1) / ROWS * groups;
        sq_units = max(1u, (static_cast<unsigned>(hi - lo) + (1u << unit) - 1) >> unit);
    };
    // The division goes over the sequences some ten times: up to 32 stay in registers, a lane each, with KEEP up to KEPT in shared memory.
    uint2* const kept = static_cast<uint2*>(room);
    const bool keep = KEEP && seqs > 32 && seqs <= KEPT;
    if (seqs <= 32) read_seq(lane);
    if (keep) {
        for (unsigned b = threadIdx.x; b < seqs; b += blockDim.x) read_seq(b), kept[b] = make_uint2(sq_units, sq_tiles);
        __syncthreads();
    }
    auto count_seq = [&](unsigned b) {
        if (!keep) return read_seq(b);
        const uint2 u = b < seqs ? kept[b] : make_uint2(1u, 0u);
        sq_units = u.x, sq_tiles = u.y;
    };
    // Sum over all sequences, 32 at a time (a lane each), every warp for itself.
    auto sum_of = [&](auto&& f) {
        unsigned v = 0;
        for (unsigned b0 = 0; b0 < seqs; b0 += 32) {
            if (seqs > 32) count_seq(b0 + lane);
            v += f();
        }
        return __reduce_add_sync(0xffffffffu, v);
    };
    const unsigned least = max(1u, few >> unit);
    const unsigned units = sum_of([&] { return sq_tiles * sq_units; }), row_tiles = sum_of([&] { return sq_tiles; });
    // A block's share.  Where there are no more row tiles than blocks, it is made as long as it takes for every block to have a part
    // of one row tile only: a second part costs a block's start and end again, some 400 keys' time.  The row tiles' keys are then
    // counted in whole shares.
    const unsigned even = max(least, (units + blocks - 1) / blocks);
    unsigned share = even;
    bool whole = row_tiles <= blocks;
    for (int n = 0; whole; ++n) {
        const unsigned need = sum_of([&] { return sq_tiles * ((sq_units + share - 1) / share); });
        if (need <= blocks) break;
        if (n == 6) whole = false, share = even;
        else share = max(share + 1, static_cast<unsigned>(static_cast<unsigned long long>(share) * need / blocks));
    }
    auto counted = [&] { return whole ? (sq_units + share - 1) / share * share : sq_units; };
    // the sequence that holds this block's start, and where it begins
    const unsigned start = me * share;
    unsigned at = 0, b = seqs, per = 1;
    for (unsigned b0 = 0; b0 < seqs; b0 += 32) {
        if (seqs > 32) count_seq(b0 + lane);
        per = counted();
        const unsigned own = sq_tiles * per;
        unsigned sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        const unsigned holds = __ballot_sync(0xffffffffu, start < at + sum);
        if (holds) {
            const int l = __ffs(holds) - 1;
            b = b0 + l;
            at += __shfl_sync(0xffffffffu, sum - own, l);
            per = __shfl_sync(0xffffffffu, per, l);
            if (keep) {
                read_seq(b);
                break;
            }
            sq.q0 = __shfl_sync(0xffffffffu, sq.q0, l), sq.n = __shfl_sync(0xffffffffu, sq.n, l);
            sq.first_pos = __shfl_sync(0xffffffffu, sq.first_pos, l), sq.usable = __shfl_sync(0xffffffffu, sq.usable, l);
            sq_tiles = __shfl_sync(0xffffffffu, sq_tiles, l);
            break;
        }
        at += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (keep) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (copies may write there next)
        __syncthreads();
    }
    if (b == seqs) return;  // past the end of the work
    unsigned nth = (start - at) / per;

    for (unsigned pos = start, end = start + share; pos < end;) {
        while (nth >= sq_tiles) {  // the next sequence with rows
            at += sq_tiles * per;
            if (++b >= seqs) return;
            read_seq(b);
            per = counted(), nth = 0;
        }
        const unsigned tile_at = at + nth * per;  // the row tile's first unit in the whole work
        const unsigned stop = min(end, tile_at + per);
        Tile t;
        t.seq = static_cast<int>(b);
        t.q0 = sq.q0, t.first_pos = sq.first_pos;
        if (sq.n * a.group <= ROWS) {
            t.kv_head = static_cast<int>(nth) * heads, t.row0 = 0;
        } else {
            const unsigned in_head = sq_tiles / groups;
            t.kv_head = static_cast<int>(nth / in_head) * heads, t.row0 = static_cast<int>(nth % in_head * ROWS);
        }
        t.rows = min(ROWS, sq.n * a.group - t.row0);
        int lo, hi;
        t.first = find_keys(a, sq, t.row0, t.rows, STEP, &lo, &hi);
        t.k0 = lo + static_cast<int>(min(static_cast<unsigned long long>(hi - lo), static_cast<unsigned long long>(pos - tile_at) << unit));
        t.k1 = lo + static_cast<int>(min(static_cast<unsigned long long>(hi - lo), static_cast<unsigned long long>(stop - tile_at) << unit));
        // the blocks with the row tile's first and last part: this one where the tile begins or ends here
        const unsigned first = tile_at >= start ? me : tile_at / share;
        t.part = static_cast<int>(me - first);
        t.parts = static_cast<int>((tile_at + per <= end ? me : (tile_at + per - 1) / share) - first + 1);
        t.index = first;
        // A block has at most two parts of split row tiles: one that another block began (record 2 b) and one that it begins
        // itself (record 2 b + 1).
        attend(t, 2 * me + (t.part == 0 ? 1 : 0));
        if (t.parts > 1) {
            // The block that arrives last joins the parts (in their order, so the result does not depend on which one that
            // is) and puts the counter back to zero.
            __syncthreads();
            if (threadIdx.x == 0) {  // (the block's writes before the barrier are released with this thread's)
                unsigned before;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(a.count + first) : "memory");
                *last = before == static_cast<unsigned>(t.parts - 1);
                if (*last) a.count[first] = 0;
            }
            __syncthreads();
            if (*last) join(t);
        }
        __syncthreads();  // shared memory is free again
        pos = stop, ++nth;
    }
}

}  // namespace qg
