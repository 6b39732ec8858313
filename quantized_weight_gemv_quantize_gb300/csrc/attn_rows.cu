// Attention of a few rows (decode, drafted tokens) over a paged cache: 16 rows a block, the keys split over its warps.
//
// Each warp walks its own 16-key pieces with its own ring of asynchronous copies and its own running maximum m and sum l
// (base 2): s = scale log2(e) q k, m' = max(m, s), p = 2^(s - m'), l = l 2^(m - m') + sum p, o = o 2^(m - m') + p v.  No
// barrier runs inside the loop; the warps' (m, l, o) are joined once at the end.  A decode step reads each key and value once
// for its whole group of query heads: the kernel is bound by those bytes.
//
// The grid is one wave of blocks whatever the batch.  All row tiles' keys, laid end to end, are cut into as many equal shares as there
// are blocks (from the lengths on the device: uneven contexts and loose bounds cost nothing); a block takes its share, which may
// be the end of one row tile, some whole ones and the start of another.  The parts of a row tile are joined through the scratch.
//
// 48 sequences of 2000 to 16384 tokens, 32 and 8 heads of 128: 208-214 us, 6.4 to 6.6 TB/s, 94 to 97% of a plain copy's rate (a grid of parts of
// 2048 keys: 264 us).  One sequence of 100003: 72 to 73 us, 5.6 to 5.7 TB/s; the rest is the one wave's start (3 us) and the joining of 38
// parts.  One of 777: 10.2 us call after call, 8.2 in a graph, all latency: launch, lengths, page table, keys, a counter, the parts.
#include "attn.cuh"

namespace qg {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    const int n = live ? 16 : 0;  // 0 source bytes: the 16 bytes are filled with zeros and src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
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

template <int DP>
struct RowsShape {
    static constexpr int WARPS = 4;
    static constexpr int STAGES = 3;
    static constexpr int ROW = DP * 2;            // bytes of one staged key
    static constexpr int STAGE = 2 * 16 * ROW;    // 16 keys and their values
    static constexpr unsigned SMEM = WARPS * STAGES * STAGE;
    // the joining of the warps reuses the ring: (m, l) and 16 rows of DP sums a warp
    static_assert(WARPS * 16 * (DP + 8 + 2) * 4 <= SMEM, "");
};

// Byte offset of 16-byte piece c of staged row r: the pieces of a row are permuted by the row (xor in the low three bits
// of the piece) so that the eight rows that a matrix load reads fall into different banks.
template <int DP>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
    return static_cast<uint32_t>(r * DP * 2 + ((c ^ (r & 7)) << 4));
}

// One row tile's part: into the result, or into its record.  Called by the whole block.
template <int DP, bool BF>
__device__ __forceinline__ void attend(const AttnArgs& a, const Tile& t, long long record, uint8_t* smem) {
    using S = RowsShape<DP>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t ring = smem_addr(smem) + warp * S::STAGES * S::STAGE;
    constexpr int PER_ROW = DP / 8;
    const int* table = a.pages + t.seq * a.pages_stride;
    const int pieces = (t.k1 - t.k0 + 15) / 16;
    const int mine = pieces > warp ? (pieces - warp + S::WARPS - 1) / S::WARPS : 0;
    const uint16_t* const kh = a.k + t.kv_head * a.k_head;
    const uint16_t* const vh = a.v + t.kv_head * a.v_head;
    const bool one_page = a.page_size % 16 == 0;  // pieces start at multiples of 16: all keys of one lie on one page

    // Where this warp's pieces lie.  With one page a piece, lane n holds page and token of piece 32 * batch + n, read a batch ahead.
    struct Where {
        int page, token;  // page -1: no such key
    };
    auto look_up = [&](int key) {
        const int nth = div_by(key, a.page_size, a.page_shift);
        Where w = {-1, key - nth * a.page_size};
        if (key < t.k1 && (one_page || key >= t.first)) {  // (with one page a piece, that of the piece's first key holds all others)
            w.page = table[nth];
            if (w.page < 0 || w.page >= a.num_pages) atomicOr(a.err, ERR_BAD_INDEX), w.page = -1;
        }
        return w;
    };
    auto key_of = [&](int i) { return t.k0 + (warp + i * S::WARPS) * 16; };
    Where batch = {-1, 0}, ahead = {-1, 0};
    if (one_page) batch = look_up(key_of(lane)), ahead = look_up(key_of(32 + lane));
    // Copies piece i into a slot of the ring; returns which of its keys are there, one bit each.
    auto issue = [&](int i, int slot) -> unsigned {
        const uint32_t kbase = ring + slot * S::STAGE, vbase = kbase + 16 * S::ROW;
        const int c = lane % PER_ROW, r_in = lane / PER_ROW;
        constexpr int STEP = 32 / PER_ROW;
        const bool col = c * 8 < a.dim;
        unsigned live = 0;
        if (one_page) {
            if (i && i % 32 == 0) batch = ahead, ahead = look_up(key_of(i + 32 + lane));
            const int page = __shfl_sync(0xffffffffu, batch.page, i % 32), token = __shfl_sync(0xffffffffu, batch.token, i % 32) + r_in;
            const int left = page < 0 ? 0 : t.k1 - key_of(i);
            live = left <= 0 ? 0u : left >= 16 ? 0xffffu : (1u << left) - 1u;
            live &= 0xffffu << max(0, t.first - key_of(i));  // (pieces start at most 15 keys before the first)
            const uint16_t* k = live ? kh + page * a.k_page + token * a.k_token + c * 8 : a.k;
            const uint16_t* v = live ? vh + page * a.v_page + token * a.v_token + c * 8 : a.v;
            const long long k_step = live ? STEP * a.k_token : 0, v_step = live ? STEP * a.v_token : 0;
#pragma unroll
            for (int r0 = 0; r0 < 16; r0 += STEP) {
                const bool in = (live >> (r0 + r_in) & 1u) && col;
                cp_async16(kbase + piece_at<DP>(r0 + r_in, c), k, in);
                cp_async16(vbase + piece_at<DP>(r0 + r_in, c), v, in);
                k += k_step, v += v_step;
            }
        } else {
            const Where w = look_up(key_of(i) + (lane & 15));
            live = __ballot_sync(0xffffffffu, w.page >= 0) & 0xffffu;
#pragma unroll 1
            for (int r0 = 0; r0 < 16; r0 += STEP) {
                const int page = __shfl_sync(0xffffffffu, w.page, r0 + r_in), token = __shfl_sync(0xffffffffu, w.token, r0 + r_in);
                const bool in = page >= 0 && col;
                cp_async16(kbase + piece_at<DP>(r0 + r_in, c), in ? kh + page * a.k_page + token * a.k_token + c * 8 : a.k, in);
                cp_async16(vbase + piece_at<DP>(r0 + r_in, c), in ? vh + page * a.v_page + token * a.v_token + c * 8 : a.v, in);
            }
        }
        return live;
    };

    // The query rows as operand fragments: lane holds rows lane/4 and lane/4 + 8, columns 2 (lane % 4) + {0, 1, 8, 9}.
    uint32_t qf[DP / 16][4];
    {
        const uint16_t* q = static_cast<const uint16_t*>(a.q);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = lane / 4 + 8 * hh;
            const uint16_t* src = q + out_at(a, t, min(r, t.rows - 1), a.q_token, a.q_head);
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d = kk * 16 + 8 * e + 2 * (lane % 4);
                    qf[kk][hh + 2 * e] = r < t.rows && d < a.dim ? *reinterpret_cast<const uint32_t*>(src + d) : 0u;
                }
        }
    }
    unsigned live_ring[S::STAGES] = {};  // which keys of a staged piece are there
    // keys that the lane's two rows see: lo <= key <= hi
    int lo[2], hi[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int pos = row_pos(a, t, lane / 4 + 8 * hh);
        hi[hh] = a.causal ? min(t.k1 - 1, pos) : t.k1 - 1;
        lo[hh] = first_key(a, pos);
    }

    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {NEG_INF, NEG_INF}, l[2] = {0.f, 0.f};

    // (the first rounds only fill the ring)
    for (int i = 1 - S::STAGES; i < mine; ++i) {
        cp_wait<S::STAGES - 2>();
        __syncwarp();  // piece i is there, and the slot that is filled next was read in the round before
        const unsigned live = live_ring[0];
#pragma unroll
        for (int j = 0; j + 1 < S::STAGES; ++j) live_ring[j] = live_ring[j + 1];
        const int next = i + S::STAGES - 1;
        live_ring[S::STAGES - 2] = next < mine ? issue(next, next % S::STAGES) : 0u;
        cp_commit();
        if (i < 0) continue;
        const int slot = i % S::STAGES;
        const uint32_t kbase = ring + slot * S::STAGE, vbase = kbase + 16 * S::ROW;
        float s[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
            uint32_t b[4];  // keys 0-7 and 8-15, each as two halves of the 16 columns
            ldsm4(b, kbase + piece_at<DP>((lane & 7) + (lane >> 4) * 8, kk * 2 + ((lane >> 3) & 1)));
            mma16816<BF>(s[0], qf[kk], b[0], b[1]);
            mma16816<BF>(s[1], qf[kk], b[2], b[3]);
        }
        const int key0 = t.k0 + (warp + i * S::WARPS) * 16;
        float top[2] = {NEG_INF, NEG_INF};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = nt * 8 + 2 * (lane % 4) + (e & 1), hh = e >> 1;
                const bool sees = (live >> c & 1u) && key0 + c >= lo[hh] && key0 + c <= hi[hh];
                s[nt][e] = sees ? s[nt][e] * a.scale_log2 : NEG_INF;
                top[hh] = fmaxf(top[hh], s[nt][e]);
            }
        float keep[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            top[hh] = fmaxf(top[hh], __shfl_xor_sync(0xffffffffu, top[hh], 1));
            top[hh] = fmaxf(top[hh], __shfl_xor_sync(0xffffffffu, top[hh], 2));
            const float mn = fmaxf(m[hh], top[hh] - Lift<BF>::ROWS);
            const float base = mn == NEG_INF ? 0.f : mn;  // a row that has seen nothing yet: 2^(-inf - 0) = 0
            keep[hh] = exp2_approx(m[hh] - base);
            m[hh] = mn;
            l[hh] *= keep[hh];
            top[hh] = base;
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nt][e] = exp2_approx(s[nt][e] - top[e >> 1]);
                l[e >> 1] += s[nt][e];
            }
        if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
            for (int d = 0; d < DP / 8; ++d)
                o[d][0] *= keep[0], o[d][1] *= keep[0], o[d][2] *= keep[1], o[d][3] *= keep[1];
        }
        const uint32_t p[4] = {pack16<BF>(s[0][0], s[0][1]), pack16<BF>(s[0][2], s[0][3]), pack16<BF>(s[1][0], s[1][1]),
                               pack16<BF>(s[1][2], s[1][3])};
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
            uint32_t b[4];  // columns d*16 .. +7 and +8 .. +15, each as keys 0-7 and 8-15
            ldsm4t(b, vbase + piece_at<DP>((lane & 7) + ((lane >> 3) & 1) * 8, d * 2 + (lane >> 4)));
            mma16816<BF>(o[2 * d], p, b[0], b[1]);
            mma16816<BF>(o[2 * d + 1], p, b[2], b[3]);
        }
    }
    cp_wait<0>();
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
    }

    // join the warps: each puts its rows into the (now idle) ring, rows 8 floats apart in the banks
    constexpr int LINE = DP + 8;
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);                // [WARPS][16][LINE]
    float* stat = acc + S::WARPS * 16 * LINE;                   // [WARPS][16][2]
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int r = lane / 4 + 8 * hh;
        if (8 * hh >= t.rows) break;
        if (lane % 4 == 0) stat[(warp * 16 + r) * 2] = m[hh], stat[(warp * 16 + r) * 2 + 1] = l[hh];
#pragma unroll
        for (int d = 0; d < DP / 8; ++d)
            *reinterpret_cast<float2*>(acc + (warp * 16 + r) * LINE + d * 8 + 2 * (lane % 4)) =
                make_float2(o[d][2 * hh], o[d][2 * hh + 1]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < t.rows * (DP / 4); i += S::WARPS * 32) {
        const int r = i / (DP / 4), d = i % (DP / 4) * 4;
        if (d >= a.dim) continue;
        float mm = NEG_INF;
#pragma unroll
        for (int w = 0; w < S::WARPS; ++w) mm = fmaxf(mm, stat[(w * 16 + r) * 2]);
        const float base = mm == NEG_INF ? 0.f : mm;
        float ll = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < S::WARPS; ++w) {
            const float f = exp2_approx(stat[(w * 16 + r) * 2] - base);
            const float4 v = *reinterpret_cast<const float4*>(acc + (w * 16 + r) * LINE + d);
            ll += f * stat[(w * 16 + r) * 2 + 1];
            x.x += f * v.x, x.y += f * v.y, x.z += f * v.z, x.w += f * v.w;
        }
        if (t.parts == 1) {
            put_row4<BF>(a, t, r, d, x, mm, ll);
        } else {
            __stcg(reinterpret_cast<float4*>(a.part_sum + (record + r) * a.dim + d), x);
            if (d == 0) __stcg(a.part_stat + record + r, make_float2(mm, ll));
        }
    }
}

// Joins the parts of a row tile that begins in block t.index: four elements of some rows a thread, one pass over the parts with the
// maxima and the sums running along.  Eight loads of each kind on their way at once: rows of one part, or parts of one row.
template <int DP, bool BF, int ITEMS>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const Tile& t) {
    constexpr int ROWS = RowsShape<DP>::WARPS * 32 / (DP / 4);
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

template <int DP, bool BF>
__global__ void __launch_bounds__(RowsShape<DP>::WARPS * 32) attn_rows_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ unsigned last;
    pdl_launch_dependents();
    pdl_wait();
    const unsigned lane = threadIdx.x % 32, me = blockIdx.x, blocks = gridDim.x, seqs = a.seqs, unit = a.unit_shift;
    // A sequence in the division of the work: its row tiles, each as many units of keys (64, or more where 32 bits would not
    // hold the whole) as any of its rows may see, at least one (a row that sees nothing has its zeros written).
    Seq sq = {};
    unsigned sq_units = 1, sq_tiles = 0;
    auto read_seq = [&](unsigned b) {
        sq_units = 1, sq_tiles = 0;
        if (b >= seqs) return;
        sq = find_seq(a, static_cast<int>(b));
        int lo, hi;
        find_keys(a, sq, 0, sq.n * a.group, 16, &lo, &hi);
        sq_tiles = (sq.n * a.group + 15) / 16 * a.kv_heads;
        sq_units = max(1u, (static_cast<unsigned>(hi - lo) + (1u << unit) - 1) >> unit);
    };
    // Sum over all sequences, 32 at a time (a lane each), every warp for itself.
    auto sum_of = [&](auto&& f) {
        unsigned v = 0;
        for (unsigned b0 = 0; b0 < seqs; b0 += 32) {
            if (seqs > 32) read_seq(b0 + lane);
            v += f();
        }
        return __reduce_add_sync(0xffffffffu, v);
    };
    if (seqs <= 32) read_seq(lane);
    const unsigned least = max(1u, 128u >> unit);  // less than 128 keys are not worth a block
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
        if (seqs > 32) read_seq(b0 + lane);
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
            sq.q0 = __shfl_sync(0xffffffffu, sq.q0, l), sq.n = __shfl_sync(0xffffffffu, sq.n, l);
            sq.first_pos = __shfl_sync(0xffffffffu, sq.first_pos, l), sq.usable = __shfl_sync(0xffffffffu, sq.usable, l);
            per = __shfl_sync(0xffffffffu, per, l), sq_tiles = __shfl_sync(0xffffffffu, sq_tiles, l);
            break;
        }
        at += __shfl_sync(0xffffffffu, sum, 31);
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
        if (sq.n * a.group <= 16) {
            t.kv_head = static_cast<int>(nth), t.row0 = 0;
        } else {
            const unsigned in_head = sq_tiles / a.kv_heads;
            t.kv_head = static_cast<int>(nth / in_head), t.row0 = static_cast<int>(nth % in_head * 16);
        }
        t.rows = min(16, sq.n * a.group - t.row0);
        int lo, hi;
        t.first = find_keys(a, sq, t.row0, t.rows, 16, &lo, &hi);
        t.k0 = lo + static_cast<int>(min(static_cast<unsigned long long>(hi - lo), static_cast<unsigned long long>(pos - tile_at) << unit));
        t.k1 = lo + static_cast<int>(min(static_cast<unsigned long long>(hi - lo), static_cast<unsigned long long>(stop - tile_at) << unit));
        // the blocks with the row tile's first and last part: this one where the tile begins or ends here
        const unsigned first = tile_at >= start ? me : tile_at / share;
        t.part = static_cast<int>(me - first);
        t.parts = static_cast<int>((tile_at + per <= end ? me : (tile_at + per - 1) / share) - first + 1);
        t.index = first;
        // A block has at most two parts of split row tiles: one that another block began (record 2 b) and one that it begins
        // itself (record 2 b + 1).
        attend<DP, BF>(a, t, (2 * me + (t.part == 0 ? 1 : 0)) * 16, smem);
        if (t.parts > 1) {
            // The block that arrives last joins the parts (in their order, so the result does not depend on which one that
            // is) and puts the counter back to zero.
            __syncthreads();
            if (threadIdx.x == 0) {  // (the block's writes before the barrier are released with this thread's)
                unsigned before;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(a.count + first) : "memory");
                last = before == static_cast<unsigned>(t.parts - 1);
                if (last) a.count[first] = 0;
            }
            __syncthreads();
            if (last) {
                if (t.rows <= RowsShape<DP>::WARPS * 32 / (DP / 4)) join_rows<DP, BF, 1>(a, t);
                else join_rows<DP, BF, DP / 32>(a, t);
            }
        }
        __syncthreads();  // shared memory is free again
        pos = stop, ++nth;
    }
}

template <int DP>
static const void* pick(bool bf16, unsigned* smem, unsigned* threads) {
    *smem = RowsShape<DP>::SMEM;
    *threads = RowsShape<DP>::WARPS * 32;
    return bf16 ? (const void*)attn_rows_kernel<DP, true> : (const void*)attn_rows_kernel<DP, false>;
}

const void* attn_rows_kernel_ptr(bool bf16, int dim, unsigned* smem, unsigned* threads) {
    if (dim <= 64) return pick<64>(bf16, smem, threads);
    return dim <= 128 ? pick<128>(bf16, smem, threads) : pick<256>(bf16, smem, threads);
}

}  // namespace qg
