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
#include "attn_rows.cuh"

namespace qg {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    const int n = live ? 16 : 0;  // 0 source bytes: the 16 bytes are filled with zeros and src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
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

// KEEP: the division over the blocks keeps the sequences in shared memory, for many of them: that takes registers and code that few pay for.  With it and without,
// us in a graph: one sequence of 777 9.3 / 9.05, 40 with 5 drafts each 59.7 / 57.8, 48 of up to 16384 211.3 / 210.4, 300 of up to 2000 182.6 / 183.4, 1000 of up to
// 600 215.4 / 223.0.
template <int DP, bool BF, bool KEEP>
__global__ void __launch_bounds__(RowsShape<DP>::WARPS * 32) attn_rows_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ unsigned last;
    pdl_launch_dependents();
    pdl_wait();
    divide_rows<16, 16, KEEP>(
        a, a.kv_heads, 1, 128, &last, smem, [&](const Tile& t, long long record) { attend<DP, BF>(a, t, record * 16, smem); },
        [&](const Tile& t) {
            constexpr int THREADS = RowsShape<DP>::WARPS * 32;
            if (t.rows <= THREADS / (DP / 4)) join_rows<DP, THREADS, BF, 1>(a, t);
            else join_rows<DP, THREADS, BF, DP / 32>(a, t);
        });
}

template <int DP>
static const void* pick(bool bf16, int seqs, unsigned* smem, unsigned* threads) {
    *smem = RowsShape<DP>::SMEM;
    *threads = RowsShape<DP>::WARPS * 32;
    if (seqs >= 300) return bf16 ? (const void*)attn_rows_kernel<DP, true, true> : (const void*)attn_rows_kernel<DP, false, true>;
    return bf16 ? (const void*)attn_rows_kernel<DP, true, false> : (const void*)attn_rows_kernel<DP, false, false>;
}

const void* attn_rows_kernel_ptr(bool bf16, int dim, int seqs, unsigned* smem, unsigned* threads) {
    if (dim <= 64) return pick<64>(bf16, seqs, smem, threads);
    return dim <= 128 ? pick<128>(bf16, seqs, smem, threads) : pick<256>(bf16, seqs, smem, threads);
}

}  // namespace qg
