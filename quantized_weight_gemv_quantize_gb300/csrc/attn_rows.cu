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

// What a sequence counts for in the division of the work: each of its row tiles as many keys as any of its rows may see, in
// units of the block's 64 keys, at least one (a row that sees nothing has its zeros written).
__device__ __forceinline__ int share_of(const AttnArgs& a, const Seq& s) {
    int lo, hi;
    find_keys(a, s, 0, s.n * a.group, &lo, &hi);
    return max(64, (hi - lo + 63) / 64 * 64);
}
__device__ __forceinline__ int tiles_of(const AttnArgs& a, const Seq& s) { return (s.n * a.group + 15) / 16 * a.kv_heads; }

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

    // Page and token of key lane % 16 of this warp's piece i, read well before the piece is copied; page -1: no such key.
    struct Where {
        int page, token;
    };
    auto look_up = [&](int i) {
        const int key = t.k0 + (warp + i * S::WARPS) * 16 + (lane & 15), nth = div_by(key, a.page_size, a.page_shift);
        Where w = {-1, key - nth * a.page_size};
        if (i < mine && key < t.k1) {
            w.page = table[nth];
            if (w.page < 0 || w.page >= a.num_pages) atomicOr(a.err, ERR_BAD_INDEX), w.page = -1;
        }
        return w;
    };
    // Copies piece i into a slot of the ring; returns which of its keys are there, one bit each.
    auto issue = [&](const Where& w, int slot) -> unsigned {
        const unsigned live = __ballot_sync(0xffffffffu, w.page >= 0) & 0xffffu;
        const uint32_t kbase = ring + slot * S::STAGE, vbase = kbase + 16 * S::ROW;
        const int c = lane % PER_ROW;
        const bool col = c * 8 < a.dim;
        const int page0 = __shfl_sync(0xffffffffu, w.page, 0), token0 = __shfl_sync(0xffffffffu, w.token, 0);
        if (one_page) {
            const uint16_t* k = kh + page0 * a.k_page + (token0 + lane / PER_ROW) * a.k_token + c * 8;
            const uint16_t* v = vh + page0 * a.v_page + (token0 + lane / PER_ROW) * a.v_token + c * 8;
#pragma unroll
            for (int j = 0; j < 16 * PER_ROW / 32; ++j) {
                const int r = j * (32 / PER_ROW) + lane / PER_ROW;
                const bool in = (live >> r & 1u) && col;
                cp_async16(kbase + piece_at<DP>(r, c), in ? k + j * (32 / PER_ROW) * a.k_token : a.k, in);
                cp_async16(vbase + piece_at<DP>(r, c), in ? v + j * (32 / PER_ROW) * a.v_token : a.v, in);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16 * PER_ROW / 32; ++j) {
                const int r = j * (32 / PER_ROW) + lane / PER_ROW;
                const int page = __shfl_sync(0xffffffffu, w.page, r), token = __shfl_sync(0xffffffffu, w.token, r);
                const bool in = page >= 0 && col;
                cp_async16(kbase + piece_at<DP>(r, c), in ? kh + page * a.k_page + token * a.k_token + c * 8 : a.k, in);
                cp_async16(vbase + piece_at<DP>(r, c), in ? vh + page * a.v_page + token * a.v_token + c * 8 : a.v, in);
            }
        }
        return live;
    };

    Where first[S::STAGES - 1];
#pragma unroll
    for (int s = 0; s < S::STAGES - 1; ++s) first[s] = look_up(s);
    Where next = look_up(S::STAGES - 1);

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
    unsigned live_ring[S::STAGES];  // which keys of a staged piece are there
#pragma unroll
    for (int s = 0; s < S::STAGES - 1; ++s) {
        live_ring[s] = issue(first[s], s);
        cp_commit();
    }
    live_ring[S::STAGES - 1] = 0u;
    // keys that the lane's two rows see: lo <= key <= hi
    int lo[2], hi[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int pos = row_pos(a, t, lane / 4 + 8 * hh);
        hi[hh] = a.causal ? min(t.k1 - 1, pos) : t.k1 - 1;
        lo[hh] = a.window > 0 ? pos - a.window + 1 : 0;
    }

    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {NEG_INF, NEG_INF}, l[2] = {0.f, 0.f};

    for (int i = 0; i < mine; ++i) {
        const int slot = i % S::STAGES;
        cp_wait<S::STAGES - 2>();
        __syncwarp();  // the piece is there, and the slot that is filled next was read in the iteration before
        const unsigned live = live_ring[0];
#pragma unroll
        for (int j = 0; j + 1 < S::STAGES; ++j) live_ring[j] = live_ring[j + 1];
        live_ring[S::STAGES - 2] = issue(next, (i + S::STAGES - 1) % S::STAGES);
        cp_commit();
        next = look_up(i + S::STAGES);
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
            const float mn = fmaxf(m[hh], top[hh]);
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
            const float inv = ll > 0.f ? 1.f / ll : 0.f;
            const long long at = out_at(a, t, r, a.out_token, a.out_head);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at + d) =
                make_uint2(pack16<BF>(x.x * inv, x.y * inv), pack16<BF>(x.z * inv, x.w * inv));
            if (d == 0) put_lse(a, t, r, mm, ll);
        } else {
            __stcg(reinterpret_cast<float4*>(a.part_sum + (record + r) * a.dim + d), x);
            if (d == 0) __stcg(a.part_stat + record + r, make_float2(mm, ll));
        }
    }
}

template <int DP, bool BF>
__global__ void __launch_bounds__(RowsShape<DP>::WARPS * 32) attn_rows_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ unsigned last;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    // The whole work, and this block's share [start, end) of it: 32 sequences at a time, every warp for itself.
    auto work_of = [&](int b) {
        if (b >= a.seqs) return 0ll;
        const Seq s = find_seq(a, b);
        return static_cast<long long>(tiles_of(a, s)) * share_of(a, s);
    };
    auto scan = [&](long long v) {  // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        return v;
    };
    long long total = 0, own = 0, sum = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        own = work_of(b0 + lane);
        sum = scan(own);
        total += __shfl_sync(0xffffffffu, sum, 31);
    }
    // (at least 128 keys: less is not worth a block)
    const long long share = max(128ll, (div_wide(total + gridDim.x - 1, gridDim.x) + 63) / 64 * 64);
    const long long start = blockIdx.x * share, end = min(total, start + share);
    if (start >= total) return;
    // the sequence that holds the start, and where it begins
    int b = 0;
    long long at = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        if (a.seqs > 32) own = work_of(b0 + lane), sum = scan(own);  // (else from above)
        const unsigned holds = __ballot_sync(0xffffffffu, start < at + sum);
        if (holds) {
            const int l = __ffs(holds) - 1;
            b = b0 + l;
            at += __shfl_sync(0xffffffffu, sum - own, l);
            break;
        }
        at += __shfl_sync(0xffffffffu, sum, 31);
    }
    Seq s = find_seq(a, b);
    int per = share_of(a, s), tiles = tiles_of(a, s), nth = static_cast<int>(div_wide(start - at, per));

    for (long long pos = start; pos < end;) {
        while (nth >= tiles) {  // the next sequence with rows
            at += static_cast<long long>(tiles) * per;
            s = find_seq(a, ++b);
            per = share_of(a, s), tiles = tiles_of(a, s), nth = 0;
        }
        const long long tile_at = at + static_cast<long long>(nth) * per;  // the row tile's first key in the whole work
        const long long stop = min(end, tile_at + per);
        Tile t;
        t.seq = b;
        t.q0 = s.q0, t.first_pos = s.first_pos;
        if (s.n * a.group <= 16) {
            t.kv_head = nth, t.row0 = 0;
        } else {
            const int row_tiles = tiles / a.kv_heads;
            t.kv_head = nth / row_tiles, t.row0 = nth % row_tiles * 16;
        }
        t.rows = min(16, s.n * a.group - t.row0);
        int lo, hi;
        find_keys(a, s, t.row0, t.rows, &lo, &hi);
        t.k0 = min(hi, lo + static_cast<int>(pos - tile_at));
        t.k1 = min(hi, lo + static_cast<int>(stop - tile_at));
        // the block with the row tile's first part: this one where the tile begins here
        const int first = tile_at >= start ? static_cast<int>(blockIdx.x) : static_cast<int>(div_wide(tile_at, share));
        t.part = static_cast<int>(blockIdx.x) - first;
        t.parts = (tile_at + per <= end ? static_cast<int>(blockIdx.x) : static_cast<int>(div_wide(tile_at + per - 1, share))) - first + 1;
        t.index = first;
        // A block has at most two parts of split row tiles: one that another block began (record 2 b) and one that it begins
        // itself (record 2 b + 1).
        attend<DP, BF>(a, t, (2ll * blockIdx.x + (t.part == 0 ? 1 : 0)) * 16, smem);
        if (t.parts > 1) {
            // The block that arrives last joins the parts (in their order, so the result does not depend on which one that
            // is) and puts the counter back to zero.
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) last = atomicAdd(a.count + first, 1u) == static_cast<unsigned>(t.parts - 1);
            __syncthreads();
            if (last) {
                __threadfence();
                if (threadIdx.x == 0) a.count[first] = 0;
                for (int r = warp; r < t.rows; r += RowsShape<DP>::WARPS)
                    join_row<(DP + 127) / 128, BF>(a, t, r, [&](int p) { return (2ll * (first + p) + (p == 0 ? 1 : 0)) * 16 + r; });
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
