// Attention of a few rows (decode, drafted tokens) over a paged cache: 16 rows a block, the keys split over its warps.
//
// Each warp walks its own 16-key pieces with its own ring of asynchronous copies and its own running maximum m and sum l
// (base 2): s = scale log2(e) q k, m' = max(m, s), p = 2^(s - m'), l = l 2^(m - m') + sum p, o = o 2^(m - m') + p v.  No
// barrier runs inside the loop; the warps' (m, l, o) are joined once at the end, and the parts of a context that is split
// over several blocks likewise through the scratch.  A decode step reads each key and value once for its whole group of
// query heads: the kernel is bound by those bytes.
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
    static constexpr int WARPS = DP <= 128 ? 8 : 4;
    static constexpr int STAGES = 3;
    static constexpr int ROW = DP * 2;            // bytes of one staged key
    static constexpr int STAGE = 2 * 16 * ROW;    // 16 keys and their values
    static constexpr unsigned SMEM = WARPS * STAGES * STAGE;
    // the joining of the warps reuses the ring: (m, l) and 16 rows of DP sums a warp
    static_assert(WARPS * 16 * (DP + 2) * 4 <= SMEM, "");
};

// Byte offset of 16-byte piece c of staged row r: the pieces of a row are permuted by the row (xor in the low three bits
// of the piece) so that the eight rows that a matrix load reads fall into different banks.
template <int DP>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
    return static_cast<uint32_t>(r * DP * 2 + ((c ^ (r & 7)) << 4));
}

template <int DP, bool BF>
__global__ void __launch_bounds__(RowsShape<DP>::WARPS * 32) attn_rows_kernel(const AttnArgs a) {
    using S = RowsShape<DP>;
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_launch_dependents();
    pdl_wait();
    Tile t;
    if (!find_tile<16, false>(a, blockIdx.x, &t)) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t ring = smem_addr(smem) + warp * S::STAGES * S::STAGE;

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
    // keys that the lane's two rows see: lo <= key <= hi
    int lo[2], hi[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int pos = row_pos(a, t, lane / 4 + 8 * hh);
        hi[hh] = a.causal ? min(t.k1 - 1, pos) : t.k1 - 1;
        lo[hh] = a.window > 0 ? pos - a.window + 1 : 0;
    }

    const int* table = a.pages + t.seq * a.pages_stride;
    const int pieces = (t.k1 - t.k0 + 15) / 16;
    const int mine = pieces > warp ? (pieces - warp + S::WARPS - 1) / S::WARPS : 0;
    unsigned live_ring[S::STAGES];  // which keys of a staged piece are there, one bit each

    auto issue = [&](int i, int slot) -> unsigned {
        const int key0 = t.k0 + (warp + i * S::WARPS) * 16;
        // lanes 0..15 look up one key each
        const int key = key0 + (lane & 15);
        bool live = key < t.k1;
        long long ko = 0, vo = 0;
        if (live) {
            const int page = table[key / a.page_size], off = key % a.page_size;
            live = page >= 0 && page < a.num_pages;
            if (!live && lane < 16) atomicOr(a.err, ERR_BAD_INDEX);
            if (live) {
                ko = page * a.k_page + off * a.k_token + t.kv_head * a.k_head;
                vo = page * a.v_page + off * a.v_token + t.kv_head * a.v_head;
            }
        }
        const unsigned mask = __ballot_sync(0xffffffffu, live);
        const uint32_t kbase = ring + slot * S::STAGE, vbase = kbase + 16 * S::ROW;
        constexpr int PER_ROW = DP / 8;
#pragma unroll
        for (int j = 0; j < 16 * PER_ROW / 32; ++j) {
            const int idx = j * 32 + lane, r = idx / PER_ROW, c = idx % PER_ROW;
            const long long kr = __shfl_sync(0xffffffffu, ko, r), vr = __shfl_sync(0xffffffffu, vo, r);
            const bool in = (mask >> r & 1u) && c * 8 < a.dim;
            cp_async16(kbase + piece_at<DP>(r, c), a.k + (in ? kr + c * 8 : 0), in);
            cp_async16(vbase + piece_at<DP>(r, c), a.v + (in ? vr + c * 8 : 0), in);
        }
        return mask & 0xffffu;
    };

    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {NEG_INF, NEG_INF}, l[2] = {0.f, 0.f};

#pragma unroll
    for (int s = 0; s < S::STAGES - 1; ++s) {
        live_ring[s] = s < mine ? issue(s, s) : 0u;
        cp_commit();
    }
    live_ring[S::STAGES - 1] = 0u;
    for (int i = 0; i < mine; ++i) {
        const int slot = i % S::STAGES;
        cp_wait<S::STAGES - 2>();
        __syncwarp();
        unsigned live = live_ring[0];
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
        __syncwarp();  // the slot that is filled next was read in the iteration before this one
#pragma unroll
        for (int j = 0; j + 1 < S::STAGES; ++j) live_ring[j] = live_ring[j + 1];
        const int next = i + S::STAGES - 1;
        live_ring[S::STAGES - 2] = next < mine ? issue(next, next % S::STAGES) : 0u;
        cp_commit();
    }
    cp_wait<0>();
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
    }

    // join the warps: each puts its rows into the (now idle) ring
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);                // [WARPS][16][DP]
    float* stat = acc + S::WARPS * 16 * DP;                     // [WARPS][16][2]
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int r = lane / 4 + 8 * hh;
        if (lane % 4 == 0) stat[(warp * 16 + r) * 2] = m[hh], stat[(warp * 16 + r) * 2 + 1] = l[hh];
#pragma unroll
        for (int d = 0; d < DP / 8; ++d)
            *reinterpret_cast<float2*>(acc + (warp * 16 + r) * DP + d * 8 + 2 * (lane % 4)) =
                make_float2(o[d][2 * hh], o[d][2 * hh + 1]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < t.rows * (DP / 2); i += S::WARPS * 32) {
        const int r = i / (DP / 2), d = i % (DP / 2) * 2;
        if (d >= a.dim) continue;
        float mm = NEG_INF;
#pragma unroll
        for (int w = 0; w < S::WARPS; ++w) mm = fmaxf(mm, stat[(w * 16 + r) * 2]);
        const float base = mm == NEG_INF ? 0.f : mm;
        float ll = 0.f, x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < S::WARPS; ++w) {
            const float f = exp2_approx(stat[(w * 16 + r) * 2] - base);
            const float2 v = *reinterpret_cast<const float2*>(acc + (w * 16 + r) * DP + d);
            ll += f * stat[(w * 16 + r) * 2 + 1];
            x += f * v.x, y += f * v.y;
        }
        if (t.parts == 1) {
            const float inv = ll > 0.f ? 1.f / ll : 0.f;
            const long long at = out_at(a, t, r, a.out_token, a.out_head);
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at + d) = pack16<BF>(x * inv, y * inv);
            if (d == 0) put_lse(a, t, r, mm, ll);
        } else {
            float* rec = part_row(a, t, t.part, r);
            __stcg(reinterpret_cast<float2*>(rec + 2 + d), make_float2(x, y));
            if (d == 0) __stcg(reinterpret_cast<float2*>(rec), make_float2(mm, ll));
        }
    }
    if (t.parts > 1) join_parts<BF>(a, t);
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
