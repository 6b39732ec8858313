// Attention of many rows (chunks of a prompt, whole prompts) over a paged cache on the fifth-generation tensor cores: two
// tiles of 128 rows a block against tiles of 128 keys.
//
// For each key tile j and row tile i: S_i = Q_i K_j^T into tensor memory (fp32), softmax by one thread a row, P_i (16 bits)
// back into the upper half of S_i's columns, O_i += P_i V_j with P_i read from tensor memory.  While the tensor cores work
// on one row tile, the other's softmax runs.  The running maximum that the exponent is taken against moves only when the
// true one has grown by more than 2^8: then O_i and l are rescaled; p stays below 2^8, so nothing is lost by the delay.
// The keys of a tile lie on pages anywhere: four warps look the rows up and copy them 16 bytes at a time into the
// 128-byte-swizzled layout that the tensor cores read (K as the K-major, V as the MN-major operand: no transpose is made).
// 4 D flops a pair of row and key against one exponential: at D = 128 the tensor cores bound it.
#include "attn.cuh"

namespace qg {

constexpr int TR = 128;          // rows of a row tile
constexpr int TK = 128;          // keys of a key tile
constexpr int TILE_THREADS = 13 * 32;
constexpr int LOAD_WARP = 8, MMA_WARP = 12;

template <int DP>
struct TilesShape {
    static constexpr int HALVES = DP / 64;               // 64-column halves: one swizzled row of 128 bytes each
    static constexpr uint32_t HALF_BYTES = TK * 128;
    static constexpr uint32_t TILE_BYTES = HALVES * HALF_BYTES;
    static constexpr uint32_t Q_AT = 0;                  // two row tiles
    static constexpr uint32_t K_AT = 2 * TILE_BYTES;     // two stages
    static constexpr uint32_t V_AT = 4 * TILE_BYTES;     // two stages
    static constexpr uint32_t BYTES = 6 * TILE_BYTES;
    static constexpr unsigned SMEM = BYTES + 1024;       // the tiles start at a multiple of 1024
    // tensor memory columns (512 allocated): scores of the two row tiles, then their sums
    static constexpr uint32_t S_COL = 0, O_COL = 2 * TK;
};

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory operand: 128-byte swizzle, 16-byte units; lbo between 64-column groups (MN-major), sbo between groups of
// eight 128-byte rows.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(lbo >> 4) << 16 |
           static_cast<uint64_t>(sbo >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// D fp32, A and B both bf16 or both f16, M = 128; transb: B is MN-major.
template <bool BF>
__device__ __forceinline__ constexpr uint32_t tc_idesc(int n, bool transb) {
    return 1u << 4 | (BF ? 1u : 0u) << 7 | (BF ? 1u : 0u) << 10 | (transb ? 1u : 0u) << 16 |
           static_cast<uint32_t>(n / 8) << 17 | static_cast<uint32_t>(TR / 16) << 24;
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

#define QG_R32(X) X(0), X(1), X(2), X(3), X(4), X(5), X(6), X(7), X(8), X(9), X(10), X(11), X(12), X(13), X(14), X(15), X(16), \
        X(17), X(18), X(19), X(20), X(21), X(22), X(23), X(24), X(25), X(26), X(27), X(28), X(29), X(30), X(31)
#define QG_LIST32 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}"

// 32 columns of this warp's 32 lanes (one row a thread); valid after tc_wait_ld.
__device__ __forceinline__ void tc_ld32(float (&r)[32], uint32_t addr) {
#define X(i) "=f"(r[i])
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " QG_LIST32 ", [%32];" : QG_R32(X) : "r"(addr) : "memory");
#undef X
}
// The registers pass through the wait, so that no use of them can be moved before it.
__device__ __forceinline__ void tc_wait_ld(float (&r)[32]) {
#define X(i) "+f"(r[i])
    asm volatile("tcgen05.wait::ld.sync.aligned;" : QG_R32(X) : : "memory");
#undef X
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const float (&r)[32]) {
#define X(i) "f"(r[i])
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " QG_LIST32 ";" ::QG_R32(X), "r"(addr) : "memory");
#undef X
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
    const int n = live ? 16 : 0;  // 0 source bytes: filled with zeros, src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

struct TilesShared {
    unsigned long long q_full, k_full[2], v_full[2], k_empty[2], v_empty[2], s_full[2], p_full[2], o_full[2], drain;
    long long k_off[2][TK], v_off[2][TK];
    uint32_t live[4][TK / 32];
    uint32_t tmem;
    int failed;
};

template <int DP, bool BF>
__global__ void __launch_bounds__(TILE_THREADS, 1) attn_tiles_kernel(const AttnArgs a) {
    using S = TilesShape<DP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ TilesShared sh;
    pdl_launch_dependents();
    pdl_wait();
    Tile t;
    if (!find_tile<2 * TR, true>(a, blockIdx.x, &t)) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int blocks = (t.k1 - t.k0 + TK - 1) / TK;
    const int tiles = t.rows > TR ? 2 : 1;

    if (threadIdx.x == 0) {
        sh.failed = 0;
        mbar_init(smem_addr(&sh.q_full), 128);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.k_full[i]), 128);
            mbar_init(smem_addr(&sh.v_full[i]), 128);
            mbar_init(smem_addr(&sh.k_empty[i]), 1);
            mbar_init(smem_addr(&sh.v_empty[i]), 1);
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.p_full[i]), 128);
            mbar_init(smem_addr(&sh.o_full[i]), 1);
        }
        mbar_init(smem_addr(&sh.drain), 1);
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int* failed = &sh.failed;
    // A bounded wait; one that runs out (it cannot in a correct run) ends every role.
    auto wait = [&](unsigned long long& bar, int parity) {
        if (mbar_wait_bounded(smem_addr(&bar), static_cast<uint32_t>(parity))) return !*failed;
        *failed = 1;
        atomicOr(a.err, ERR_WAIT_TIMEOUT);
        return false;
    };

    if (warp >= LOAD_WARP && warp < MMA_WARP) {
        // ---- four warps copy Q once, then the key tiles
        const int lt = threadIdx.x - LOAD_WARP * 32, lw = lt / 32;
        constexpr int PER_ROW = DP / 8, ROWS_PASS = 128 / PER_ROW;  // 16-byte pieces of a row; rows of a pass of 128 threads
        const int c = lt % PER_ROW, r_in = lt / PER_ROW;
        const bool col = c * 8 < a.dim;
        auto place = [&](uint32_t base, int r) {
            return base + (c / 8) * S::HALF_BYTES + r * 128 + (((c % 8) ^ (r & 7)) << 4);
        };
        bool ok = true;
        // The barrier counts this thread's arrival when its copies so far have landed; the thread itself goes on.
        auto arrive_when_landed = [&](unsigned long long& bar) {
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&bar)) : "memory");
        };
        const int* table = a.pages + t.seq * a.pages_stride;
        // The page of this thread's key of block j, read one block ahead; -1 past the end.
        auto page_of = [&](int j) {
            const int key = t.k0 + j * TK + lt;
            return key < t.k1 ? table[key / a.page_size] : -1;
        };
        int page = page_of(0);
        if (blocks > 0) {
            const uint16_t* q = static_cast<const uint16_t*>(a.q);
            for (int r0 = 0; r0 < tiles * TR; r0 += ROWS_PASS) {
                const int r = r0 + r_in;
                const bool in = r < t.rows && col;
                const long long off = in ? out_at(a, t, r, a.q_token, a.q_head) + c * 8 : 0;
                cp16(place(smem + S::Q_AT + (r / TR) * S::TILE_BYTES, r % TR), q + off, in);
            }
            arrive_when_landed(sh.q_full);
        }
        for (int j = 0; j < blocks && ok; ++j) {
            const int st = j & 1;
            {
                const int key = t.k0 + j * TK + lt, off = key % a.page_size;
                const bool live = page >= 0 && page < a.num_pages;
                if (!live && key < t.k1) atomicOr(a.err, ERR_BAD_INDEX);
                sh.k_off[st][lt] = live ? page * a.k_page + off * a.k_token + t.kv_head * a.k_head : -1;
                sh.v_off[st][lt] = live ? page * a.v_page + off * a.v_token + t.kv_head * a.v_head : -1;
                const unsigned mask = __ballot_sync(0xffffffffu, live);
                if (lane == 0) sh.live[j & 3][lw] = mask;
                page = page_of(j + 1);
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (j >= 2) ok = wait(sh.k_empty[st], (j / 2 - 1) & 1);
            if (!ok) break;
#pragma unroll 8
            for (int r = r_in; r < TK; r += ROWS_PASS) {
                const long long off = sh.k_off[st][r];
                const bool in = off >= 0 && col;
                cp16(place(smem + S::K_AT + st * S::TILE_BYTES, r), a.k + (in ? off + c * 8 : 0), in);
            }
            arrive_when_landed(sh.k_full[st]);
            if (j >= 2) ok = wait(sh.v_empty[st], (j / 2 - 1) & 1);
            if (!ok) break;
#pragma unroll 8
            for (int r = r_in; r < TK; r += ROWS_PASS) {
                const long long off = sh.v_off[st][r];
                const bool in = off >= 0 && col;
                cp16(place(smem + S::V_AT + st * S::TILE_BYTES, r), a.v + (in ? off + c * 8 : 0), in);
            }
            arrive_when_landed(sh.v_full[st]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == MMA_WARP) {
        // ---- one thread issues every product
        if (lane == 0 && blocks > 0) {
            constexpr uint32_t qk = tc_idesc<BF>(TK, false), pv = tc_idesc<BF>(DP, true);
            auto scores = [&](int i, int st) {
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    const uint32_t off = (kk / 4) * S::HALF_BYTES + (kk % 4) * 32;
                    tc_mma_ss(tmem + S::S_COL + i * TK, tc_desc(smem + S::Q_AT + i * S::TILE_BYTES + off, 16, 1024),
                              tc_desc(smem + S::K_AT + st * S::TILE_BYTES + off, 16, 1024), qk, kk > 0);
                }
                tc_commit(smem_addr(&sh.s_full[i]));
            };
            // the copies were made through the generic proxy, the tensor cores read through the asynchronous one
            auto landed = [&](unsigned long long& bar, int parity) {
                const bool ok = wait(bar, parity);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                return ok;
            };
            bool ok = landed(sh.q_full, 0) && landed(sh.k_full[0], 0);
            if (ok) {
                tc_fence_after();
                for (int i = 0; i < tiles; ++i) scores(i, 0);
                tc_commit(smem_addr(&sh.k_empty[0]));
            }
            for (int j = 0; j < blocks && ok; ++j) {
                const int st = j & 1;
                for (int i = 0; i < tiles; ++i) {
                    ok = wait(sh.p_full[i], j & 1);
                    if (ok && i == 0) ok = landed(sh.v_full[st], (j / 2) & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < TK / 16; ++kk)
                        tc_mma_ts(tmem + S::O_COL + i * DP, tmem + S::S_COL + i * TK + TK / 2 + kk * 8,
                                  tc_desc(smem + S::V_AT + st * S::TILE_BYTES + kk * 2048, S::HALF_BYTES, 1024), pv, j > 0 || kk > 0);
                    if (i == tiles - 1) tc_commit(smem_addr(&sh.v_empty[st]));
                    if (j + 1 < blocks) {
                        if (i == 0) {
                            ok = landed(sh.k_full[st ^ 1], ((j + 1) / 2) & 1);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        scores(i, st ^ 1);
                        if (i == tiles - 1) tc_commit(smem_addr(&sh.k_empty[st ^ 1]));
                    } else {
                        tc_commit(smem_addr(&sh.o_full[i]));
                    }
                }
            }
            // nothing is left in flight when the block ends
            tc_commit(smem_addr(&sh.drain));
            (void)mbar_wait_bounded(smem_addr(&sh.drain), 0);
        }
        __syncwarp();
    } else if (warp / 4 < tiles) {
        // ---- softmax: one thread a row
        const int i = warp / 4, r = i * TR + threadIdx.x % TR;  // row of the pair of tiles
        const uint32_t lanes = static_cast<uint32_t>(warp % 4) << 21;  // 32 lanes a warp, in the upper half of the address
        const uint32_t s_at = tmem + lanes + S::S_COL + i * TK, o_at = tmem + lanes + S::O_COL + i * DP;
        const int last = min(t.rows, (i + 1) * TR) - 1;  // last row of this tile
        const int pos = row_pos(a, t, r);
        const int hi = a.causal ? min(t.k1 - 1, pos) : t.k1 - 1, lo = a.window > 0 ? pos - a.window + 1 : 0;
        // keys that all rows of the tile see
        const int all_hi = a.causal ? min(t.k1 - 1, row_pos(a, t, i * TR)) : t.k1 - 1;
        const int all_lo = a.window > 0 ? row_pos(a, t, last) - a.window + 1 : 0;
        float m = NEG_INF, l = 0.f;  // m: the maximum in use, in units of the scaled scores (base 2)
        bool ok = true;
        for (int j = 0; j < blocks; ++j) {
            ok = wait(sh.s_full[i], j & 1);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int key0 = t.k0 + j * TK;
            const uint32_t* live = sh.live[j & 3];
            const bool mask = key0 + TK - 1 > all_hi || key0 < all_lo || (live[0] & live[1] & live[2] & live[3]) != 0xffffffffu;
            float s0[32], s1[32];
            float tops[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};  // four chains
            auto hide = [&](float (&s)[32], int q) {  // the keys that this row does not see
                if (!mask) return;
                const uint32_t lv = live[q];
                const int k = key0 + q * 32;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (!(lv >> e & 1u) || k + e > hi || k + e < lo) s[e] = NEG_INF;
            };
            auto largest = [&](const float (&s)[32]) {
#pragma unroll
                for (int e = 0; e < 32; ++e) tops[e & 3] = fmaxf(tops[e & 3], s[e]);
            };
            tc_ld32(s0, s_at), tc_ld32(s1, s_at + 32);
            tc_wait_ld(s0), tc_wait_ld(s1);
            hide(s0, 0), hide(s1, 1);
            largest(s0), largest(s1);
            tc_ld32(s0, s_at + 64), tc_ld32(s1, s_at + 96);
            tc_wait_ld(s0), tc_wait_ld(s1);
            hide(s0, 2), hide(s1, 3);
            largest(s0), largest(s1);
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * a.scale_log2;
            // move the maximum only when it has to: by more than 2^8
            const bool move = top > m + 8.f;
            if (__any_sync(0xffffffffu, move)) {
                const float f = move ? exp2_approx(m - top) : 1.f;  // 0 for the first keys that the row sees
                if (move) m = top;
                l *= f;
                if (j > 0) {
                    // S_j is there, so the product before it, into O, has ended
                    float o[32];
#pragma unroll 1
                    for (int d = 0; d < DP; d += 32) {
                        tc_ld32(o, o_at + d);
                        tc_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tc_st32(o_at + d, o);
                    }
                }
            }
            const float base = m == NEG_INF ? 0.f : m;
            auto weigh = [&](float (&s)[32], uint32_t to) {
                uint32_t p[16];
                float sum[4] = {};
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float x = exp2_approx(fmaf(s[e], a.scale_log2, -base)), y = exp2_approx(fmaf(s[e + 1], a.scale_log2, -base));
                    sum[e & 2] += x, sum[(e & 2) + 1] += y;
                    p[e / 2] = pack16<BF>(x, y);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tc_st16(to, p);
            };
            // keys 64..127 first: their scores are in registers, and P goes where those were
            weigh(s0, s_at + 96), weigh(s1, s_at + 112);
            tc_ld32(s0, s_at), tc_ld32(s1, s_at + 32);
            tc_wait_ld(s0), tc_wait_ld(s1);
            hide(s0, 0), hide(s1, 1);
            weigh(s0, s_at + 64), weigh(s1, s_at + 80);
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(smem_addr(&sh.p_full[i]));
        }
        if (ok && blocks > 0) ok = __all_sync(0xffffffffu, wait(sh.o_full[i], 0));
        if (ok) {
            tc_fence_after();
            const bool whole = t.parts == 1, row = r < t.rows;
            const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
            const long long at = row ? out_at(a, t, r, a.out_token, a.out_head) : 0;
            float* rec = row && !whole ? part_row(a, t, t.part, r) : nullptr;
#pragma unroll 1
            for (int d = 0; d < DP; d += 32) {
                float o[32];
                __syncwarp();
                if (blocks > 0) {
                    tc_ld32(o, o_at + d);
                    tc_wait_ld(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (row && whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        if (d + e < a.dim)
                            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at + d + e) =
                                make_uint4(pack16<BF>(o[e] * inv, o[e + 1] * inv), pack16<BF>(o[e + 2] * inv, o[e + 3] * inv),
                                           pack16<BF>(o[e + 4] * inv, o[e + 5] * inv), pack16<BF>(o[e + 6] * inv, o[e + 7] * inv));
                } else if (row) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        if (d + e < a.dim) __stcg(reinterpret_cast<float2*>(rec + 2 + d + e), make_float2(o[e], o[e + 1]));
                }
            }
            if (row && whole) put_lse(a, t, r, m, l);
            if (row && !whole) __stcg(reinterpret_cast<float2*>(rec), make_float2(m, l));
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    if (t.parts > 1) join_parts<BF>(a, t);
}

template <int DP>
static const void* pick(bool bf16, unsigned* smem, unsigned* threads) {
    *smem = TilesShape<DP>::SMEM;
    *threads = TILE_THREADS;
    return bf16 ? (const void*)attn_tiles_kernel<DP, true> : (const void*)attn_tiles_kernel<DP, false>;
}

const void* attn_tiles_kernel_ptr(bool bf16, int dim, unsigned* smem, unsigned* threads) {
    return dim <= 64 ? pick<64>(bf16, smem, threads) : pick<128>(bf16, smem, threads);
}

}  // namespace qg
