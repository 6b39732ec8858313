// Attention of many rows (chunks of a prompt, whole prompts) over a paged cache on the fifth-generation tensor cores: two
// tiles of 128 rows a block against tiles of 128 keys.
//
// For each key tile j and row tile i: S_i = Q_i K_j^T into tensor memory (fp32), softmax by two threads a row, P_i (16 bits)
// back into S_i's columns, O_i += P_i V_j with P_i read from tensor memory.  While the tensor cores work
// on one row tile, the other's softmax runs.  The running maximum that the exponent is taken against moves only when the
// true one has grown by more than 2^8: then O_i and l are rescaled; p stays below 2^8, so nothing is lost by the delay.
// The keys of a tile lie on pages anywhere: two warps look the rows up, one for K and one for V.  A key tile whose keys are all there
// comes by tensor-map copies, one a page (or 128 tokens) and 64 columns, one with gaps 16 bytes at a time, both in the
// 128-byte-swizzled layout that the tensor cores read (K as the K-major, V as the MN-major operand: no transpose is made).
//
// Work a pair of row tiles and a key tile at D = 128: 2048 cycles of the tensor cores, 1024 of the exponential units; measured about 2720, the
// time of one row tile's round: softmax 1200, its products 1024, some 500 of barriers and of the products' latency.  The scores of the
// next keys wait for P V, because P lies in their columns; two row tiles' scores and sums (2 x (128 + 128) columns) are all of tensor
// memory, so that no third round hides the wait.  A chunk of 2000 tokens over 24000 (32 and 8 heads): 531 to 539 us over four GPUs,
// 1.40 to 1.42 PFLOP/s; two prompts of 6000: 384 to 387 us, 1.37 PFLOP/s (cuBLAS bf16: 1.72 sustained).
// What the steps gave, for the chunk: 1302 us with one softmax thread a row, row-by-row copies and a wait for each of them; 1062 with
// copies that announce themselves; 777 with tensor-map copies, two threads a row and exponentials ahead of the maximum; 694 with a
// warp that waits in the issuing warp's place; 612 with parts by cost and a kernel that joins them; 580 with blocks that stay (prompts:
// 435 to 397): the next part's keys and queries come under the end of the last one, and the warps' numbers and loop bounds are
// uniform for the compiler, which took 400 to 180 cycles from a probability's arrival to its product; 541 with the parts' records and
// launch in their cost.  Stores of 32 bytes (a whole sector) a thread in place of 16: prompts 429 to 420, chunks in parts 76 to 74.  Key
// tiles with gaps (a row tile's last keys, a window's first) copied with one shuffle a row in place of two rows' pages and tokens: prompts of
// 6001 and 4000 tokens 314 to 305, 2000 tokens over 24000 with a window of 1024 76 to 65.
#include "attn.cuh"

namespace qg {

constexpr int TR = 128;          // rows of a row tile
constexpr int TK = 128;          // keys of a key tile
// Warps 0..15: softmax, two groups of four a row tile; 16, 17: copies of keys and of values; 18: products; 19: waits for the
// copies in its place (a wait costs the issuing warp some 250 cycles, even for what is there).  With at most five warps a quarter of
// the SM a thread has 96 registers, enough for its 64 scores (spills would go past the small L1 that is left).
constexpr int K_WARP = 16, V_WARP = 17, MMA_WARP = 18, GATE_WARP = 19;
constexpr int TILE_THREADS = 20 * 32;

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
// The products and commits are issued by the one lane with `one` set, in code that the whole warp runs: control flow,
// descriptors and addresses then stay uniform over the warp.
__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(one)
        : "memory");
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
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}

// Two fp32 operations in one instruction, and the largest of three.
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float m, float c) {
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmov.b64 r, {%5, %5};\n\t"
        "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}" : "=f"(x), "=f"(y) : "f"(a), "f"(b), "f"(m), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tadd.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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
#define QG_R16(X) X(0), X(1), X(2), X(3), X(4), X(5), X(6), X(7), X(8), X(9), X(10), X(11), X(12), X(13), X(14), X(15)
#define QG_LIST16 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}"
__device__ __forceinline__ void tc_ld16(float (&r)[16], uint32_t addr) {
#define X(i) "=f"(r[i])
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 " QG_LIST16 ", [%16];" : QG_R16(X) : "r"(addr) : "memory");
#undef X
}
__device__ __forceinline__ void tc_wait_ld(float (&r)[16]) {
#define X(i) "+f"(r[i])
    asm volatile("tcgen05.wait::ld.sync.aligned;" : QG_R16(X) : : "memory");
#undef X
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const float (&r)[16]) {
#define X(i) "f"(r[i])
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], " QG_LIST16 ";" ::QG_R16(X), "r"(addr) : "memory");
#undef X
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
#define X(i) "r"(r[i])
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " QG_LIST32 ";" ::QG_R32(X), "r"(addr) : "memory");
#undef X
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
    const int n = live ? 16 : 0;  // 0 source bytes: filled with zeros, src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Copies `box` tokens of one page, 64 elements of one head, into swizzled rows; completion is counted on the barrier.
__device__ __forceinline__ void tma_box(uint32_t dst, const unsigned long long* map, int x, int token, int page, int head,
                                        uint32_t bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(dst),
        "l"(map), "r"(x), "r"(token), "r"(page), "r"(head), "r"(bar), "r"(one)
        : "memory");
}
// 32 bytes, a whole sector, at once.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}
__device__ __forceinline__ uint32_t elect() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}

constexpr int ITEMS = 4;

struct TilesShared {
    unsigned long long item_full[ITEMS], item_empty[ITEMS], q_full, q_empty, k_full[2], v_full[2], k_empty[2], v_empty[2], s_full[2],
        p_full[2], o_full[2], o_empty[2], drain;
    Tile item[ITEMS];           // the parts that the block works on, in a ring; seq -1: no more
    uint32_t live[4][TK / 32];  // which keys of a key tile are there, one bit each
    float top[2][2][TR], sum[2][2][TR];  // by row tile and half of the keys: a row's maximum, at a part's end its sum
    uint32_t tmem;  // the allocation's answer, always column 0 (all 512 are asked for)
};

// The row tiles with the most keys (the last ones, under a causal mask) of all sequences and heads come first, so that the grid ends
// with short ones.  False: nothing to do (past the sequence's rows or the tile's parts).
__device__ __forceinline__ bool find_tile(const AttnArgs& a, long long block, Tile* t) {
    const int pairs = a.kv_heads * a.seqs;
    const long long of_parts = block - a.whole;
    t->part = of_parts < 0 ? 0 : static_cast<int>(of_parts % a.parts);
    t->index = of_parts < 0 ? block : a.whole + of_parts / a.parts;
    const int pair = static_cast<int>(t->index % pairs), rt = static_cast<int>(a.row_tiles - 1 - t->index / pairs);
    t->kv_head = pair % a.kv_heads;
    t->seq = pair / a.kv_heads;
    const Seq s = find_seq(a, t->seq);
    t->q0 = s.q0, t->first_pos = s.first_pos;
    t->row0 = rt * 2 * TR;
    t->rows = min(2 * TR, s.n * a.group - t->row0);
    if (t->rows <= 0) return false;
    int lo, hi;
    t->first = find_keys(a, s, t->row0, t->rows, TK, &lo, &hi);  // key tiles start at multiples of their size
    const int chunk = of_parts < 0 ? max(hi - lo, 1) : a.chunk;
    t->parts = max(1, (hi - lo + chunk - 1) / chunk);
    t->k0 = lo + t->part * chunk;
    t->k1 = min(hi, t->k0 + chunk);
    return t->part < t->parts;
}
__device__ __forceinline__ long long part_at(const AttnArgs& a, const Tile& t, int part, int r) {
    return ((t.index - a.whole) * a.parts + part) * a.rows_part + r;
}

// A block takes parts of row tiles one after the other, the next one's number from a counter (the first from its own), until there
// are no more; each role goes on to the next as soon as its own work on this one is done, so that the next one's keys and queries are on
// their way while the last rows are written.  What a part computes does not depend on who takes it.
template <int DP, bool BF>
__global__ void __launch_bounds__(TILE_THREADS, 1) attn_tiles_kernel(const __grid_constant__ AttnTileArgs ta) {
    using S = TilesShape<DP>;
    const AttnArgs& a = ta.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ TilesShared sh;
    pdl_launch_dependents();
    pdl_wait();
    // A value that all lanes have, in a form that is uniform for the compiler too: control flow, addresses and descriptors that hang on it
    // then are, and take no registers of the threads.
    auto uniform = [](int v) { return __reduce_max_sync(0xffffffffu, v); };
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    constexpr int PER_ROW = DP / 8;  // 16-byte pieces of a row

    const unsigned all = a.whole + static_cast<unsigned>(a.parts) * (a.row_tiles * (a.kv_heads * a.seqs) - a.whole);
    // The n-th part that this block takes, the first from its own number.
    auto next_part = [&](unsigned n) {
        Tile* t = &sh.item[n % ITEMS];
        unsigned at = n == 0 ? blockIdx.x : gridDim.x + atomicAdd(a.count, 1u);
#pragma unroll 1
        while (at < all && !find_tile(a, at, t)) at = gridDim.x + atomicAdd(a.count, 1u);
        if (at >= all) t->seq = -1;
    };
    if (threadIdx.x == K_WARP * 32) next_part(0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(smem_addr(&sh.item_full[i]), 1);
            mbar_init(smem_addr(&sh.item_empty[i]), TILE_THREADS / 32 - 1);  // a warp each but K_WARP, which fills it
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.k_full[i]), 32);
            mbar_init(smem_addr(&sh.v_full[i]), 32);
            mbar_init(smem_addr(&sh.k_empty[i]), 1);
            mbar_init(smem_addr(&sh.v_empty[i]), 1);
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.p_full[i]), i == 0 ? 9 : 8);  // a softmax warp each, and the gate
            mbar_init(smem_addr(&sh.o_full[i]), 1);
            mbar_init(smem_addr(&sh.o_empty[i]), 8);
        }
        mbar_init(smem_addr(&sh.q_full), a.q_map ? 2 : 512);  // K_WARP and V_WARP, else the softmax threads
        mbar_init(smem_addr(&sh.q_empty), 1);
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
    constexpr uint32_t tmem = 0;  // all 512 columns are this block's, so they start at column 0
    // A bounded wait; where one runs out (it cannot in a correct run) the role ends, and those that wait for it likewise.
    auto wait = [&](unsigned long long& bar, unsigned round) {
        if (mbar_wait_bounded(smem_addr(&bar), round & 1u)) return true;
        atomicOr(a.err, ERR_WAIT_TIMEOUT);
        return false;
    };
    auto await = [&](unsigned long long& bar, unsigned round) { return __all_sync(0xffffffffu, wait(bar, round)) != 0; };
    // The n-th part that this block takes, good until done(n); false: no more (or a wait ran out).
    auto take = [&](unsigned n) {
        if (n > 0 && !await(sh.item_full[n % ITEMS], n / ITEMS - (n % ITEMS == 0))) return false;
        return uniform(sh.item[n % ITEMS].seq) >= 0;
    };
    auto done = [&](unsigned n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.item_empty[n % ITEMS]));
    };
    auto blocks_of = [&](const Tile& t) { return max(0, uniform(t.k1 - t.k0) + TK - 1) / TK; };
    auto tiles_of = [&](const Tile& t) { return uniform(t.rows) > TR ? 2 : 1; };
    // 16-byte piece c of row r in a tile's swizzled layout
    auto place = [&](uint32_t base, int r, int c) {
        return base + (c / 8) * S::HALF_BYTES + r * 128 + (((c % 8) ^ (r & 7)) << 4);
    };

    // 512 x 104 + 128 x 64 registers: the launch's 640 x 96.  The softmax then keeps its scores without spills in its loop.
    if (warp >= K_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == K_WARP || warp == V_WARP) {
            // ---- copies of the key tiles, one warp for each side; and of the queries, a row tile each
            const bool side = warp == V_WARP;
            const uint32_t one = elect();
            unsigned long long* const full = side ? sh.v_full : sh.k_full;
            unsigned long long* const empty = side ? sh.v_empty : sh.k_empty;
            const long long page_stride = side ? a.v_page : a.k_page, token_stride = side ? a.v_token : a.k_token;
            const unsigned long long* const map = side ? ta.v_map : ta.k_map;
            unsigned g = 0, queries = 0;  // key tiles so far, parts with keys so far
            bool ok = true;
            // The keys' warp also fetches the parts' numbers, in a wait of its own.
            auto publish = [&](unsigned n) {
                if (n >= ITEMS && !await(sh.item_empty[n % ITEMS], n / ITEMS - 1)) return false;
                if (lane == 0) {
                    next_part(n);
                    mbar_arrive(smem_addr(&sh.item_full[n % ITEMS]));
                }
                __syncwarp();
                return true;
            };
            for (unsigned n = 0; ok && (side ? take(n) : uniform(sh.item[n % ITEMS].seq) >= 0); ++n) {
                const Tile& t = sh.item[n % ITEMS];
                const int blocks = blocks_of(t);
                if (blocks == 0) {
                    if (side) done(n);
                    else ok = publish(n + 1);
                    continue;
                }
                const uint16_t* const src = (side ? a.v : a.k) + t.kv_head * (side ? a.v_head : a.k_head);
                const int* const table = a.pages + t.seq * a.pages_stride;
                // Page and token of this lane's four keys (lane, lane + 32, ..) of block j, read one block ahead; page -1: no such key.
                int page[4], token[4];
                auto look_up = [&](int j) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int key = t.k0 + j * TK + h * 32 + lane, nth = div_by(key, a.page_size, a.page_shift);
                        token[h] = key - nth * a.page_size;
                        page[h] = key >= t.first && key < t.k1 ? table[nth] : -1;
                    }
                };
                auto of_row = [&](const int (&v)[4], int row) {
                    return __shfl_sync(0xffffffffu, row < 64 ? (row < 32 ? v[0] : v[1]) : (row < 96 ? v[2] : v[3]), row & 31);
                };
                look_up(0);
                for (int j = 0; j < blocks; ++j) {
                    const unsigned st = g & 1;
                    uint32_t all = 0xffffffffu;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const bool live = page[h] >= 0 && page[h] < a.num_pages;
                        const int key = t.k0 + j * TK + h * 32 + lane;
                        if (!live && !side && key >= t.first && key < t.k1) atomicOr(a.err, ERR_BAD_INDEX);
                        if (!live) page[h] = -1;
                        const uint32_t mask = __ballot_sync(0xffffffffu, live);
                        if (!side && lane == 0) sh.live[g & 3][h] = mask;
                        all &= mask;
                    }
                    if (g >= 2 && !(ok = await(empty[st], g / 2 - 1))) break;
                    const uint32_t to = smem + (side ? S::V_AT : S::K_AT) + st * S::TILE_BYTES, bar = smem_addr(&full[st]);
                    if (a.box && all == 0xffffffffu) {  // every key is there: one tensor-map copy a box of tokens and 64 columns
                        if (lane == 0) mbar_arrive_expect_tx(bar, S::TILE_BYTES);
                        else mbar_arrive(bar);
                        for (int row = 0; row < TK; row += a.box) {
                            const int tk = of_row(token, row), pg = of_row(page, row);
#pragma unroll
                            for (int h = 0; h < S::HALVES; ++h)
                                tma_box(to + h * S::HALF_BYTES + row * 128, map, h * 64, tk, pg, t.kv_head, bar, one);
                        }
                    } else {  // row by row, the missing ones as zeros
                        const int c = lane % PER_ROW;
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            // where this lane's key lies; its row's lanes ask for it
                            const long long at = page[h] < 0 ? -1 : page[h] * page_stride + token[h] * token_stride;
#pragma unroll 4
                            for (int r0 = 0; r0 < 32; r0 += 32 / PER_ROW) {
                                const long long off = __shfl_sync(0xffffffffu, at, r0 + lane / PER_ROW);
                                const bool in = off >= 0 && c * 8 < a.dim;
                                cp16(place(to, h * 32 + r0 + lane / PER_ROW, c), src + (in ? off + c * 8 : 0), in);
                            }
                        }
                        // the barrier counts this lane's arrival when its copies have landed; the lane itself goes on
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
                    }
                    ++g;
                    if (j == 0 && a.q_map) {  // this part's queries, a row tile each
                        if (queries > 0 && !(ok = await(sh.q_empty, queries - 1))) break;
                        const bool there = !side || tiles_of(t) > 1;
                        if (lane == 0) {
                            if (there) mbar_arrive_expect_tx(smem_addr(&sh.q_full), S::TILE_BYTES);
                            else mbar_arrive(smem_addr(&sh.q_full));
                        }
                        __syncwarp();
                        if (there) {
                            const int token = t.q0 + (t.row0 + (side ? TR : 0)) / a.group;
#pragma unroll
                            for (int h = 0; h < S::HALVES; ++h)
                                tma_box(smem + S::Q_AT + (side ? S::TILE_BYTES : 0) + h * S::HALF_BYTES, ta.q_map, h * 64,
                                        t.kv_head * a.group, token, 0, smem_addr(&sh.q_full), one);
                        }
                    }
                    if (!side && j == min(1, blocks - 1) && !(ok = publish(n + 1))) break;
                    look_up(j + 1);
                }
                if (side) done(n);
                ++queries;
            }
            // the last block to come here puts the counters back to zero: every block has taken its last number then
            if (!side && lane == 0) {
                __threadfence();
                if (atomicAdd(a.count + 1, 1u) == gridDim.x - 1) {
                    __threadfence();
                    a.count[0] = 0, a.count[1] = 0;
                }
            }
            // nothing of its own is in flight when it ends
            for (unsigned back = min(g, 2u); back > 0; --back) (void)mbar_wait_bounded(smem_addr(&full[(g - back) & 1]), (g - back) / 2 & 1);
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == MMA_WARP) {
            // ---- one thread issues every product
            const uint32_t one = elect();
            constexpr uint32_t qk = tc_idesc<BF>(TK, false), pv = tc_idesc<BF>(DP, true);
            const uint64_t q_desc = tc_desc(smem + S::Q_AT, 16, 1024), k_desc = tc_desc(smem + S::K_AT, 16, 1024),
                           v_desc = tc_desc(smem + S::V_AT, S::HALF_BYTES, 1024);
            auto scores = [&](int i, unsigned st) {
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    const uint32_t off = (kk / 4) * S::HALF_BYTES + (kk % 4) * 32;  // descriptors count 16 bytes
                    tc_mma_ss(S::S_COL + i * TK, q_desc + ((i * S::TILE_BYTES + off) >> 4),
                              k_desc + ((st * S::TILE_BYTES + off) >> 4), qk, kk > 0, one);
                }
                tc_commit(smem_addr(&sh.s_full[i]), one);
            };
            // key tiles and parts so far; of the second row tile (every part has the first) likewise
            unsigned g = 0, queries = 0, g1 = 0, queries1 = 0;
            bool ok = true;
            for (unsigned n = 0; ok && take(n); done(n), ++n) {
                const Tile& t = sh.item[n % ITEMS];
                const int blocks = blocks_of(t), tiles = tiles_of(t);
                if (blocks == 0) continue;
                ok = await(sh.q_full, queries) && await(sh.k_full[g & 1], g / 2);
                if (!ok) break;
                // copies row by row came through the generic proxy, and the tensor cores read through the asynchronous one
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_after();
                for (int i = 0; i < tiles; ++i) scores(i, g & 1);
                tc_commit(smem_addr(&sh.k_empty[g & 1]), one);
                if (blocks == 1) tc_commit(smem_addr(&sh.q_empty), one);
                // the sums of the parts before have been read
                if (queries > 0) ok = await(sh.o_empty[0], queries - 1);
                if (queries1 > 0 && tiles > 1) ok = ok && await(sh.o_empty[1], queries1 - 1);
                for (int j = 0; j < blocks && ok; ++j, ++g) {
                    const unsigned st = g & 1;
#pragma unroll 1
                    for (int i = 0; i < tiles; ++i) {
                        ok = await(sh.p_full[i], i == 0 ? g : g1);  // for the first row tile also: V_j and K_j+1 are there
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < TK / 16; ++kk)
                            tc_mma_ts(S::O_COL + i * DP, S::S_COL + i * TK + kk / 4 * 64 + kk % 4 * 8,
                                      v_desc + ((st * S::TILE_BYTES + kk * 2048) >> 4), pv, j > 0 || kk > 0, one);
                        if (i == tiles - 1) tc_commit(smem_addr(&sh.v_empty[st]), one);
                        if (j + 1 < blocks) {
                            scores(i, st ^ 1);
                            if (i == tiles - 1) {
                                tc_commit(smem_addr(&sh.k_empty[st ^ 1]), one);
                                if (j + 2 == blocks) tc_commit(smem_addr(&sh.q_empty), one);
                            }
                        } else {
                            tc_commit(smem_addr(&sh.o_full[i]), one);
                        }
                    }
                    g1 += tiles - 1;
                }
                ++queries, queries1 += tiles - 1;
            }
            // nothing is left in flight when the block ends
            tc_commit(smem_addr(&sh.drain), one);
            (void)mbar_wait_bounded(smem_addr(&sh.drain), 0);
            __syncwarp();
        } else if (warp == GATE_WARP) {
            // ---- the waits for the copies.  Rows that were copied one by one were written through the generic proxy, and the products read
            // through the asynchronous one: the fence between them lies on the path from the copies' arrival, which every lane here has
            // waited for, to lane 0's arrival, which the issuing thread waits for.  (The copying lanes do not wait for their copies.)
            auto landed = [&](unsigned long long& bar, unsigned g) {
                if (!await(bar, g / 2)) return false;
                const uint32_t* lv = sh.live[g & 3];
                if (!a.box || (lv[0] & lv[1] & lv[2] & lv[3]) != 0xffffffffu) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                return true;
            };
            unsigned g = 0;
            bool ok = true;
            for (unsigned n = 0; ok && take(n); done(n), ++n) {
                const int blocks = blocks_of(sh.item[n % ITEMS]);
                for (int j = 0; j < blocks && ok; ++j, ++g) {
                    // (not before S_j is there: the barrier's round for the block before has ended then)
                    ok = await(sh.s_full[0], g) && landed(sh.v_full[g & 1], g) && (j + 1 == blocks || landed(sh.k_full[(g + 1) & 1], g + 1));
                    if (ok && lane == 0) mbar_arrive(smem_addr(&sh.p_full[0]));
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        // ---- softmax: two threads a row, one for each half of the keys
        const int i = warp / 8, half = warp / 4 % 2, tr = threadIdx.x % TR, r = i * TR + tr;  // r: row of the two tiles
        const uint32_t lanes = static_cast<uint32_t>(warp % 4) << 21;  // 32 lanes a warp, in the upper half of the address
        const uint32_t o_at = tmem + lanes + S::O_COL + i * DP + half * (DP / 2);
        const uint32_t at = tmem + lanes + S::S_COL + i * TK + half * 64;  // this half's scores, and then its probabilities
        // the two warps of the same rows
        auto pair_sync = [&] { asm volatile("bar.sync %0, 64;" ::"r"(2 + i * 4 + warp % 4) : "memory"); };
        unsigned g = 0, queries = 0, round = 0, outs = 0;
        bool ok = true;
        for (unsigned n = 0; ok && take(n); done(n), ++n) {
            const Tile& t = sh.item[n % ITEMS];
            const int blocks = blocks_of(t);
            if (blocks > 0 && !a.q_map) {  // the queries, one row after the other
                if (queries > 0 && !(ok = await(sh.q_empty, queries - 1))) break;
                if (i < tiles_of(t)) {
                    const uint16_t* q = static_cast<const uint16_t*>(a.q);
                    const int c = threadIdx.x % PER_ROW;
#pragma unroll 4
                    for (int qr = threadIdx.x % 256 / PER_ROW; qr < TR; qr += 256 / PER_ROW) {
                        const bool in = i * TR + qr < t.rows && c * 8 < a.dim;
                        const long long off = in ? out_at(a, t, i * TR + qr, a.q_token, a.q_head) + c * 8 : 0;
                        cp16(place(smem + S::Q_AT + i * S::TILE_BYTES, qr, c), q + off, in);
                    }
                }
                asm volatile("cp.async.wait_all;\n\tfence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(smem_addr(&sh.q_full));
                ++queries;
            }
            if (i >= tiles_of(t)) {
                g += blocks;
                continue;
            }
            const int pos = row_pos(a, t, r);
            const int hi = a.causal ? min(t.k1 - 1, pos) : t.k1 - 1, lo = first_key(a, pos);
            float m = NEG_INF, l = 0.f;  // m: the maximum in use (less the lift), in units of the scaled scores (base 2)
            for (int j = 0; j < blocks; ++j, ++g) {
                if (!(ok = await(sh.s_full[i], round++))) break;
                tc_fence_after();
                const int key0 = t.k0 + j * TK + half * 64;
                const uint32_t* live = sh.live[g & 3] + half * 2;
                const bool mask = __any_sync(0xffffffffu, key0 + 63 > hi || key0 < lo) || (live[0] & live[1]) != 0xffffffffu;
                // 64 scores: p = 2^(s - base) in 16 bits; the sum of p and the maximum of s.
                uint32_t p[32];
                float top, sum;
                auto weigh = [&](float base) {
                    float s[2][32], tops[2] = {NEG_INF, NEG_INF}, sums[4] = {};
                    tc_ld32(s[0], at), tc_ld32(s[1], at + 32);
                    tc_wait_ld(s[0]), tc_wait_ld(s[1]);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float (&c)[32] = s[q];
                        if (mask) {  // the keys that this row does not see
                            const uint32_t lv = live[q];
                            const int k = key0 + q * 32;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(lv >> e & 1u) || k + e > hi || k + e < lo) c[e] = NEG_INF;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            tops[e / 2 & 1] = max3(tops[e / 2 & 1], c[e], c[e + 1]);
                            float x, y;
                            fma2(x, y, c[e], c[e + 1], a.scale_log2, -base);
                            x = exp2_approx(x), y = exp2_approx(y);
                            add2(sums[e & 2], sums[(e & 2) + 1], x, y);
                            p[q * 16 + e / 2] = pack16<BF>(x, y);
                        }
                    }
                    top = fmaxf(tops[0], tops[1]);
                    sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
                };
                // The exponentials are taken against the maximum in use while the new one is being found; only where that turns
                // out to be larger by more than 2^LAG (and for the first keys that a row sees) are they taken again.
                weigh(m == NEG_INF ? 0.f : m);
                sh.top[i][half][tr] = top;
                pair_sync();
                top = fmaxf(top, sh.top[i][half ^ 1][tr]) * a.scale_log2;
                const bool move = top > m + (Lift<BF>::TILES + Lift<BF>::LAG);
                if (__any_sync(0xffffffffu, move)) {
                    const float to = top - Lift<BF>::TILES, f = move ? exp2_approx(m - to) : 1.f;  // 0 for the first keys that the row sees
                    if (move) m = to;
                    l *= f;
                    if (j > 0) {
                        // S_j is there, so the product before it, into O, has ended
                        float o[16];
#pragma unroll 1
                        for (int d = 0; d < DP / 2; d += 16) {
                            tc_ld16(o, o_at + d);
                            tc_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f;
                            tc_st16(o_at + d, o);
                        }
                    }
                    weigh(m == NEG_INF ? 0.f : m);
                }
                l += sum;
                tc_st32(at, p);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[i]));  // (256 arrivals on one barrier would take their time)
            }
            if (!ok) break;
            if (blocks > 0) {
                if (!(ok = await(sh.o_full[i], outs++))) break;
                tc_fence_after();
                sh.sum[i][half][tr] = l;
                pair_sync();
                l += sh.sum[i][half ^ 1][tr];
            }
            const bool whole = t.parts == 1, row = r < t.rows;
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            const long long to = row ? out_at(a, t, r, a.out_token, a.out_head) + half * (DP / 2) : 0;
            float* rec = row && !whole ? a.part_sum + part_at(a, t, t.part, r) * a.dim + half * (DP / 2) : nullptr;
            const int dims = a.dim - half * (DP / 2);  // of this half
#pragma unroll 1
            for (int d = 0; d < DP / 2; d += 32) {
                float o[32];
                __syncwarp();
                if (blocks > 0) {
                    tc_ld32(o, o_at + d);
                    tc_wait_ld(o);
                    if (d + 32 >= DP / 2) {  // the last of them: the next part's sums may come
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&sh.o_empty[i]));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (row && whole) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = pack16<BF>(o[2 * e] * inv, o[2 * e + 1] * inv);
                    uint16_t* out = static_cast<uint16_t*>(a.out) + to + d;
                    if (a.wide) {
#pragma unroll
                        for (int e = 0; e < 16; e += 8)
                            if (d + 2 * e < dims)
                                store32(out + 2 * e, {w[e], w[e + 1], w[e + 2], w[e + 3], w[e + 4], w[e + 5], w[e + 6], w[e + 7]});
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            if (d + 2 * e < dims) *reinterpret_cast<uint4*>(out + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                    }
                } else if (row && a.wide) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        if (d + e < dims) store32(rec + d + e, reinterpret_cast<const uint32_t(&)[8]>(o[e]));
                } else if (row) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        if (d + e < dims) __stcg(reinterpret_cast<float4*>(rec + d + e), make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                }
            }
            if (row && half == 0) {
                if (whole) put_lse(a, t, r, m, l);
                else __stcg(a.part_stat + part_at(a, t, t.part, r), make_float2(m, l));
            }
        }
        // A warp whose wait ran out (it cannot in a correct run) may have a partner that got past the same wait and stands in pair_sync: it
        // leaves one arrival there.  The partner's next wait then runs out too, for want of this warp's arrivals.
        asm volatile("bar.arrive %0, 64;" ::"r"(2 + i * 4 + warp % 4) : "memory");
        tc_fence_before();
    }
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// Joins the parts of the rows of split tiles, one warp a row.
template <bool BF>
__global__ void __launch_bounds__(JOIN_WARPS * 32) attn_join_kernel(const AttnArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const long long w = static_cast<long long>(blockIdx.x) * JOIN_WARPS + threadIdx.x / 32;
    const long long index = w / a.rows_part;  // among the row tiles that are cut
    const int r = static_cast<int>(w % a.rows_part);
    if (index >= static_cast<long long>(a.row_tiles) * a.kv_heads * a.seqs - a.whole) return;
    Tile t;
    if (!find_tile(a, a.whole + index * a.parts, &t) || t.parts == 1 || r >= t.rows) return;
    join_row<BF>(a, t, r, [&](int p) { return part_at(a, t, p, r); });
}

template <int DP>
static const void* pick(bool bf16, unsigned* smem, unsigned* threads) {
    *smem = TilesShape<DP>::SMEM;
    *threads = TILE_THREADS;
    return bf16 ? (const void*)attn_tiles_kernel<DP, true> : (const void*)attn_tiles_kernel<DP, false>;
}

const void* attn_join_kernel_ptr(bool bf16) {
    return bf16 ? (const void*)attn_join_kernel<true> : (const void*)attn_join_kernel<false>;
}

const void* attn_tiles_kernel_ptr(bool bf16, int dim, unsigned* smem, unsigned* threads) {
    return dim <= 64 ? pick<64>(bf16, smem, threads) : pick<128>(bf16, smem, threads);
}

}  // namespace qg
