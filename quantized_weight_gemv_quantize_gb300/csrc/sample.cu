// Sampling from logits with temperature, top-k, top-p and min-p: one cluster of blocks a row.
//
// Weights are whole numbers, w = floor(2^42 exp((x - max) / T)): their sums are exact in 64 bits whatever the order, so
// the result is the same on every run and for every split of the work (and the blocks may sum with atomics).  Nothing is
// sorted.  With c = (key bits of x, reversed index) as one number, the tokens that top-k and top-p keep are those with
// c >= cut.
//  - Few tokens by top-k (up to one a thread): the k-th largest of the threads' own largest logits is a bound that at least k tokens reach, and few
//    more than k do.  Those are gathered and sorted: ranks, masses and the draw come from that list.
//  - Else a histogram of 1024 bins linear in (max - x) / T (counts for top-k, masses for top-p) tells the bin in which the count or the
//    mass reaches its bound.  Where the tokens up to that bin are surely few, the list is made of them.  Else the bin's tokens alone are
//    gathered and give the cut, and the draw takes one more pass over the row; a bin of more than CAP tokens is split again, by c, until
//    one has at most CAP (c differs for all tokens, so this ends even for a row of equal logits).
// Each block keeps its slice of the row in shared memory; the row is read once from global memory.  At 151936 logits: one row with top-k and
// top-p 12.2 us in a graph (15 to 17 call after call, with the caller's part): four cluster barriers and the passes between them one after
// the other (load 1.5 us, maximum 1.4, bound 2.8, gathering 1.8, list 5);
// 16 rows of mixed settings 39 us, set by the slowest, a top-k beyond the list and then top-p; 320 rows of bf16 logits, top-p alone, 215 to 221 us:
// 44 us of them the histogram's arithmetic (some 30 instructions a token, of which the exponential is 8), the rest barriers and lists
// that two blocks an SM do not hide (issue slots 53% busy).  One block a row with a radix sort's passes took 4108, 4816 and 7278 us.
#include "common.cuh"
#include "internal.h"
#include "step.h"

namespace qg {

using u64 = unsigned long long;

constexpr int ST = SAMPLE_THREADS, SW = ST / 32;  // threads and warps of a block
constexpr int CAP = ST;                           // tokens of a list: one a thread
constexpr int BINS = 1024, GROUP = 32;            // 32 groups of 32 bins: a warp's width each
constexpr int PER = BINS / ST;                    // bins of a thread

// ---- cluster: barrier, and the same shared-memory address in another block
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ uint32_t peer(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ u64 peer_ld64(uint32_t a) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void peer_st64(uint32_t a, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// Unsigned key that orders as x does (both zeros alike), and x from its key.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float x_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key); }
__device__ __forceinline__ u64 place_of(uint32_t key, int i) { return static_cast<u64>(key) << 20 | (0xFFFFFu - i); }
__device__ __forceinline__ float e_of(float x, float top, float rate) { return expf((x - top) * rate); }
// floor(2^42 e) for 0 <= e <= 1, from the bits of e: the 24-bit significand, as 2^42 for e = 1, shifted down by the exponent.
__device__ __forceinline__ u64 mass_of(float e) {
    const uint32_t b = __float_as_uint(e);
    const u64 one = static_cast<u64>((b & 0x7fffffu) | 0x800000u) << 19;
    u64 w;
    asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"(one), "r"(127u - (b >> 23)));  // (a shift of 64 or more gives 0)
    return w;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Monotone in x: 1024 bins over the 30 nats below the largest logit (2^-42 is 29.1), everything further in the last.
constexpr float BIN_RATE = BINS / 30.0f;
__device__ __forceinline__ int bin_of(float x, float top, float rate) {
    return min(BINS - 1, static_cast<int>((x - top) * rate * -BIN_RATE));  // (the first product is e_of's)
}

template <int XK>
struct Raw {
    using type = uint16_t;
};
template <>
struct Raw<ACT_F32> {
    using type = float;
};
template <int XK>
__device__ __forceinline__ float widen(typename Raw<XK>::type w) {
    if constexpr (XK == ACT_F32) return w;
    else if constexpr (XK == ACT_BF16) return __uint_as_float(static_cast<uint32_t>(w) << 16);
    else return h2f(w);
}
template <int XK>
__device__ __forceinline__ void widen_all(const uint4& w, float (&x)[16 / sizeof(typename Raw<XK>::type)]) {
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (XK == ACT_F32) x[j] = __uint_as_float(p[j]);
        else if constexpr (XK == ACT_BF16) x[2 * j] = __uint_as_float(p[j] << 16), x[2 * j + 1] = __uint_as_float(p[j] & 0xffff0000u);
        else x[2 * j] = h2f(p[j]), x[2 * j + 1] = h2f(p[j] >> 16);
    }
}

struct alignas(16) SampleShared {  // the slice follows it in shared memory, written 16 bytes at a time
    uint32_t lo[BINS], hi[BINS], count[BINS];  // masses as two words (hi takes the carries of lo), counts
    u64 list[ST];                             // c of the tokens of this block that were gathered
    u64 line[2 * ST];                          // two words a thread, for the lists
    u64 group_m[32], group_n[32];
    u64 found[2][5];                           // by level: which, count and mass before it, mass in it, the whole mass
    u64 got_m[2][8][32], got_n[2][8][32];      // masses and counts of groups of bins, and of a group's bins, from each block
    u64 push[2][2][8];                         // what the blocks tell each other, by kind and block; two sets in turn
    u64 red[3][ST / 32];
    unsigned used;
};
static_assert(sizeof(SampleShared) % 16 == 0, "");

template <class T, class Op>
__device__ __forceinline__ T warp_reduce(T v, Op op) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

template <int XK>
__global__ void __launch_bounds__(ST, 2) sample_kernel(const SampleArgs a) {
    using raw = typename Raw<XK>::type;
    constexpr int V = 16 / sizeof(raw);
    extern __shared__ __align__(16) uint8_t smem[];
    SampleShared& s = *reinterpret_cast<SampleShared*>(smem);
    uint4* const stage = reinterpret_cast<uint4*>(smem + sizeof(SampleShared));
    u64* const line = s.line;
    // Another block's shared memory may be written only once that block runs: every block says so here, and waits for the
    // others before the first exchange, when the slice's load has long covered it.
    if (a.blocks > 1) cluster_arrive();
    pdl_launch_dependents();
    pdl_wait();
    const int CS = a.blocks, rank = static_cast<int>(blockIdx.x) % CS, row = static_cast<int>(blockIdx.x) / CS;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, N = a.N;
    const int first = rank * a.slice, n = max(0, min(a.slice, N - first));  // this block's tokens
    const int vecs = (n + V - 1) / V;                                       // in 16-byte pieces, the last filled up with -inf
    const raw* const src = static_cast<const raw*>(a.x) + row * a.row_stride + first;
    const float NONE = __int_as_float(0xff800000);
    // A piece from global memory: whole where it can be read so.
    const bool wide = reinterpret_cast<uintptr_t>(src) % 16 == 0;
    auto from_global = [&](int i, float (&x)[V]) {
        if (wide && (i + 1) * V <= n) {
            widen_all<XK>(reinterpret_cast<const uint4*>(src)[i], x);
        } else {
#pragma unroll
            for (int q = 0; q < V; ++q) x[q] = i * V + q < n ? widen<XK>(src[i * V + q]) : NONE;
        }
    };
    auto piece = [&](int i, float (&x)[V]) {
        if (a.staged) widen_all<XK>(stage[i], x);
        else from_global(i, x);
    };
    auto token = [&](int i) {  // i < vecs * V
        if (a.staged) return widen<XK>(reinterpret_cast<const raw*>(stage)[i]);
        return i < n ? widen<XK>(src[i]) : NONE;
    };
    // Every piece of the slice, several at a time: f(x, i); every token: f(x, i).
    auto for_pieces = [&](auto&& f) {
        constexpr int U = V == 4 ? 4 : 2;
        int i = tid;
        for (; i + (U - 1) * ST < vecs; i += U * ST) {
            float x[U][V];
#pragma unroll
            for (int j = 0; j < U; ++j) piece(i + j * ST, x[j]);
#pragma unroll
            for (int j = 0; j < U; ++j) f(x[j], i + j * ST);
        }
        for (; i < vecs; i += ST) {
            float x[V];
            piece(i, x);
            f(x, i);
        }
    };
    auto for_all = [&](auto&& f) {
        for_pieces([&](const float (&x)[V], int i) {
#pragma unroll
            for (int q = 0; q < V; ++q) f(x[q], i * V + q);
        });
    };
    auto sync_all = [&] {
        if (CS > 1) cluster_sync();
        else __syncthreads();
    };
    int turn = 0;
    // Every block gives two values (the same in all its threads) and gets all blocks': s.push[turn][kind][block].  Two sets in
    // turn: a set is written again only after another exchange, whose barrier lies after every read of it.
    auto exchange = [&](u64 v0, u64 v1) {
        turn ^= 1;
        if (tid < CS) {
            const uint32_t base = peer(smem_addr(&s.push[turn][0][rank]), tid);
            peer_st64(base, v0), peer_st64(base + 64, v1);
        }
        sync_all();
    };
    auto max64 = [](u64 p, u64 q) { return p > q ? p : q; };
    auto min64 = [](u64 p, u64 q) { return p < q ? p : q; };
    auto add64 = [](u64 p, u64 q) { return p + q; };
    auto block_reduce = [&](u64 v, int set, auto&& op) {
        v = warp_reduce(v, op);
        __syncthreads();
        if (lane == 0) s.red[set][warp] = v;
        __syncthreads();
        v = s.red[set][0];
        for (int w = 1; w < SW; ++w) v = op(v, s.red[set][w]);
        return v;
    };

    const float T = a.temperature ? a.temperature[row] : 1.f;
    int k = a.top_k ? a.top_k[row] : 0;
    const float top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f;
    const float u = a.u[row];
    // (a rate of 0 would make NaN of a -inf logit)
    const float rate = fmaxf(1.f / T, 1e-38f);
    // filters that leave rank 0 alone, whatever the weights: greedy, and bounds that nothing else can meet
    if (!(T > 0.f) || !(rate < 3e38f) || !(top_p > 0.f) || !(min_p <= 1.f)) k = 1;
    if (k <= 0 || k > N) k = N;

    // ---- the slice into shared memory, and its largest logit (NaN ranks above everything, as in torch.argmax)
    float largest = NONE;
    {
        constexpr int U = 5;
        for (int i0 = tid; i0 < vecs; i0 += U * ST) {
            uint4 w[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (wide && (i0 + j * ST + 1) * V <= n) w[j] = reinterpret_cast<const uint4*>(src)[i0 + j * ST];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int i = i0 + j * ST;
                if (i >= vecs) break;
                if (!wide || (i + 1) * V > n) {
                    alignas(16) raw p[V];
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        if (i * V + q < n) p[q] = src[i * V + q];
                        else if constexpr (XK == ACT_F32) p[q] = NONE;
                        else p[q] = XK == ACT_BF16 ? 0xff80 : 0xfc00;
                    }
                    w[j] = *reinterpret_cast<const uint4*>(p);
                }
                if (a.staged) stage[i] = w[j];
                float x[V];
                widen_all<XK>(w[j], x);
#pragma unroll
                for (int q = 0; q < V; ++q) largest = max_nan(largest, x[q]);
            }
        }
    }
    u64 best = block_reduce(largest != largest ? 0xffffffffull : static_cast<u64>(key_of(largest)), 0, max64);
    if (CS > 1) cluster_wait();  // the other blocks run
    exchange(best, 0);
    for (int b = 0; b < CS; ++b) best = max64(best, s.push[turn][0][b]);
    const uint32_t top_key = static_cast<uint32_t>(best);
    const float top = x_of(top_key);
    // NaN or +inf; nothing but -inf; or rank 0 alone
    const bool broken = top_key >= 0xff800000u, none = top_key <= 0x007fffffu;
    if (broken || none || k == 1) {
        u64 at = ~0ull;
        if (!none) for_all([&](float x, int i) {
            if (top_key == 0xffffffffu ? x != x : x == top) at = min64(at, static_cast<u64>(first + i));
        });
        at = block_reduce(at, 1, min64);
        exchange(at, 0);
        for (int b = 0; b < CS; ++b) at = min64(at, s.push[turn][0][b]);
        if (tid == 0 && rank == 0) {
            a.token[row] = none ? -1 : static_cast<int>(at);
            if (a.prob) a.prob[row] = none ? 0.f : broken ? __int_as_float(0x7fc00000) : 1.f;
        }
        return;
    }

    // ---- histogram of the undecided tokens: all (linear), or lo <= c <= hi in bins of 2^shift
    u64 lo = 0, hi = 0;
    bool linear = true;
    int shift = 0;
    auto c_of = [&](float x, int i) { return place_of(key_of(x), first + i); };
    auto fill = [&](bool counts, bool masses) {
        for (int b = tid; b < BINS; b += ST) s.lo[b] = s.hi[b] = s.count[b] = 0;
        __syncthreads();
        auto add = [&](int b, float x) {
            if (counts) atomicAdd(&s.count[b], 1u);
            if (!masses) return;
            const u64 w = mass_of(e_of(x, top, rate));
            const uint32_t w0 = static_cast<uint32_t>(w);
            uint32_t w1 = static_cast<uint32_t>(w >> 32);
            w1 += atomicAdd(&s.lo[b], w0) > ~w0;  // the carry of the lower word
            if (w1) atomicAdd(&s.hi[b], w1);
        };
        if (linear) for_all([&](float x, int) { add(bin_of(x, top, rate), x); });
        else for_all([&](float x, int i) {
            const u64 c = c_of(x, i);
            if (c >= lo && c <= hi) add(static_cast<int>((hi - c) >> shift), x);
        });
        __syncthreads();
    };
    // Adds up all blocks' bins, first in groups of 32, then in the group that reaches the bound; every block comes to the same bin.  above_*: before the bin, within_m: in it.  `all` receives the whole mass (first call).
    u64 above_n = 0, above_m = 0, within_m = 0, all = 0;
    auto find_bin = [&](auto&& reached) {
        int group = 0;
#pragma unroll 1
        for (int level = 0; level < 2; ++level) {
            u64 m, c;
            if (level == 0) {
                // a group is 32 / PER threads
                m = c = 0;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    m += (static_cast<u64>(s.hi[PER * tid + j]) << 32) + s.lo[PER * tid + j], c += s.count[PER * tid + j];
#pragma unroll
                for (int o = GROUP / PER / 2; o; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o), c += __shfl_xor_sync(0xffffffffu, c, o);
                if (tid % (GROUP / PER) == 0) s.group_m[tid / (GROUP / PER)] = m, s.group_n[tid / (GROUP / PER)] = c;
                __syncthreads();
                if (tid < 32 * CS) {
                    peer_st64(peer(smem_addr(&s.got_m[0][rank][lane]), warp), s.group_m[lane]);
                    peer_st64(peer(smem_addr(&s.got_n[0][rank][lane]), warp), s.group_n[lane]);
                }
            } else if (tid < 32 * CS) {
                const int at = group * GROUP + lane;
                m = (static_cast<u64>(s.hi[at]) << 32) + s.lo[at], c = s.count[at];
                peer_st64(peer(smem_addr(&s.got_m[1][rank][lane]), warp), m);
                peer_st64(peer(smem_addr(&s.got_n[1][rank][lane]), warp), c);
            }
            sync_all();
            if (warp == 0) {
                m = c = 0;
                for (int b = 0; b < CS; ++b) m += s.got_m[level][b][lane], c += s.got_n[level][b][lane];
                const u64 sm = warp_scan(m, lane), sc = warp_scan(c, lane);
                if (level == 0 && linear) all = __shfl_sync(0xffffffffu, sm, 31);
                const unsigned hit = __ballot_sync(0xffffffffu, reached(above_n + sc, above_m + sm));
                const int l = hit ? __ffs(hit) - 1 : 31;
                if (lane == l) s.found[level][0] = l, s.found[level][1] = above_n + sc - c, s.found[level][2] = above_m + sm - m, s.found[level][3] = m;
                if (lane == 0) s.found[level][4] = all;
            }
            __syncthreads();
            const int l = static_cast<int>(s.found[level][0]);
            above_n = s.found[level][1], above_m = s.found[level][2], within_m = s.found[level][3], all = s.found[level][4];
            group = level == 0 ? l : group * GROUP + l;
        }
        return group;
    };
    // Gathers tokens into the block's list; tells all blocks how many there are.
    unsigned members = 0;
    auto put = [&](float x, int i) {
        const unsigned p = atomicAdd(&s.used, 1u);
        if (p < CAP) s.list[p] = c_of(x, i);
    };
    auto gather = [&](auto&& all_of) {
        if (tid == 0) s.used = 0;
        __syncthreads();
        all_of();
        __syncthreads();
        exchange(s.used, 0);
        members = 0;
        for (int b = 0; b < CS; ++b) members += static_cast<unsigned>(s.push[turn][0][b]);
    };
    // Logits of the bins up to `bin` are at least least_of, those of the bins from `bin` on at most most_of (bin_of has three
    // roundings, these two more: the margins are wider).
    const float INF = __int_as_float(0x7f800000);
    auto edge = [&](float bins, float margin) {
        const float x = top - bins / (rate * BIN_RATE) * (1.f + margin);
        return x - (fabsf(x) + fabsf(top)) * (0.4f * margin);
    };
    auto least_of = [&](int bin) { return bin >= BINS - 1 ? NONE : edge(static_cast<float>(bin + 1), 1e-6f); };
    auto most_of = [&](int bin) {
        if (bin == 0) return INF;
        const float x = edge(static_cast<float>(bin), -1e-6f);
        return x == x ? x : INF;  // (NaN where the edge lies below every fp32: a temperature above 1e37)
    };
    // the tokens from `least` to `most` that take(x, i) wants
    auto gather_range = [&](float least, float most, auto&& take) {
        gather([&] {
            for_pieces([&](const float (&x)[V], int i) {
                bool any = false;
#pragma unroll
                for (int q = 0; q < V; ++q) any |= x[q] >= least && x[q] <= most;
                if (!any) return;
#pragma unroll
                for (int q = 0; q < V; ++q)
                    if (x[q] >= least && x[q] <= most && take(x[q], i * V + q)) put(x[q], i * V + q);
            });
        });
    };
    // All blocks' lists, at most CAP tokens, sorted: thread t gets the c of rank t (0 past the last).
    auto sorted = [&](u64 v, unsigned count) {  // descending, over the first threads; a bitonic network
        int width = 1;
        while (static_cast<unsigned>(width) < count) width <<= 1;
        const bool in = warp * 32 < width;  // (the other warps would only take turns from these)
        auto turn_with = [&](u64 o, int j, int size) {
            const bool larger = ((tid & j) == 0) == ((tid & size) == 0);
            v = (v > o) == larger ? v : o;
        };
#pragma unroll 1
        for (int size = 2; size <= width; size <<= 1) {
#pragma unroll 1
            for (int j = size >> 1; j >= 32; j >>= 1) {
                __syncthreads();
                if (in) line[tid] = v;
                __syncthreads();
                if (in) turn_with(line[tid ^ j], j, size);
            }
            if (!in) continue;
#pragma unroll
            for (int j = 16; j; j >>= 1)
                if (j < size) turn_with(__shfl_xor_sync(0xffffffffu, v, j), j, size);
        }
        return v;
    };
    auto collect = [&] {
        unsigned base = 0;
        u64 c = 0;
        for (int b = 0; b < CS; ++b) {
            const unsigned nb = static_cast<unsigned>(s.push[turn][0][b]);
            if (tid >= base && tid < base + nb) c = peer_ld64(peer(smem_addr(s.list), b) + 8 * (tid - base));
            base += nb;
        }
        return sorted(c, members);
    };
    auto x_at = [&](u64 c) { return x_of(static_cast<uint32_t>(c >> 20)); };
    // Sum over the threads up to this one, and over all of them.
    auto block_scan = [&](u64 v, u64* total) {
        const u64 run = warp_scan(v, lane);
        __syncthreads();
        if (lane == 31) s.red[2][warp] = run;
        __syncthreads();
        u64 before = 0, sum = 0;
        for (int w = 0; w < SW; ++w) {
            if (w < warp) before += s.red[2][w];
            sum += s.red[2][w];
        }
        *total = sum;
        return before + run;
    };
    // The draw from a list that holds every token that may be kept; `of`: the mass that top-p is a share of, 0 for that of the tokens that
    // top-k keeps.
    auto draw_from_list = [&](u64 of) {
        if (rank == 0) {
            const u64 c = collect();
            const float e = e_of(x_at(c), top, rate);
            const u64 w = tid < members ? mass_of(e) : 0;
            u64 among;
            const u64 before = block_scan(tid < k ? w : 0, &among) - w;  // (of use where tid < k)
            bool keep = tid < members && tid < k && e >= min_p;
            if (top_p < 1.f) keep = keep && static_cast<double>(before) < static_cast<double>(top_p) * static_cast<double>(of ? of : among);
            // in index order (the lower bits of c fall as the index grows): a short list by comparing each token with all, with as many
            // threads a token as there are; a long one by sorting once more
            u64 W, until, its = c, its_w = keep ? w : 0;
            float its_e = e;
            if (members <= 128) {
                __syncthreads();
                line[tid] = c, line[ST + tid] = its_w;
                __syncthreads();
                int bits = 2;
                while (members << (bits + 1) <= ST && bits < 5) ++bits;
                const int which = tid >> bits, part = tid & ((1 << bits) - 1);
                its = line[which], its_w = line[ST + which], its_e = e_of(x_at(its), top, rate);
                u64 sum = 0, upto = 0;
#pragma unroll 4
                for (int j = part; j < static_cast<int>(members); j += 1 << bits) {
                    const u64 v = line[ST + j];
                    sum += v;
                    if ((line[j] & 0xFFFFFu) >= (its & 0xFFFFFu)) upto += v;
                }
                for (int o = 1 << bits >> 1; o; o >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, o), upto += __shfl_xor_sync(0xffffffffu, upto, o);
                W = sum, until = upto;
                if (which >= static_cast<int>(members) || part) until = 0;  // (one thread a token tells)
            } else {
                const u64 next = sorted(keep ? 1ull << 62 | (c & 0xFFFFFu) << 32 | static_cast<unsigned>(tid) : 0, members);
                __syncthreads();
                line[tid] = c;
                __syncthreads();
                its = next ? line[next & (ST - 1)] : 0;
                its_e = e_of(x_at(its), top, rate);
                its_w = next ? mass_of(its_e) : 0;
                until = block_scan(its_w, &W);
            }
            u64 target = static_cast<u64>(static_cast<double>(u) * static_cast<double>(W));
            if (target >= W) target = W - 1;
            if (until > target && until - its_w <= target) {
                a.token[row] = static_cast<int>(0xFFFFFu - (its & 0xFFFFFu));
                if (a.prob) a.prob[row] = its_e / (static_cast<float>(W) * 0x1p-42f);
            }
        }
        sync_all();  // no block ends while its list is read
    };
    // The smallest c that a filter keeps, from the histogram's bin on; *mass: the sum of w over c >= cut, *own: of this block's.
    auto cut_of = [&](int bin, auto&& reached, u64* mass, u64* own) {
        auto own_above = [&] {  // this block's mass in the bins before
            u64 m = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (PER * tid + j < bin) m += (static_cast<u64>(s.hi[PER * tid + j]) << 32) + s.lo[PER * tid + j];
            return block_reduce(m, 0, add64);
        };
        *own = own_above();
        for (;;) {
            auto in_bin = [&](float x, int i) {
                if (linear) return bin_of(x, top, rate) == bin;
                const u64 c = c_of(x, i);
                return c >= lo && c <= hi && static_cast<int>((hi - c) >> shift) == bin;
            };
            gather_range(linear ? least_of(bin) : NONE, linear ? most_of(bin) : INF, in_bin);
            if (members <= CAP) break;
            // too many: split the bin by c
            u64 cmin = ~0ull, cmax = 0;
            for_all([&](float x, int i) {
                if (in_bin(x, i)) cmin = min64(cmin, c_of(x, i)), cmax = max64(cmax, c_of(x, i));
            });
            cmin = block_reduce(cmin, 0, min64), cmax = block_reduce(cmax, 1, max64);
            exchange(cmin, cmax);
            for (int b = 0; b < CS; ++b) cmin = min64(cmin, s.push[turn][0][b]), cmax = max64(cmax, s.push[turn][1][b]);
            lo = cmin, hi = cmax, linear = false;
            const int bits = 64 - __clzll(static_cast<long long>(hi - lo));
            shift = max(0, bits - 10);
            fill(true, true);
            bin = find_bin(reached);
            *own += own_above();
        }
        // the first block decides on the list, and tells the others the cut and the mass
        u64 cut = 0, kept = 0;
        if (rank == 0) {
            const u64 c = collect();
            const u64 w = tid < members ? mass_of(e_of(x_at(c), top, rate)) : 0;
            u64 unused;
            const u64 until = block_scan(w, &unused);
            const bool keep = tid < members && !reached(above_n + tid, above_m + until - w);  // rank < k, or mass before < reach
            kept = above_m + block_reduce(keep ? w : 0, 1, add64);
            cut = block_reduce(keep ? c : ~0ull, 0, min64);
        }
        const unsigned listed = min(s.used, static_cast<unsigned>(CAP));
        exchange(cut, kept);
        cut = s.push[turn][0][0], *mass = s.push[turn][1][0];
        const u64 c = tid < listed ? s.list[tid] : 0;
        *own += block_reduce(c >= cut ? mass_of(e_of(x_at(c), top, rate)) : 0, 0, add64);
        return cut;
    };

    u64 cut = 0, kept_mass = 0, own_mass = 0;
    if (k < N) {
        auto reached = [&](u64 qc, u64) { return qc >= static_cast<u64>(k); };
        if (k <= CAP) {
            for (int b = tid; b < BINS; b += ST) s.lo[b] = s.hi[b] = s.count[b] = 0;
            __syncthreads();
            if (tid < vecs) atomicAdd(&s.count[bin_of(largest, top, rate)], 1u);
            __syncthreads();
            gather_range(least_of(find_bin(reached)), INF, [](float, int) { return true; });
            if (members <= CAP) {
                draw_from_list(0);
                return;
            }
            above_n = above_m = 0;
        }
        fill(true, true);
        cut = cut_of(find_bin(reached), reached, &kept_mass, &own_mass);
    }
    if (top_p < 1.f) {
        // (top-k's histogram still holds unless it was split)
        above_n = above_m = 0;
        if (k == N || !linear) linear = true, fill(false, true);
        // (the whole mass is known from the first level of the search on)
        auto reached = [&](u64, u64 qm) {
            return static_cast<double>(qm) >= static_cast<double>(top_p) * static_cast<double>(k < N ? kept_mass : all);
        };
        const int bin = find_bin(reached);
        // a token of the bins up to this one weighs at least so much (with a margin for the roundings)
        const u64 least = mass_of(expf(-(bin + 1) / BIN_RATE) * 0.999f);
        if (k == N && (above_m + within_m) / 4 < least * (CAP / 4)) {
            gather_range(least_of(bin), INF, [](float, int) { return true; });
            if (members <= CAP) {
                draw_from_list(all);
                return;
            }
        }
        u64 mass, own;
        const u64 c = cut_of(bin, reached, &mass, &own);
        if (c >= cut) cut = c, own_mass = own;
    }

    // ---- the draw by a pass over the row: each thread owns a contiguous part of the slice (an odd number of pieces: the
    // threads of a quarter warp then read different banks).  With a cut and no min-p the blocks' masses are known, and only the block
    // that holds the target makes the pass.
    const int own_vecs = (vecs + ST - 1) / ST | 1, v0 = min(vecs, tid * own_vecs), v1 = min(vecs, v0 + own_vecs);
    const uint32_t cut_key = static_cast<uint32_t>(cut >> 20);
    auto weight = [&](float x, int i) -> u64 {
        const uint32_t key = key_of(x);
        const float e = e_of(x, top, rate);
        const bool in = (key > cut_key || (key == cut_key && place_of(key, first + i) >= cut)) && e >= min_p;
        return in ? mass_of(e) : 0;
    };
    u64 own = 0, mine = own_mass, start = 0;
    auto pass = [&] {
#pragma unroll 2
        for (int i = v0; i < v1; ++i) {
            float x[V];
            piece(i, x);
#pragma unroll
            for (int q = 0; q < V; ++q) own += weight(x[q], i * V + q);
        }
        start = block_scan(own, &mine) - own;
    };
    const bool known = cut != 0 && !(min_p > 0.f);
    if (!known) pass();
    exchange(mine, 0);
    u64 W = 0, block_start = 0;
    for (int b = 0; b < CS; ++b) {
        if (b < rank) block_start += s.push[turn][0][b];
        W += s.push[turn][0][b];
    }
    u64 target = static_cast<u64>(static_cast<double>(u) * static_cast<double>(W));
    if (target >= W) target = W - 1;
    if (target < block_start || target >= block_start + mine) return;
    if (known) pass();
    start += block_start;
    // the thread whose part holds the target; its warp shares the part
    const unsigned holds = __ballot_sync(0xffffffffu, start <= target && target < start + own);
    if (!holds) return;
    const int owner = __ffs(holds) - 1;
    u64 base = __shfl_sync(0xffffffffu, start, owner);
    const int i0 = __shfl_sync(0xffffffffu, v0 * V, owner), i1 = __shfl_sync(0xffffffffu, v1 * V, owner);
    for (int j = i0; j < i1; j += 32) {
        const int i = j + lane;
        const float x = i < i1 ? token(i) : NONE;
        const u64 w = i < i1 ? weight(x, i) : 0, sum = warp_scan(w, lane) + base;
        if (sum > target && sum - w <= target) {
            a.token[row] = first + i;
            if (a.prob) a.prob[row] = e_of(x, top, rate) / (static_cast<float>(W) * 0x1p-42f);
        }
        base = __shfl_sync(0xffffffffu, sum, 31);
        if (base > target) break;
    }
}

unsigned sample_smem_base() { return sizeof(SampleShared); }
const void* sample_kernel_ptr(int kind) {
    if (kind == ACT_F32) return (const void*)sample_kernel<ACT_F32>;
    return kind == ACT_BF16 ? (const void*)sample_kernel<ACT_BF16> : (const void*)sample_kernel<ACT_F16>;
}

}  // namespace qg
