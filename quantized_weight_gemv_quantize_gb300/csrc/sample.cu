// Sampling from logits with temperature, top-k, top-p and min-p: one cluster of blocks a row.
//
// Weights are whole numbers, w = floor(2^42 exp((x - max) / T)): their sums are exact in 64 bits whatever the order, so
// the result is the same on every run and for every split of the work (and the blocks may sum with atomics).  Nothing is
// sorted.  With c = (key bits of x, reversed index) as one number, the tokens that top-k and top-p keep are those with
// c >= cut.  The cut is found from a histogram (counts for top-k, masses for top-p) of 1024 bins that are linear in
// (max - x) / T: the bin in which the count or the mass reaches its bound is gathered, and each of its few tokens compares
// itself with the others.  A bin with more than CAP tokens is first split again, by c, until one has at most CAP (c differs
// for all tokens, so this ends even for a row of equal logits).
// Each block keeps its slice of the row in shared memory; the row is read once from global memory.  One row is bound by the
// latency of its few passes and cluster barriers, many rows by the arithmetic a token (one expf, one or two shared atomics).
#include "common.cuh"
#include "internal.h"
#include "step.h"

namespace qg {

using u64 = unsigned long long;

constexpr int ST = SAMPLE_THREADS, SW = ST / 32;
constexpr int BINS = 1024;
constexpr int CAP = 512;  // one token a thread in the comparison
static_assert(CAP <= ST, "");

// ---- cluster: barrier, and the same shared-memory address in another block
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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
__device__ __forceinline__ uint32_t peer_ld32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void peer_st64(uint32_t a, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// Unsigned key that orders as x does (both zeros alike).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ u64 place_of(uint32_t key, int i) { return static_cast<u64>(key) << 20 | (0xFFFFFu - i); }
__device__ __forceinline__ float e_of(float x, float top, float rate) { return expf((x - top) * rate); }
__device__ __forceinline__ u64 mass_of(float e) { return static_cast<u64>(__float2ull_rz(e * 0x1p42f)); }
// Monotone in x: 1024 bins over the 30 nats below the largest logit (2^-42 is 29.1), everything further in the last.
__device__ __forceinline__ int bin_of(float x, float top, float rate) {
    return min(BINS - 1, static_cast<int>((top - x) * rate * (BINS / 30.0f)));
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

struct alignas(16) SampleShared {  // the slice follows it in shared memory, written 16 bytes at a time
    uint32_t lo[BINS], hi[BINS], count[BINS];  // masses as two words (hi takes the carries of lo), counts
    u64 list_c[CAP], list_w[CAP];              // the tokens of this block in the bin that is split
    u64 all_c[CAP], all_w[CAP];                // and of the whole cluster
    u64 push[2][4][8];                         // what the blocks tell each other, by kind and block; two sets in turn
    u64 red[3][SW];
    u64 bc[8];
    unsigned used;
};

static_assert(sizeof(SampleShared) % 16 == 0, "");

template <class T, class Op>
__device__ __forceinline__ T warp_reduce(T v, Op op) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <int XK>
__global__ void __launch_bounds__(ST) sample_kernel(const SampleArgs a) {
    using raw = typename Raw<XK>::type;
    extern __shared__ __align__(16) uint8_t smem[];
    SampleShared& s = *reinterpret_cast<SampleShared*>(smem);
    raw* stage = reinterpret_cast<raw*>(smem + sizeof(SampleShared));
    pdl_launch_dependents();
    pdl_wait();
    const int CS = a.blocks, rank = static_cast<int>(blockIdx.x) % CS, row = static_cast<int>(blockIdx.x) / CS;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, N = a.N;
    const int first = rank * a.slice, n = max(0, min(a.slice, N - first));  // this block's tokens
    const raw* src = static_cast<const raw*>(a.x) + row * a.row_stride + first;
    auto at = [&](int i) { return widen<XK>(a.staged ? stage[i] : src[i]); };
    auto sync_all = [&] {
        if (CS > 1) cluster_sync();
        else __syncthreads();
    };
    int turn = 0;
    // Every block gives up to 3 values (thread 0's) and gets all blocks': s.push[turn][kind][block].  Two sets in turn: a set
    // is written again only after another exchange, whose barrier lies after every read of it.
    auto exchange = [&](u64 v0, u64 v1, u64 v2) {
        turn ^= 1;
        if (tid < CS) {
            const uint32_t base = peer(smem_addr(&s.push[turn][0][rank]), tid);
            peer_st64(base, v0), peer_st64(base + 64, v1), peer_st64(base + 128, v2);
        }
        sync_all();
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

    // ---- the slice into shared memory, and its largest token (NaN ranks above everything, as in torch.argmax)
    u64 best = 0;
    auto see = [&](raw w, int i) {
        const float x = widen<XK>(w);
        const u64 c = place_of(x != x ? 0xffffffffu : key_of(x), first + i);
        best = c > best ? c : best;
    };
    constexpr int V = 16 / sizeof(raw);
    const int vecs = reinterpret_cast<uintptr_t>(src) % 16 == 0 ? n / V : 0;
    {
        const uint4* sv = reinterpret_cast<const uint4*>(src);
        constexpr int U = 4;
        for (int i0 = tid; i0 < vecs; i0 += U * ST) {
            uint4 w[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (i0 + j * ST < vecs) w[j] = sv[i0 + j * ST];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int i = i0 + j * ST;
                if (i >= vecs) break;
                if (a.staged) reinterpret_cast<uint4*>(stage)[i] = w[j];
                const raw* e = reinterpret_cast<const raw*>(&w[j]);
#pragma unroll
                for (int q = 0; q < V; ++q) see(e[q], i * V + q);
            }
        }
        for (int i = vecs * V + tid; i < n; i += ST) {
            const raw w = src[i];
            if (a.staged) stage[i] = w;
            see(w, i);
        }
    }
    auto max64 = [](u64 p, u64 q) { return p > q ? p : q; };
    auto min64 = [](u64 p, u64 q) { return p < q ? p : q; };
    auto add64 = [](u64 p, u64 q) { return p + q; };
    best = warp_reduce(best, max64);
    if (lane == 0) s.red[0][warp] = best;
    __syncthreads();
    best = s.red[0][0];
    for (int w = 1; w < SW; ++w) best = max64(best, s.red[0][w]);
    exchange(best, 0, 0);
    for (int b = 0; b < CS; ++b) best = max64(best, s.push[turn][0][b]);
    const uint32_t top_key = static_cast<uint32_t>(best >> 20);
    const int top_at = static_cast<int>(0xFFFFFu - (best & 0xFFFFFu));
    // NaN or +inf; nothing but -inf; or rank 0 alone
    const bool broken = top_key >= 0xff800000u, none = top_key <= 0x007fffffu;
    if (broken || none || k == 1) {
        if (tid == 0 && rank == 0) {
            a.token[row] = none ? -1 : top_at;
            if (a.prob) a.prob[row] = none ? 0.f : broken ? __int_as_float(0x7fc00000) : 1.f;
        }
        return;
    }
    const float top = __uint_as_float(top_key & 0x80000000u ? top_key & 0x7fffffffu : ~top_key);

    // ---- the smallest c that a filter keeps: by count (rank < k) or by mass (the mass before < reach)
    // Returns the cut; *mass is the sum of w over c >= cut.  The reach is top_p of `of`, or of all mass where that is 0.
    auto find_cut = [&](bool by_count, u64 of, u64* mass) {
        const u64 bound_count = static_cast<u64>(k);
        u64 lo = 0, hi = 0, above_count = 0, above_mass = 0;
        double reach = 0.0;
        bool linear = true;
        int shift = 0;
        for (;;) {
            // the histogram of the undecided tokens (all, or lo <= c <= hi)
            for (int b = tid; b < BINS; b += ST) s.lo[b] = s.hi[b] = s.count[b] = 0;
            if (tid == 0) s.used = 0;
            __syncthreads();
            for (int i = tid; i < n; i += ST) {
                const float x = at(i);
                int b;
                if (linear) {
                    b = bin_of(x, top, rate);
                } else {
                    const u64 c = place_of(key_of(x), first + i);
                    if (c < lo || c > hi) continue;
                    b = static_cast<int>((hi - c) >> shift);
                }
                if (by_count) atomicAdd(&s.count[b], 1u);
                const u64 w = mass_of(e_of(x, top, rate));
                const uint32_t w0 = static_cast<uint32_t>(w);
                uint32_t w1 = static_cast<uint32_t>(w >> 32);
                if (w0) w1 += atomicAdd(&s.lo[b], w0) > ~w0;  // the carry of the lower word
                if (w1) atomicAdd(&s.hi[b], w1);
            }
            sync_all();
            // all blocks sum all blocks' bins (two a thread) and look for the bin that reaches the bound
            constexpr int PER = BINS / ST;
            u64 bm[PER] = {}, bn[PER] = {};
            for (int r = 0; r < CS; ++r) {
                const uint32_t l = peer(smem_addr(s.lo), r), h = peer(smem_addr(s.hi), r), c = peer(smem_addr(s.count), r);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const uint32_t off = 4u * (tid * PER + j);
                    bm[j] += static_cast<u64>(peer_ld32(l + off)) + (static_cast<u64>(peer_ld32(h + off)) << 32);
                    if (by_count) bn[j] += peer_ld32(c + off);
                }
            }
            u64 m = 0, cnt = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) m += bm[j], cnt += bn[j];
            const u64 own_m = m, own_c = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 pm = __shfl_up_sync(0xffffffffu, m, o), pc = __shfl_up_sync(0xffffffffu, cnt, o);
                if (lane >= o) m += pm, cnt += pc;
            }
            if (lane == 31) s.red[0][warp] = m, s.red[1][warp] = cnt;
            __syncthreads();
            u64 total = 0;
            for (int w = 0; w < SW; ++w) {
                if (w < warp) m += s.red[0][w], cnt += s.red[1][w];
                total += s.red[0][w];
            }
            if (linear) reach = static_cast<double>(top_p) * static_cast<double>(of ? of : total);
            // before this thread's bins
            u64 pm = above_mass + m - own_m, pc = above_count + cnt - own_c;
            auto reached = [&](u64 qc, u64 qm) { return by_count ? qc >= bound_count : static_cast<double>(qm) >= reach; };
            if (!reached(pc, pm)) {
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    if (!reached(pc, pm) && reached(pc + bn[j], pm + bm[j])) s.bc[0] = tid * PER + j, s.bc[1] = pc, s.bc[2] = pm;
                    pm += bm[j], pc += bn[j];
                }
            }
            __syncthreads();
            const int bin = static_cast<int>(s.bc[0]);
            above_count = s.bc[1], above_mass = s.bc[2];
            // gather the bin's tokens
            u64 cmin = ~0ull, cmax = 0;
            for (int i = tid; i < n; i += ST) {
                const float x = at(i);
                if (linear && bin_of(x, top, rate) != bin) continue;
                const u64 c = place_of(key_of(x), first + i);
                if (!linear && (c < lo || c > hi || static_cast<int>((hi - c) >> shift) != bin)) continue;
                cmin = min64(cmin, c), cmax = max64(cmax, c);
                const unsigned p = atomicAdd(&s.used, 1u);
                if (p < CAP) s.list_c[p] = c, s.list_w[p] = mass_of(e_of(x, top, rate));
            }
            cmin = warp_reduce(cmin, min64), cmax = warp_reduce(cmax, max64);
            if (lane == 0) s.red[0][warp] = cmin, s.red[1][warp] = cmax;
            __syncthreads();
            for (int w = 0; w < SW; ++w) cmin = min64(cmin, s.red[0][w]), cmax = max64(cmax, s.red[1][w]);
            exchange(s.used, cmin, cmax);
            unsigned members = 0;
            for (int b = 0; b < CS; ++b) {
                members += static_cast<unsigned>(s.push[turn][0][b]);
                cmin = min64(cmin, s.push[turn][1][b]), cmax = max64(cmax, s.push[turn][2][b]);
            }
            if (members > CAP) {  // split the bin by c
                lo = cmin, hi = cmax, linear = false;
                const int bits = 64 - __clzll(static_cast<long long>(hi - lo));
                shift = max(0, bits - 10);
                continue;
            }
            // each token of the bin against the others
            unsigned base = 0;
            for (int b = 0; b < CS; ++b) {
                const unsigned nb = static_cast<unsigned>(s.push[turn][0][b]);
                const uint32_t c = peer(smem_addr(s.list_c), b), w = peer(smem_addr(s.list_w), b);
                for (unsigned i = tid; i < nb; i += ST) s.all_c[base + i] = peer_ld64(c + 8 * i), s.all_w[base + i] = peer_ld64(w + 8 * i);
                base += nb;
            }
            __syncthreads();
            u64 cut = ~0ull, kept = 0;
            if (tid < members) {
                const u64 c = s.all_c[tid];
                u64 before = above_mass, place = above_count;
                for (unsigned j = 0; j < members; ++j)
                    if (s.all_c[j] > c) before += s.all_w[j], ++place;
                if (!reached(place, before)) cut = c, kept = s.all_w[tid];  // rank < k, or mass before < reach
            }
            cut = warp_reduce(cut, min64), kept = warp_reduce(kept, add64);
            if (lane == 0) s.red[0][warp] = cut, s.red[1][warp] = kept;
            __syncthreads();
            kept = above_mass;
            for (int w = 0; w < SW; ++w) cut = min64(cut, s.red[0][w]), kept += s.red[1][w];
            *mass = kept;
            return cut;
        }
    };
    u64 cut = 0, kept = 0;
    if (k < N) cut = find_cut(true, 0, &kept);
    if (top_p < 1.f) {
        u64 unused;
        cut = max64(cut, find_cut(false, kept, &unused));
    }

    // ---- the kept mass, by warp: each owns a contiguous piece of the slice
    const int piece = (n + SW - 1) / SW, p0 = min(n, warp * piece), p1 = min(n, p0 + piece);
    auto weight = [&](int i) {
        const float x = at(i), e = e_of(x, top, rate);
        return place_of(key_of(x), first + i) >= cut && e >= min_p ? mass_of(e) : 0ull;
    };
    u64 sum = 0;
    for (int i = p0 + lane; i < p1; i += 32) sum += weight(i);
    sum = warp_reduce(sum, add64);
    __syncthreads();
    if (lane == 0) s.red[2][warp] = sum;
    __syncthreads();
    u64 mine = 0, before_warp = 0;
    for (int w = 0; w < SW; ++w) {
        if (w < warp) before_warp += s.red[2][w];
        mine += s.red[2][w];
    }
    exchange(mine, 0, 0);
    u64 W = 0, before = 0;
    for (int b = 0; b < CS; ++b) {
        if (b < rank) before += s.push[turn][0][b];
        W += s.push[turn][0][b];
    }
    u64 target = static_cast<u64>(static_cast<double>(u) * static_cast<double>(W));
    if (target >= W) target = W - 1;
    // ---- the warp whose piece holds the target: its lanes sum a contiguous part each, then share the part that holds it
    const u64 start = before + before_warp;
    if (target < start || target >= start + sum) return;
    const int part = (p1 - p0 + 31) / 32, q0 = min(p1, p0 + lane * part), q1 = min(p1, q0 + part);
    u64 own = 0;
    for (int i = q0; i < q1; ++i) own += weight(i);
    u64 run = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
    }
    run += start;
    const int owner = __ffs(__ballot_sync(0xffffffffu, run > target)) - 1;
    u64 base = __shfl_sync(0xffffffffu, run - own, owner);
    const int r0 = __shfl_sync(0xffffffffu, q0, owner), r1 = __shfl_sync(0xffffffffu, q1, owner);
    for (int i0 = r0; i0 < r1; i0 += 32) {
        const int i = i0 + lane;
        u64 v = i < r1 ? weight(i) : 0ull;
        const u64 w = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        v += base;
        if (v > target && v - w <= target) {
            a.token[row] = first + i;
            if (a.prob) a.prob[row] = e_of(at(i), top, rate) / (static_cast<float>(W) * 0x1p-42f);
        }
        base = __shfl_sync(0xffffffffu, v, 31);
        if (base > target) break;
    }
}

unsigned sample_smem_base() { return sizeof(SampleShared); }
const void* sample_kernel_ptr(int kind) {
    if (kind == ACT_F32) return (const void*)sample_kernel<ACT_F32>;
    return kind == ACT_BF16 ? (const void*)sample_kernel<ACT_BF16> : (const void*)sample_kernel<ACT_F16>;
}

}  // namespace qg
