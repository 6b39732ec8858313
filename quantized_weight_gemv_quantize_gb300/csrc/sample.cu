// Sampling from logits with temperature, top-k, top-p and min-p: one block a row.
//
// Weights are whole numbers, w = floor(2^42 exp((x - max) / T)): their sums are exact in 64 bits whatever the order, so
// the result is the same on every run and for every split of the work.  Nothing is sorted.  The tokens that the filters
// keep are a prefix of the order (x descending, index ascending); its end is found by a radix descent over the 32 key
// bits of x (8 bits a pass, counts and masses per bin), for top-k by count and for top-p by mass.
#include "common.cuh"
#include "internal.h"
#include "step.h"

namespace qg {

using u64 = unsigned long long;

constexpr int SAMPLE_THREADS = 1024;

template <int XK>
__device__ __forceinline__ float logit(const void* x, long long i) {
    if constexpr (XK == ACT_F32) return static_cast<const float*>(x)[i];
    const uint16_t w = static_cast<const uint16_t*>(x)[i];
    if constexpr (XK == ACT_BF16) return __uint_as_float(static_cast<uint32_t>(w) << 16);
    return h2f(w);
}

// Unsigned key that orders as x does (both zeros alike).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float e_of(float x, float top, float rate) { return expf((x - top) * rate); }
__device__ __forceinline__ u64 mass_of(float e) { return static_cast<u64>(__float2ull_rz(e * 0x1p42f)); }

template <class T, class Op>
__device__ __forceinline__ T block_reduce(T v, T* buf, Op op) {
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    v = buf[0];
    for (int w = 1; w < SAMPLE_THREADS / 32; ++w) v = op(v, buf[w]);
    return v;
}

// End of a prefix of the order: every key above `key`, and the first `ties` (by index) of the tokens with that key.
struct Cut {
    uint32_t key;
    u64 ties;
};

template <int XK>
__global__ void __launch_bounds__(SAMPLE_THREADS) sample_kernel(const SampleArgs a) {
    __shared__ u64 mass[256];
    __shared__ unsigned count[256];
    __shared__ u64 red[32];
    __shared__ u64 bc[4];
    pdl_launch_dependents();
    pdl_wait();
    const int row = blockIdx.x, tid = threadIdx.x, N = a.N;
    const long long x0 = row * a.row_stride;
    const float T = a.temperature ? a.temperature[row] : 1.f;
    int k = a.top_k ? a.top_k[row] : 0;
    float top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f;
    const float u = a.u[row];
    // (a rate of 0 would make NaN of a -inf logit)
    const float rate = fmaxf(1.f / T, 1e-38f);
    // filters that leave rank 0 alone, whatever the weights: greedy, and bounds that nothing else can meet
    if (!(T > 0.f) || !(rate < 3e38f) || !(top_p > 0.f) || !(min_p <= 1.f)) k = 1;
    if (k <= 0 || k > N) k = N;
    if (k == 1) top_p = 1.f;

    // the largest key and its first index; NaN ranks above everything, as in torch.argmax
    u64 best = 0;
    for (int i = tid; i < N; i += SAMPLE_THREADS) {
        const float x = logit<XK>(a.x, x0 + i);
        const uint32_t key = x != x ? 0xffffffffu : key_of(x);
        const u64 c = static_cast<u64>(key) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
        best = c > best ? c : best;
    }
    best = block_reduce(best, red, [](u64 p, u64 q) { return p > q ? p : q; });
    const uint32_t top_key = static_cast<uint32_t>(best >> 32);
    const int top_at = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
    const float top = logit<XK>(a.x, x0 + top_at);
    if (top_key >= 0xff800000u || top_key <= 0x007fffffu) {  // NaN or +inf; or nothing but -inf
        if (tid == 0) {
            const bool none = top_key <= 0x007fffffu;
            a.token[row] = none ? -1 : top_at;
            if (a.prob) a.prob[row] = none ? 0.f : __int_as_float(0x7fc00000);
        }
        return;
    }
    if (k == 1) {
        if (tid == 0) {
            a.token[row] = top_at;
            if (a.prob) a.prob[row] = 1.f;
        }
        return;
    }
    auto total_if = [&](auto&& keep) {
        u64 s = 0;
        for (int i = tid; i < N; i += SAMPLE_THREADS) {
            const float x = logit<XK>(a.x, x0 + i), e = e_of(x, top, rate);
            if (keep(x, e)) s += mass_of(e);
        }
        return block_reduce(s, red, [](u64 p, u64 q) { return p + q; });
    };

    // Radix descent: `done(count, mass)` says whether a prefix with these sums reaches past the cut.
    auto descend = [&](auto&& done, u64* above_count, u64* above_mass, u64* ties, u64* tie_mass) {
        uint32_t prefix = 0, fixed = 0;  // key bits that are settled
        u64 ac = 0, am = 0, tc = 0, tm = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            for (int b = tid; b < 256; b += SAMPLE_THREADS) mass[b] = 0, count[b] = 0;
            __syncthreads();
            for (int i = tid; i < N; i += SAMPLE_THREADS) {
                const float x = logit<XK>(a.x, x0 + i);
                const uint32_t key = key_of(x);
                if ((key & fixed) != prefix) continue;
                const int b = key >> shift & 255;
                atomicAdd(&count[b], 1u);
                const u64 w = mass_of(e_of(x, top, rate));
                if (w) atomicAdd(&mass[b], w);
            }
            __syncthreads();
            if (tid == 0) {
                int b = 255, last = 255;
                u64 c = ac, m = am, lc = ac, lm = am;
                for (; b >= 0; --b) {
                    if (!count[b]) continue;
                    last = b, lc = c, lm = m;
                    c += count[b], m += mass[b];
                    if (done(c, m)) break;
                }
                bc[0] = last, bc[1] = lc, bc[2] = lm;
            }
            __syncthreads();
            const uint32_t b = static_cast<uint32_t>(bc[0]);
            ac = bc[1], am = bc[2], tc = count[b], tm = mass[b];
            prefix |= b << shift;
            fixed |= 255u << shift;
        }
        *above_count = ac, *above_mass = am, *ties = tc, *tie_mass = tc ? tm / tc : 0;
        return prefix;
    };

    Cut cut = {0u, static_cast<u64>(N)};
    u64 total = 0;
    u64 ac, am, tc, tw;
    if (k < N) {
        const u64 kk = static_cast<u64>(k);
        cut.key = descend([&](u64 c, u64) { return c >= kk; }, &ac, &am, &tc, &tw);
        cut.ties = kk - ac;
        total = am + cut.ties * tw;
    }
    if (top_p < 1.f) {
        if (k == N) total = total_if([](float, float) { return true; });
        const double reach = static_cast<double>(top_p) * static_cast<double>(total);
        const uint32_t key =
            descend([&](u64, u64 m) { return static_cast<double>(m) >= reach; }, &ac, &am, &tc, &tw);
        // ties kept: those i whose mass before, am + i tw, is below the reach
        u64 lo = 0, hi = tc;
        while (lo < hi) {
            const u64 mid = (lo + hi) / 2;
            if (static_cast<double>(am + mid * tw) < reach) lo = mid + 1;
            else hi = mid;
        }
        if (key > cut.key || (key == cut.key && lo < cut.ties)) cut.key = key, cut.ties = lo;
    }
    // kept: above the cut or among its first ties, and not below min-p (rank 0 always is: its e is 1)
    u64 W = 0, tied = 0;
    for (int i = tid; i < N; i += SAMPLE_THREADS) {
        const float x = logit<XK>(a.x, x0 + i), e = e_of(x, top, rate);
        const uint32_t key = key_of(x);
        if (key > cut.key && e >= min_p) W += mass_of(e);
        else if (key == cut.key && e >= min_p) ++tied;
    }
    W = block_reduce(W, red, [](u64 p, u64 q) { return p + q; });
    tied = block_reduce(tied, red, [](u64 p, u64 q) { return p + q; });
    if (tied) {
        const float xc = __uint_as_float(cut.key & 0x80000000u ? cut.key & 0x7fffffffu : ~cut.key);
        W += (tied < cut.ties ? tied : cut.ties) * mass_of(e_of(xc, top, rate));
    }
    u64 target = static_cast<u64>(static_cast<double>(u) * static_cast<double>(W));
    if (target >= W) target = W - 1;

    // walk the tokens in index order, a block's width at a time, to the first whose running mass exceeds the target
    u64 run = 0, tied_run = 0;
    for (int i0 = 0; i0 < N; i0 += SAMPLE_THREADS) {
        const int i = i0 + tid;
        float x = 0.f, e = 0.f;
        bool in = false, tie = false;
        if (i < N) {
            x = logit<XK>(a.x, x0 + i);
            e = e_of(x, top, rate);
            const uint32_t key = key_of(x);
            tie = key == cut.key && e >= min_p;
            in = key > cut.key && e >= min_p;
        }
        // rank among the ties
        const unsigned tb = __ballot_sync(0xffffffffu, tie);
        __syncthreads();
        if (tid % 32 == 0) count[tid / 32] = __popc(tb);
        __syncthreads();
        u64 before = tied_run, all = 0;
        for (int w = 0; w < SAMPLE_THREADS / 32; ++w) {
            if (w < tid / 32) before += count[w];
            all += count[w];
        }
        before += __popc(tb & ((1u << (tid % 32)) - 1u));
        tied_run += all;
        in = in || (tie && before < cut.ties);
        u64 s = in ? mass_of(e) : 0;
        const u64 own = s;
        for (int o = 1; o < 32; o <<= 1) {
            const u64 v = __shfl_up_sync(0xffffffffu, s, o);
            if (tid % 32 >= o) s += v;
        }
        if (tid % 32 == 31) red[tid / 32] = s;
        __syncthreads();
        u64 base = run, sum = 0;
        for (int w = 0; w < SAMPLE_THREADS / 32; ++w) {
            if (w < tid / 32) base += red[w];
            sum += red[w];
        }
        s += base;
        if (in && s > target && s - own <= target) {
            a.token[row] = i;
            if (a.prob) a.prob[row] = e / (static_cast<float>(W) * 0x1p-42f);
        }
        run += sum;
        if (run > target) break;
    }
}

const void* sample_kernel_ptr(int kind) {
    if (kind == ACT_F32) return (const void*)sample_kernel<ACT_F32>;
    return kind == ACT_BF16 ? (const void*)sample_kernel<ACT_BF16> : (const void*)sample_kernel<ACT_F16>;
}

}  // namespace qg
