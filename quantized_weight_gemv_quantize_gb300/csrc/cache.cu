// Writing into and reading from a packed cache.
//
// Both move a token's pieces of 8 elements, keys' heads first, then values': a piece's place within the token is worked out once a thread and
// kept over the tokens of a block; the tokens' places in the cache are looked up once a block, into shared memory.
//
// Both are bound by memory for long runs, with the arithmetic of a value close behind (issue slots 65% taken by the write, 71% by the read), and by their launch for short
// ones.  8 heads of 128 (us; bytes at a copy's rate in brackets): 16000 tokens written in 4 bits from bf16 23 to 25 (12.6), from fp32 29 (22), in 8 bits 25 (15), 31 (25); read back
// to bf16 18.8 (12.6); 100003 tokens read to bf16 97 (79), in 8 bits 109 (89); one token either way 7, of which 5 are the caller's.  Steps on the way, writing
// and reading 16000: values converted as they came, one token a thread in flight 55.7 and 31; values packed until they are stored, four tokens
// in flight, the codes' arithmetic as in codes8 27 and 20.6; codes made floats where they stand (Packed8) 18.8; a block's step and base found once, not
// by each of its four lanes, 24.8.  Blocks of 128 threads write as fast or faster than ones of 256 (fp32 29 for 33) and read 16000 tokens slower (20.7), long
// runs a little faster (8 bits 105).
#include "attn.cuh"
#include "cache_rows.cuh"

namespace qg {

// Threads of a block over a token's pieces: `wide` of them side by side, and as many tokens at a time as there is room for.  (Pieces a
// token are a multiple of 8, so that a block of 32 elements stays with four neighbouring lanes.)
struct Lay {
    int wide, at, deep, row;  // this thread: pieces at, at + wide, ... of the block's tokens row, row + deep, ...
    __device__ __forceinline__ Lay(int pieces, int threads) {
        wide = min(pieces, threads);
        deep = threads / wide;
        at = threadIdx.x % wide, row = threadIdx.x / wide;
    }
};

// Four tokens' loads of a thread are on their way at once, as many as lanes share a block of 32 elements.
constexpr int AHEAD = 4;

template <int BITS, int XK>
__global__ void __launch_bounds__(WRITE_THREADS) cache_write_kernel(const CacheWriteArgs a) {
    __shared__ long long ks[CACHE_TOKENS], vs[CACHE_TOKENS];
    pdl_launch_dependents();
    pdl_wait();
    const long long first = static_cast<long long>(blockIdx.x) * a.block_tokens;
    const int n = static_cast<int>(min(static_cast<long long>(a.block_tokens), a.tokens - first));
    if (threadIdx.x < n) {
        const long long slot = a.slots[first + threadIdx.x];
        long long k = -1, v = -1;
        if (slot >= a.num_slots) {
            atomicOr(a.err, ERR_BAD_INDEX);
        } else if (slot >= 0) {
            const long long page = a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page_size, token = slot - page * a.page_size;
            k = page * a.kc_page + token * a.kc_token, v = page * a.vc_page + token * a.vc_token;
        }
        ks[threadIdx.x] = k, vs[threadIdx.x] = v;
    }
    __syncthreads();
    const int per_head = a.dim / 8, half = a.heads * per_head;
    const Lay lay(2 * half, WRITE_THREADS);
    if (lay.row >= lay.deep) return;  // (threads beyond the last whole token)
    const unsigned team = 0xFu << (threadIdx.x & 28);
    for (int p = lay.at; p < 2 * half; p += lay.wide) {
        const bool is_v = p >= half;
        const int h = (is_v ? p - half : p) / per_head, e = (p - (is_v ? half : 0) - h * per_head) * 8;
        const long long src = (is_v ? a.v_head : a.k_head) * h + e, token_step = is_v ? a.v_token : a.k_token;
        const void* x = is_v ? a.v : a.k;
        uint8_t* rows = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (is_v ? a.vc_head : a.kc_head) * h;
        const long long* place = is_v ? vs : ks;
        for (int t0 = lay.row; t0 < n; t0 += lay.deep * AHEAD) {
            Raw8<XK> v[AHEAD] = {};
            long long to[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int t = t0 + j * lay.deep;
                to[j] = t < n ? place[t] : -1;
                if (to[j] >= 0) v[j].load(x, (first + t) * token_step + src);
            }
            float lo[AHEAD], hi[AHEAD], w[8];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                v[j].values(w);
                ends8(w, lo[j], hi[j]);
            }
            // The four lanes of a block of 32 have a token each: its ends from the others, its step and base for them.
#pragma unroll
            for (int half = 2; half; half /= 2) {
#pragma unroll
                for (int i = 0; i < half; ++i) {
                    const bool upper = threadIdx.x & half;
                    const float lo_in = __shfl_xor_sync(team, upper ? lo[i] : lo[i + half], half), lo_own = upper ? lo[i + half] : lo[i];
                    const float hi_in = __shfl_xor_sync(team, upper ? hi[i] : hi[i + half], half), hi_own = upper ? hi[i + half] : hi[i];
                    lo[i] = fminf(lo_own, lo_in), hi[i] = max_or_nan(hi_own, hi_in);
                }
            }
            const BlockScale<BITS> s(lo[0], hi[0]);
            const long long own = threadIdx.x & 2 ? (threadIdx.x & 1 ? to[3] : to[2]) : (threadIdx.x & 1 ? to[1] : to[0]);
            if (own >= 0) s.put(rows + own, a.dim, e);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const float m = __shfl_sync(team, s.m, j, 4), rate = __shfl_sync(team, s.rate, j, 4);
                if (to[j] < 0) continue;
                v[j].values(w);
                codes8<BITS>(rows + to[j], e, w, m, rate);
            }
        }
    }
}

template <int BITS>
__global__ void __launch_bounds__(READ_THREADS) cache_read_kernel(const CacheReadArgs a) {
    __shared__ long long ks[CACHE_TOKENS], vs[CACHE_TOKENS];  // place of a row in the cache, -1: zeros, -2: not a row of any sequence
    pdl_launch_dependents();
    pdl_wait();
    const long long first = static_cast<long long>(blockIdx.x) * a.block_tokens;
    const int n = static_cast<int>(min(static_cast<long long>(a.block_tokens), a.tokens - first));
    if (threadIdx.x < n) {
        const int r = static_cast<int>(first) + threadIdx.x;
        // the last sequence that starts at or before the row
        int lo = 0, hi = a.seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.out_start[mid] <= r) lo = mid;
            else hi = mid;
        }
        long long k = -2, v = -2;
        const int start = max(0, a.out_start[lo]);
        if (r >= start && r < a.out_start[lo + 1]) {
            const long long t = static_cast<long long>(a.first ? a.first[lo] : 0) + (r - start);
            k = v = -1;
            if (t >= 0 && t < a.reach) {
                const long long nth = a.page_shift >= 0 ? t >> a.page_shift : t / a.page_size, token = t - nth * a.page_size;
                const int page = a.pages[lo * a.pages_stride + nth];
                if (page >= 0 && page < a.num_pages) k = page * a.kc_page + token * a.kc_token, v = page * a.vc_page + token * a.vc_token;
            }
            if (k < 0) atomicOr(a.err, ERR_BAD_INDEX);
        }
        ks[threadIdx.x] = k, vs[threadIdx.x] = v;
    }
    __syncthreads();
    const int per_head = a.dim / 8, half = a.heads * per_head;
    const int pieces = half * ((a.k_out ? 1 : 0) + (a.v_out ? 1 : 0));
    const Lay lay(pieces, READ_THREADS);
    if (lay.row >= lay.deep) return;
    for (int p = lay.at; p < pieces; p += lay.wide) {
        const bool is_v = !a.k_out || p >= half;
        const int in = p >= half ? p - half : p, h = in / per_head, e = (in - h * per_head) * 8;
        const int size = a.out_kind == ACT_F32 ? 4 : 2;
        const long long token_step = (is_v ? a.v_token : a.k_token) * size;
        char* y = static_cast<char*>(is_v ? a.v_out : a.k_out) + ((is_v ? a.v_head : a.k_head) * h + e) * size + (first + lay.row) * token_step;
        const uint8_t* rows = (is_v ? a.v_cache : a.k_cache) + (is_v ? a.vc_head : a.kc_head) * h;
        const uint8_t *codes = rows + e * BITS / 8, *step = rows + a.dim * BITS / 8 + e / 32 * 2;
        const long long* place = is_v ? vs : ks;
        for (int t0 = lay.row; t0 < n; t0 += lay.deep * AHEAD) {
            Packed8<BITS> v[AHEAD] = {};
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int t = t0 + j * lay.deep;
                if (t < n && place[t] >= 0) v[j].load(codes, step, a.dim / 16, place[t]);
            }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int t = t0 + j * lay.deep;
                float x[8];
                v[j].values(x);  // (nothing: zeros)
                if (t < n && place[t] >= -1) store8(a.out_kind, y, 0, x);
                y += lay.deep * token_step;
            }
        }
    }
}

// The keys and values that a batch's new tokens may see, in f16 and the order [page, head, token, dim] with pages of `page_size` tokens (a
// divisor of the cache's), page n of sequence b at b * per_seq + n, and their page table (-1: a page outside the cache).  A block takes
// CACHE_TOKENS tokens (blockIdx.x) of a sequence (blockIdx.y).  For attention by the 128-row kernel: every row tile of a sequence reads the copy.
//
// The copy is f16 whatever the queries' type: 11 bits of a value, where bf16's 8 would cost a context of 24000 keys as much again as the rounding of
// the result (0.0076 of it against 0.0017).  bf16 queries are taken along: in f16, times the power of two that brings the row's largest element to
// [2^9, 2^10), so that elements down to 2^-23 of it keep their 8 bits.
template <int BITS>
__global__ void __launch_bounds__(READ_THREADS) cache_unpack_kernel(const CacheUnpackArgs u) {
    __shared__ long long ks[CACHE_TOKENS], vs[CACHE_TOKENS];
    const AttnArgs& a = u.a;
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.y;
    const Seq s = find_seq(a, b);
    if (static_cast<int>(blockIdx.x) >= u.key_blocks) {  // a warp a row of dim elements, up to 128
        const int j0 = (static_cast<int>(blockIdx.x) - u.key_blocks) * UNPACK_QUERIES, rows = min(UNPACK_QUERIES, s.n - j0) * a.heads;
        const int lane = threadIdx.x % 32, e = 4 * lane;
        for (int i = threadIdx.x / 32; i < rows; i += READ_THREADS / 32) {
            const long long tok = s.q0 + j0 + i / a.heads;
            const int h = i % a.heads;
            uint2 w = make_uint2(0u, 0u);
            if (e < a.dim) w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + tok * a.q_token + h * a.q_head + e);
            float x[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
            float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int up = top > 0.f ? min(126, 136 - static_cast<int>(__float_as_uint(top) >> 23)) : 0;
            const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23), back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
            if (e < a.dim)
                *reinterpret_cast<uint2*>(u.q_copy + (tok * a.heads + h) * a.dim + e) =
                    make_uint2(pack16<false>(x[0] * by, x[1] * by), pack16<false>(x[2] * by, x[3] * by));
            if (lane == 0) u.units[tok * a.heads + h] = fminf(fmaxf(back * a.scale_log2, 1e-37f), 3e38f);
        }
        return;
    }
    const int t0 = static_cast<int>(blockIdx.x) * CACHE_TOKENS;
    const int from = max(t0, first_key(a, s.first_pos)), to = min(t0 + CACHE_TOKENS, s.usable);
    if (s.n <= 0 || from >= to) return;
    if (threadIdx.x < CACHE_TOKENS) {
        const int t = t0 + static_cast<int>(threadIdx.x);
        long long k = -1, v = -1;
        if (t >= from && t < to) {
            const int nth = div_by(t, a.page_size, a.page_shift), token = t - nth * a.page_size;
            const int page = a.pages[b * a.pages_stride + nth];
            const bool there = page >= 0 && page < a.num_pages;
            if (there) k = page * a.k_page + token * a.k_token, v = page * a.v_page + token * a.v_token;
            else atomicOr(a.err, ERR_BAD_INDEX);
            const int n = t >> u.page_shift;
            if ((t & (u.page_size - 1)) == 0 || t == from) u.table[b * u.per_seq + n] = there ? static_cast<int>(b * u.per_seq + n) : -1;
        }
        ks[threadIdx.x] = k, vs[threadIdx.x] = v;
    }
    __syncthreads();
    const int per_head = a.dim / 8, half = a.kv_heads * per_head;
    const Lay lay(2 * half, READ_THREADS);
    if (lay.row >= lay.deep) return;
    for (int p = lay.at; p < 2 * half; p += lay.wide) {
        const bool is_v = p >= half;
        const int in = is_v ? p - half : p, h = in / per_head, e = (in - h * per_head) * 8;
        void* y = is_v ? u.v_copy : u.k_copy;
        const uint8_t* rows = (is_v ? u.v + h * a.v_head : u.k + h * a.k_head);
        const uint8_t *codes = rows + e * BITS / 8, *step = rows + a.dim * BITS / 8 + e / 32 * 2;
        const long long* place = is_v ? vs : ks;
        for (int i0 = from - t0 + lay.row; i0 < to - t0; i0 += lay.deep * AHEAD) {
            Packed8<BITS> w[AHEAD] = {};
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int i = i0 + j * lay.deep;
                if (i < to - t0 && place[i] >= 0) w[j].load(codes, step, a.dim / 16, place[i]);
            }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int i = i0 + j * lay.deep;
                if (i >= to - t0 || place[i] < 0) continue;
                const int n = (t0 + i) >> u.page_shift;  // (a power of two)
                const long long row = ((b * u.per_seq + n) * a.kv_heads + h) * u.page_size + (t0 + i - (n << u.page_shift));
                float x[8];
                w[j].values(x);
#pragma unroll
                for (float& v : x) v = min_or_nan(max_or_nan(v, -65504.f), 65504.f);  // (d c + m may end a step's rounding beyond the largest f16)
                store8(ACT_F16, y, row * a.dim + e, x);
            }
        }
    }
}

template <int BITS>
static const void* pick_write(int x_kind) {
    if (x_kind == ACT_F32) return (const void*)cache_write_kernel<BITS, ACT_F32>;
    return x_kind == ACT_BF16 ? (const void*)cache_write_kernel<BITS, ACT_BF16> : (const void*)cache_write_kernel<BITS, ACT_F16>;
}

const void* cache_write_kernel_ptr(int bits, int x_kind) { return bits == 4 ? pick_write<4>(x_kind) : pick_write<8>(x_kind); }
const void* cache_unpack_kernel_ptr(int bits) { return bits == 4 ? (const void*)cache_unpack_kernel<4> : (const void*)cache_unpack_kernel<8>; }
const void* cache_read_kernel_ptr(int bits) { return bits == 4 ? (const void*)cache_read_kernel<4> : (const void*)cache_read_kernel<8>; }

}  // namespace qg
