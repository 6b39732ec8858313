// Rotary positions of new tokens' queries and keys, with the write of keys and values into a paged cache.
//
// A pair (a, b) of a head turns by t = 2 pi frac(p F / 2^64): p F wraps in 64-bit integer arithmetic, its upper 32
// bits are the signed fraction of a turn, and sincospif takes them without a range reduction.  The kernel reads q, k and
// v once and writes each result once; it is bound by those bytes, and by the launch for a few tokens.
#include "cache_rows.cuh"

namespace qg {

// 16000 tokens of 32 and 8 heads of 128, bf16: 68.1 us, 5.78 TB/s, 85% of what a plain copy reaches.  Small blocks suit it: 64 threads 68.1 us,
// 128 69.3, 256 77.9, 448 (one piece a thread) 101; two pieces a thread on their way before the table is ready cost registers and
// took 89.4, streaming loads changed nothing (69.7).  24 blocks an SM (40 registers): with more registers 81.8 us, with 32 spilled ones 70.0; interleaved pairs need no more than 32.
//
// With a packed cache (PACKED) the block takes its keys and values in a pass of their own, by blocks of 32 elements: four lanes turn 8 elements each
// (a key's partner elements are read again, from L1) and pack them together.  16000 tokens as above, us, 8 bits and 4 bits with the bytes at a copy's rate in
// brackets: bf16 74 (54) and 74 (51), interleaved 76 and 75, fp32 92 (83) and 90 (80), interleaved 88 and 86.  As many blocks an SM as without:
// with 16 88, with 20 80 (half); 28 and more spill there (77).
//
// One block serves one token (blockIdx.x) and every gridDim.y-th group of its pieces.  A piece of a query or key head is
// 8 pairs (half layout: 8 elements and their 8 partners), 4 pairs (interleaved: 8 elements) or 8 elements that are copied;
// without VEC it is one pair or one element.  Pieces of the value heads are copied.
// Elements e .. e + 7 of a head at `src`, turned where they lie in the rotated part.
template <int XK, bool HALF, bool VEC>
__device__ __forceinline__ void turned8(const RopeArgs& a, const float2* cs, const void* x, long long src, int e, float (&y)[8]) {
    const int half = a.rot / 2;
    load8<XK>(x, src + e, y);
    if (e >= a.rot) return;
    if constexpr (VEC && HALF) {  // (pieces lie wholly in one half of the rotated part)
        const bool upper = e >= half;
        const int at = upper ? e - half : e;
        float z[8];
        load8<XK>(x, src + (upper ? at : e + half), z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 t = cs[at + j];
            y[j] = upper ? y[j] * t.x + z[j] * t.y : y[j] * t.x - z[j] * t.y;
        }
    } else if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = cs[e / 2 + j];
            const float u = y[2 * j], v = y[2 * j + 1];
            y[2 * j] = u * t.x - v * t.y, y[2 * j + 1] = v * t.x + u * t.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = e + j;
            if (i >= a.rot) continue;
            const bool second = HALF ? i >= half : i % 2;
            const int other = HALF ? (second ? i - half : i + half) : i ^ 1;
            const float2 t = cs[HALF ? (second ? other : i) : i / 2];
            const float z = load1<XK>(x, src + other);
            y[j] = second ? y[j] * t.x + z * t.y : y[j] * t.x - z * t.y;
        }
    }
}

template <int XK, bool HALF, bool VEC, int BITS>
__device__ __forceinline__ void pack_token(const RopeArgs& a, const float2* cs, long long tok, long long kslot, long long vslot) {
    const int per_head = a.dim / 8, half = a.kv_heads * per_head;
    for (int p = blockIdx.y * blockDim.x + threadIdx.x; p < 2 * half; p += blockDim.x * gridDim.y) {
        const bool is_v = p >= half;
        const int in = is_v ? p - half : p, h = in / per_head, e = (in - h * per_head) * 8;
        float y[8];
        if (is_v) load8<XK>(a.v, tok * a.v_token + h * a.v_head + e, y);
        else turned8<XK, HALF, VEC>(a, cs, a.k, tok * a.k_token + h * a.k_head, e, y);
        put8<BITS>(static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (is_v ? vslot + h * a.vc_head : kslot + h * a.kc_head), a.dim, e, y);
    }
}

template <int XK, bool HALF, bool VEC, bool PACKED>
__global__ void __launch_bounds__(ROPE_THREADS, HALF && VEC || PACKED && !VEC ? 24 : 32) rope_kernel(const RopeArgs a) {
    __shared__ float2 cs[128];
    pdl_launch_dependents();
    pdl_wait();
    const long long tok = blockIdx.x;
    const int half = a.rot / 2;
    const long long p = a.positions[tok];
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
        const unsigned long long turn = static_cast<unsigned long long>(p) * a.freqs[i];
        float s, c;
        // the signed upper word is the fraction of a turn in units of 2^-32; sincospif takes half turns
        sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c * a.mscale, s * a.mscale);
    }
    long long kslot = -1, vslot = -1;
    if (a.k_cache) {
        const long long slot = a.slots[tok];
        if (slot >= a.num_slots) {
            if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, ERR_BAD_INDEX);
        } else if (slot >= 0) {
            kslot = slot / a.page_size * a.kc_page + slot % a.page_size * a.kc_token;
            vslot = slot / a.page_size * a.vc_page + slot % a.page_size * a.vc_token;
        }
    }
    __syncthreads();
    if constexpr (PACKED) {
        if (kslot >= 0) {
            if (a.cache_kind == QGEMV_CACHE_Q4) pack_token<XK, HALF, VEC, 4>(a, cs, tok, kslot, vslot);
            else pack_token<XK, HALF, VEC, 8>(a, cs, tok, kslot, vslot);
        }
        __syncthreads();  // (keys that are turned in place have been read: one block takes the whole token then)
    }
    constexpr int W = VEC ? 8 : 1;
    const int turned = VEC && !HALF ? a.rot / 8 : half / W;  // pieces that turn, then those that are copied
    const int per_head = turned + (a.dim - a.rot) / W;
    const int copied = a.v && !PACKED ? a.dim / W : 0;  // pieces of a value head
    const int turning = a.heads + (PACKED && !a.k_out ? 0 : a.kv_heads);
    const int total = turning * per_head + a.kv_heads * copied;
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < total; i += blockDim.x * gridDim.y) {
        if (i >= turning * per_head) {
            const int j = i - turning * per_head;
            const int h = j / copied, e = j % copied * W;
            if (vslot < 0) continue;
            const long long src = tok * a.v_token + h * a.v_head + e, dst = vslot + h * a.vc_head + e;
            if constexpr (VEC) {
                float v[8];
                load8<XK>(a.v, src, v);
                store8(a.cache_kind, a.v_cache, dst, v);
            } else {
                store1(a.cache_kind, a.v_cache, dst, load1<XK>(a.v, src));
            }
            continue;
        }
        const int h = i / per_head, piece = i % per_head;
        const bool is_q = h < a.heads;
        const int hk = h - a.heads;
        const void* x = is_q ? a.q : a.k;
        const long long src = is_q ? tok * a.q_token + h * a.q_head : tok * a.k_token + hk * a.k_head;
        void* y = is_q ? a.q_out : a.k_out;
        const long long dst = is_q ? tok * a.q_out_token + h * a.q_out_head : tok * a.k_out_token + hk * a.k_out_head;
        const long long cdst = !PACKED && !is_q && kslot >= 0 ? kslot + hk * a.kc_head : -1;
        if (piece < turned) {
            if constexpr (VEC && HALF) {
                const int e = piece * 8;
                float u[8], v[8], r[8], s[8];
                load8<XK>(x, src + e, u);
                load8<XK>(x, src + e + half, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 t = cs[e + j];
                    r[j] = u[j] * t.x - v[j] * t.y;
                    s[j] = v[j] * t.x + u[j] * t.y;
                }
                if (y) store8(a.out_kind, y, dst + e, r), store8(a.out_kind, y, dst + e + half, s);
                if (cdst >= 0)
                    store8(a.cache_kind, a.k_cache, cdst + e, r), store8(a.cache_kind, a.k_cache, cdst + e + half, s);
            } else if constexpr (VEC) {
                const int e = piece * 8;
                float u[8], r[8];
                load8<XK>(x, src + e, u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 t = cs[e / 2 + j];
                    r[2 * j] = u[2 * j] * t.x - u[2 * j + 1] * t.y;
                    r[2 * j + 1] = u[2 * j + 1] * t.x + u[2 * j] * t.y;
                }
                if (y) store8(a.out_kind, y, dst + e, r);
                if (cdst >= 0) store8(a.cache_kind, a.k_cache, cdst + e, r);
            } else {
                const int e0 = HALF ? piece : 2 * piece, e1 = HALF ? piece + half : 2 * piece + 1;
                const float u = load1<XK>(x, src + e0), v = load1<XK>(x, src + e1);
                const float2 t = cs[piece];
                const float r = u * t.x - v * t.y, s = v * t.x + u * t.y;
                if (y) store1(a.out_kind, y, dst + e0, r), store1(a.out_kind, y, dst + e1, s);
                if (cdst >= 0)
                    store1(a.cache_kind, a.k_cache, cdst + e0, r), store1(a.cache_kind, a.k_cache, cdst + e1, s);
            }
        } else {
            const int e = a.rot + (piece - turned) * W;
            if constexpr (VEC) {
                float u[8];
                load8<XK>(x, src + e, u);
                if (y) store8(a.out_kind, y, dst + e, u);
                if (cdst >= 0) store8(a.cache_kind, a.k_cache, cdst + e, u);
            } else {
                const float u = load1<XK>(x, src + e);
                if (y) store1(a.out_kind, y, dst + e, u);
                if (cdst >= 0) store1(a.cache_kind, a.k_cache, cdst + e, u);
            }
        }
    }
}

template <int XK, bool PACKED>
static const void* pick(bool half, bool vec) {
    if (half) return vec ? (const void*)rope_kernel<XK, true, true, PACKED> : (const void*)rope_kernel<XK, true, false, PACKED>;
    return vec ? (const void*)rope_kernel<XK, false, true, PACKED> : (const void*)rope_kernel<XK, false, false, PACKED>;
}

const void* rope_kernel_ptr(int x_kind, bool half, bool vec, bool packed) {
    if (x_kind == ACT_F32) return packed ? pick<ACT_F32, true>(half, vec) : pick<ACT_F32, false>(half, vec);
    if (x_kind == ACT_BF16) return packed ? pick<ACT_BF16, true>(half, vec) : pick<ACT_BF16, false>(half, vec);
    return packed ? pick<ACT_F16, true>(half, vec) : pick<ACT_F16, false>(half, vec);
}

}  // namespace qg
