// Rotary positions of new tokens' queries and keys, with the write of keys and values into a paged cache.
//
// A pair (a, b) of a head turns by t = 2 pi frac(p F / 2^64): p F wraps in 64-bit integer arithmetic, its upper 32
// bits are the signed fraction of a turn, and sincospif takes them without a range reduction.  The kernel reads q, k and
// v once and writes each result once; it is bound by those bytes, and by the launch for a few tokens.
#include "common.cuh"
#include "internal.h"
#include "step.h"

namespace qg {

template <int XK>
__device__ __forceinline__ float load1(const void* x, long long i) {
    if constexpr (XK == ACT_F32) return static_cast<const float*>(x)[i];
    const uint16_t w = static_cast<const uint16_t*>(x)[i];
    if constexpr (XK == ACT_BF16) return __uint_as_float(static_cast<uint32_t>(w) << 16);
    return h2f(w);
}

// Eight consecutive values, 16-byte aligned, widened exactly.
template <int XK>
__device__ __forceinline__ void load8(const void* x, long long i, float (&v)[8]) {
    if constexpr (XK == ACT_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = XK == ACT_BF16 ? __uint_as_float(w[j] << 16) : h2f(w[j]);
            v[2 * j + 1] = XK == ACT_BF16 ? __uint_as_float(w[j] & 0xFFFF0000u) : h2f(w[j] >> 16);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(int kind, float a, float b) {
    uint32_t r;  // the first operand of the conversion goes to the upper half
    if (kind == ACT_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ void store1(int kind, void* y, long long i, float v) {
    if (kind == ACT_F32) static_cast<float*>(y)[i] = v;
    else static_cast<uint16_t*>(y)[i] = static_cast<uint16_t>(pack2(kind, v, v));
}

__device__ __forceinline__ void store8(int kind, void* y, long long i, const float (&v)[8]) {
    if (kind == ACT_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(y) + i);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + i) =
            make_uint4(pack2(kind, v[0], v[1]), pack2(kind, v[2], v[3]), pack2(kind, v[4], v[5]), pack2(kind, v[6], v[7]));
    }
}

// 16000 tokens of 32 and 8 heads of 128, bf16: 68.1 us, 5.78 TB/s, 85% of what a plain copy reaches.  Small blocks suit it: 64 threads 68.1 us,
// 128 69.3, 256 77.9, 448 (one piece a thread) 101; two pieces a thread on their way before the table is ready cost registers and
// took 89.4, streaming loads changed nothing (69.7).  24 blocks an SM (40 registers): with more registers 81.8 us, with 32 spilled ones 70.0; interleaved pairs need no more than 32.
//
// One block serves one token (blockIdx.x) and every gridDim.y-th group of its pieces.  A piece of a query or key head is
// 8 pairs (half layout: 8 elements and their 8 partners), 4 pairs (interleaved: 8 elements) or 8 elements that are copied;
// without VEC it is one pair or one element.  Pieces of the value heads are copied.
template <int XK, bool HALF, bool VEC>
__global__ void __launch_bounds__(ROPE_THREADS, HALF && VEC ? 24 : 32) rope_kernel(const RopeArgs a) {
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
    constexpr int W = VEC ? 8 : 1;
    const int turned = VEC && !HALF ? a.rot / 8 : half / W;  // pieces that turn, then those that are copied
    const int per_head = turned + (a.dim - a.rot) / W;
    const int copied = a.v ? a.dim / W : 0;  // pieces of a value head
    const int total = (a.heads + a.kv_heads) * per_head + a.kv_heads * copied;
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < total; i += blockDim.x * gridDim.y) {
        if (i >= (a.heads + a.kv_heads) * per_head) {
            const int j = i - (a.heads + a.kv_heads) * per_head;
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
        const long long cdst = !is_q && kslot >= 0 ? kslot + hk * a.kc_head : -1;
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

template <int XK>
static const void* pick(bool half, bool vec) {
    if (half) return vec ? (const void*)rope_kernel<XK, true, true> : (const void*)rope_kernel<XK, true, false>;
    return vec ? (const void*)rope_kernel<XK, false, true> : (const void*)rope_kernel<XK, false, false>;
}

const void* rope_kernel_ptr(int x_kind, bool half, bool vec) {
    if (x_kind == ACT_F32) return pick<ACT_F32>(half, vec);
    return x_kind == ACT_BF16 ? pick<ACT_BF16>(half, vec) : pick<ACT_F16>(half, vec);
}

}  // namespace qg
