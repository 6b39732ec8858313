// Rows of a packed cache: codes of 4 or 8 bits, a step and a base in fp16 for every 32 of them (the layout is in qgemv.h).
#pragma once
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

// Eight consecutive values, 16-byte aligned, as they lie there; widened exactly.
template <int XK>
struct Raw8 {
    uint4 u[XK == ACT_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* x, long long i) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + i * (XK == ACT_F32 ? 4 : 2));
        u[0] = p[0];
        if constexpr (XK == ACT_F32) u[1] = p[1];
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        if constexpr (XK == ACT_F32) {
            v[0] = __uint_as_float(u[0].x), v[1] = __uint_as_float(u[0].y), v[2] = __uint_as_float(u[0].z), v[3] = __uint_as_float(u[0].w);
            v[4] = __uint_as_float(u[1].x), v[5] = __uint_as_float(u[1].y), v[6] = __uint_as_float(u[1].z), v[7] = __uint_as_float(u[1].w);
        } else {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = XK == ACT_BF16 ? __uint_as_float(w[j] << 16) : h2f(w[j]);
                v[2 * j + 1] = XK == ACT_BF16 ? __uint_as_float(w[j] & 0xFFFF0000u) : h2f(w[j] >> 16);
            }
        }
    }
};
template <int XK>
__device__ __forceinline__ void load8(const void* x, long long i, float (&v)[8]) {
    Raw8<XK> r;
    r.load(x, i);
    r.values(v);
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

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float min_or_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The step and base of a block by its least and largest value (NaN where one is).
//
// The base is rounded down and the step up, so that every value lies within the codes: none is cut off by more than the rounding of
// the fp32 arithmetic.  The product with 1 / d stands for the quotient (one instruction an element instead of eight); it moves a code by
// one only where the value lies within 2^-14 steps of the middle of two.
template <int BITS>
struct BlockScale {
    static constexpr float TOP = (1 << BITS) - 1;
    float m, rate;
    uint16_t d16, m16;
    __device__ __forceinline__ BlockScale(float lo, float hi) {
        const bool nan = hi != hi;
        lo = fminf(fmaxf(lo, -65504.f), 65504.f), hi = fminf(fmaxf(hi, -65504.f), 65504.f);
        const __half mh = __float2half_rd(lo);
        m = __half2float(mh);
        __half d = __float2half_ru(__fdiv_rn(__fsub_rn(hi, m), TOP));
        if (nan) d = __ushort_as_half(0);
        const float df = __half2float(d);
        rate = df == 0.f ? 0.f : __frcp_rn(df);
        d16 = __half_as_ushort(d), m16 = nan ? 0x7E00 : __half_as_ushort(mh);
    }
    // at element e of a row
    __device__ __forceinline__ void put(uint8_t* row, int dim, int e) const {
        uint16_t* scale = reinterpret_cast<uint16_t*>(row + dim * BITS / 8);
        scale[e / 32] = d16, scale[dim / 32 + e / 32] = m16;
    }
};

__device__ __forceinline__ void ends8(const float (&x)[8], float& lo, float& hi) {
    lo = hi = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) lo = fminf(lo, x[j]), hi = max_or_nan(hi, x[j]);
}

// The codes of 8 values, for element e.  Values beyond +-65504 need no clamp of their own: the block's ends are clamped, and the codes
// to 0 .. L.  A code comes out of the low bits of t + 1.5 2^23, which rounds t to a whole number, ties to even; the
// sum of those words times powers of two packs the codes, with the words' upper bits taken off at once.
template <int BITS>
__device__ __forceinline__ void codes8(uint8_t* row, int e, const float (&x)[8], float m, float rate) {
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = fminf(fmaxf(__fmul_rn(__fsub_rn(x[j], m), rate), 0.f), BlockScale<BITS>::TOP);
        c[j] = __float_as_uint(__fadd_rn(t, 12582912.f));  // 0x4B400000 + code
    }
    constexpr uint32_t BIAS = 0x4B400000u;
    if constexpr (BITS == 4) {
        uint32_t w = 0u - BIAS * 0x11111111u;
#pragma unroll
        for (int j = 0; j < 8; ++j) w += c[j] * (1u << (4 * j));
        *reinterpret_cast<uint32_t*>(row + e / 2) = w;
    } else {
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[j] = c[4 * j] + c[4 * j + 1] * (1u << 8) + c[4 * j + 2] * (1u << 16) + c[4 * j + 3] * (1u << 24) - BIAS * 0x01010101u;
        *reinterpret_cast<uint2*>(row + e) = make_uint2(w[0], w[1]);
    }
}

// Elements e .. e + 7 (e a multiple of 8) of a row of `dim`.  Four consecutive lanes, the first at a multiple of 4, hold a block: they
// find its least and largest value together, and each writes its own codes.  All four call this, with the same `row`.
template <int BITS>
__device__ __forceinline__ void put8(uint8_t* row, int dim, int e, const float (&x)[8]) {
    const unsigned team = 0xFu << (threadIdx.x & 28);
    float lo, hi;
    ends8(x, lo, hi);
#pragma unroll
    for (int o = 1; o < 4; o *= 2) {
        lo = fminf(lo, __shfl_xor_sync(team, lo, o));
        hi = max_or_nan(hi, __shfl_xor_sync(team, hi, o));
    }
    const BlockScale<BITS> s(lo, hi);
    codes8<BITS>(row, e, x, s.m, s.rate);
    if (e % 32 == 0) s.put(row, dim, e);
}

// Elements e .. e + 7 of a row as they lie there, and their values.  The places of the codes, the step and the base within a row are a thread's own.
template <int BITS>
struct Packed8 {
    uint32_t w[BITS / 4];
    uint16_t d, m;
    // codes, step: those of the first row, `place` bytes before this one; the base lies `base` bytes after the step
    __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* step, int base, long long place) {
        if constexpr (BITS == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(codes + place);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(codes + place);
            w[0] = u.x, w[1] = u.y;
        }
        const uint8_t* const s = step + place;
        d = *reinterpret_cast<const uint16_t*>(s), m = *reinterpret_cast<const uint16_t*>(s + base);
    }
    // A code becomes a float where it stands: its bits, anywhere below bit 20, in the mantissa of 2^23, which is taken off again (exactly); the power of
    // 16 by which it stands too high is taken off the step.  (d c is exact in fp32, so that the last step alone rounds.)
    __device__ __forceinline__ void values(float (&x)[8]) const {
        const float df = h2f(d), mf = h2f(m);
        constexpr uint32_t TWO23 = 0x4B000000u;
        if constexpr (BITS == 4) {
            const float ds[4] = {df, df * 0.0625f, df * 0.00390625f, df * 0.000244140625f};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = __fmaf_rn(ds[j & 3], __uint_as_float(((j < 4 ? w[0] : w[0] >> 16) & 0xFu << (4 * (j & 3))) | TWO23) - 8388608.f, mf);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __fmaf_rn(df, __uint_as_float(__byte_perm(w[j / 4], TWO23, 0x7650 | (j & 3))) - 8388608.f, mf);
        }
    }
};

}  // namespace qg
