// f8.cuh -- e4m3 codes with a scale for each block: the quantizer's arithmetic.
#pragma once

#include <cuda_fp8.h>

#include "actq.cuh"
#include "layer.cuh"

namespace w4a8 {

constexpr int kF8Block = 128;  // values of K (and, of weights, rows) that share a scale

// Two codes, the first in the low byte: nearest, ties to even, at most 448.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
    return d;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | e4m3x2(c, d) << 16;
}

__device__ __forceinline__ float f8_scale(float amax) { return __fmul_rn(amax, 1.f / 448.f); }

// The code of the quotient x / s itself.  Rounding it to fp32 first can only make
// a difference where the rounded quotient is a tie between two codes and the
// exact one is not: the remainder, which an fma gives exactly, then tells the side.  (At a tie it is a multiple of
// 2^-10 units in the last place of s: small scales and their values, of at most 448 s, go up together, so that it
// is no less than the smallest number.)
static __device__ __noinline__ uint32_t f8_codes4_exact(float4 v, float s) {
    if (s == 0.f) return 0u;
    if (s < 0x1p-64f) {
        constexpr float kUp = 0x1p64f;
        s *= kUp, v.x *= kUp, v.y *= kUp, v.z *= kUp, v.w *= kUp;
    }
    const float x[4] = {v.x, v.y, v.z, v.w};
    float q[4];
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float d = __fdiv_rn(x[k], s);
        // a tie lies half a step from a code: steps of 2^-9 below 2^-6, of 2^-3 relative above
        const float t = fabsf(d) * 1024.f;
        const bool tie = fabsf(d) < 0x1p-6f ? t == rintf(t) && ((int)t & 1) : (__float_as_uint(d) & 0xFFFFFu) == 0x80000u;
        const float rem = fmaf(-d, s, x[k]);  // of x's sign: the exact quotient is larger in magnitude
        q[k] = d;
        if (tie && rem != 0.f && isfinite(rem))
            q[k] = __uint_as_float(__float_as_uint(d) + (((rem < 0.f) == (d < 0.f)) ? 1u : 0xFFFFFFFFu));
    }
    return e4m3x4(q[0], q[1], q[2], q[3]);
}
// The same with 1 / s bracketed by lo and hi (quant_bracket): where both products
// round to one code that is the quotient's, which lies between them.  Needs a normal, finite s.
__device__ __forceinline__ uint32_t f8_codes4(float4 v, float s, float lo, float hi) {
    if (!(s >= 0x1p-100f && s < INFINITY)) return f8_codes4_exact(v, s);
    const uint32_t a = e4m3x4(v.x * lo, v.y * lo, v.z * lo, v.w * lo);
    const uint32_t b = e4m3x4(v.x * hi, v.y * hi, v.z * hi, v.w * hi);
    return a == b ? a : f8_codes4_exact(v, s);
}

// Eight values of a row as they are in memory.
template <typename T>
struct Eight;
template <>
struct Eight<__half> {
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    __device__ __forceinline__ void load(const __half* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float4& a, float4& b) const {
        const __half2* h = reinterpret_cast<const __half2*>(&u);
        const float2 p = __half22float2(h[0]), q = __half22float2(h[1]), s = __half22float2(h[2]), t = __half22float2(h[3]);
        a = make_float4(p.x, p.y, q.x, q.y);
        b = make_float4(s.x, s.y, t.x, t.y);
    }
};
template <>
struct Eight<float> {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void load(const float* p) { x = load4(p), y = load4(p + 4); }
    __device__ __forceinline__ void get(float4& a, float4& b) const { a = x, b = y; }
};

// The scale of a block of 128 values, 8 in each of sixteen lanes side by side.
__device__ __forceinline__ float f8_row_scale(const float4& a, const float4& b) {
    float top = max_nan(absmax4_nan(a), absmax4_nan(b));
    #pragma unroll
    for (int o = 8; o >= 1; o /= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    return f8_scale(top);
}

}  // namespace w4a8
