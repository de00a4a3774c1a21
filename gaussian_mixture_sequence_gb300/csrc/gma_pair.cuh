// Unevaluated sums of two fp32 values, (x, y) for x + y with |y| at most half a step of x: about 48 bits
// on the fp32 pipe.  The FP64 pipe of this GPU takes 16 cycles for an instruction of any warp.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace gma {
namespace {

// Knuth's sum of two values and its error, and Dekker's for ordered ones.
__device__ __forceinline__ float2 two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}
__device__ __forceinline__ float2 quick_sum(float a, float b)   // |a| >= |b|
{
    const float s = __fadd_rn(a, b);
    return make_float2(s, __fsub_rn(b, __fsub_rn(s, a)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    const float2 s = two_sum(a.x, b.x);
    return quick_sum(s.x, __fadd_rn(s.y, __fadd_rn(a.y, b.y)));
}

// Logarithms and exponentials to about 2^-30, as sums of two fp32 values.
// Cody and Waite's split: ln 2 = hi + lo, hi = 355 / 512 of 9 bits, so that n hi is exact.
constexpr float kLn2Hi = 0.693359375f, kLn2Lo = -2.12194440054690581e-4f;

__device__ __forceinline__ float2 div2(float2 a, float2 b)
{
    const float q = a.x / b.x;
    const float r = __fmaf_rn(-q, b.x, a.x);
    return quick_sum(q, (r + __fmaf_rn(-q, b.y, a.y)) / b.x);
}

// 2 atanh z = 2 (z + z^3 / 3 + z^5 / 5 + ...), |z| <= 1/3: the terms past the first are at most a
// 27th of it, so fp32 suffices for them.
__device__ __forceinline__ float2 atanh2(float2 z)
{
    const float s = z.x * z.x;
    float p = 1.f / 19.f;
    p = fmaf(p, s, 1.f / 17.f);
    p = fmaf(p, s, 1.f / 15.f);
    p = fmaf(p, s, 1.f / 13.f);
    p = fmaf(p, s, 1.f / 11.f);
    p = fmaf(p, s, 1.f / 9.f);
    p = fmaf(p, s, 1.f / 7.f);
    p = fmaf(p, s, 1.f / 5.f);
    p = fmaf(p, s, 1.f / 3.f);
    const float2 r = quick_sum(z.x, fmaf(p, s * z.x, z.y));
    return make_float2(2.f * r.x, 2.f * r.y);
}

// exp t for t <= 0 (0 below the fp32 range): t = n ln 2 + f, |f| <= ln 2 / 2, and the series of exp f,
// its terms past the second in fp32.
__device__ __forceinline__ float2 exp2v(float t)
{
    const float n = rintf(fmaxf(t, -126.f) * 1.4426950408889634f);
    const float2 f = two_sum(__fmaf_rn(-n, kLn2Hi, t), -n * kLn2Lo);   // the first part is exact
    float p = 1.f / 40320.f;
    p = fmaf(p, f.x, 1.f / 5040.f);
    p = fmaf(p, f.x, 1.f / 720.f);
    p = fmaf(p, f.x, 1.f / 120.f);
    p = fmaf(p, f.x, 1.f / 24.f);
    p = fmaf(p, f.x, 1.f / 6.f);
    const float h = 0.5f * f.x * f.x, hl = __fmaf_rn(0.5f * f.x, f.x, -h);
    float2 r = two_sum(f.x, h);
    r.y += f.y + (hl + fmaf(f.x, f.y, p * f.x * f.x * f.x));
    r = add2(make_float2(1.f, 0.f), quick_sum(r.x, r.y));
    const float sc = __uint_as_float((uint32_t)(max((int)n, -126) + 127) << 23);
    return t < -126.f * 0.69f ? make_float2(expf(t), 0.f) : make_float2(r.x * sc, r.y * sc);
}

// log v, v > 0: v = 2^k m with m in [1/sqrt 2, sqrt 2], log m = 2 atanh((m - 1) / (m + 1)).
__device__ __forceinline__ float2 log2v(float2 v)
{
    const uint32_t u = __float_as_uint(v.x) - 0x3f3504f3u;   // relative to 1/sqrt 2
    const int k = (int)u >> 23;
    const float sc = __uint_as_float((uint32_t)(127 - k) << 23);
    const float2 m = make_float2(v.x * sc, v.y * sc);
    const float2 l = atanh2(div2(add2(m, make_float2(-1.f, 0.f)), add2(m, make_float2(1.f, 0.f))));
    return add2(two_sum((float)k * kLn2Hi, (float)k * kLn2Lo), l);
}

} // namespace
} // namespace gma
