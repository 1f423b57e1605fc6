// rotary.cuh -- the rotations of rotary positions: cos and sin of p t 2 pi to about
// 2^-33, for t in turns per position.
//
// The angle.  t is a 64-bit fixed-point fraction of a turn, so p t modulo one turn
// is the low 64 bits of an integer product: exact for every position, where a
// 32-bit p f has lost 2^-24 p radians (0.06 at a million).
//
// cos and sin.  The fraction is the nearest of 64 points of the circle, whose cos
// and sin are tabulated in two floats each, and a rest of at most pi / 64, for
// which sin d = d - d^3 / 6 + d^5 / 120, cos d - 1 = -d^2 / 2 + d^4 / 24 - d^6 / 720
// (next terms 2^-43 and 2^-50).  The sum theorem is evaluated with the products of
// leading parts and their sum kept exactly: what is left is the rounding of terms
// below 2^-9.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace ddg {
namespace {

// cos and sin of k / 64 turns, each as a float and what it leaves
__device__ const float4 kTurnPoints[64] = {
    {0x1.0000000000000p+0f, 0.0f, 0.0f, 0.0f},
    {0x1.fd88da0000000p-1f, 0x1.e892920000000p-28f, 0x1.917a6c0000000p-4f, -0x1.eb25ea0000000p-31f},
    {0x1.f6297c0000000p-1f, 0x1.feeb960000000p-26f, 0x1.8f8b840000000p-3f, -0x1.cb2cfa0000000p-30f},
    {0x1.e9f4160000000p-1f, -0x1.273a440000000p-26f, 0x1.2940620000000p-2f, 0x1.dab3e00000000p-27f},
    {0x1.d906bc0000000p-1f, 0x1.e651a80000000p-26f, 0x1.87de2a0000000p-2f, 0x1.abaa580000000p-28f},
    {0x1.c38b300000000p-1f, -0x1.cfe84a0000000p-26f, 0x1.e2b5d40000000p-2f, -0x1.fe42720000000p-28f},
    {0x1.a9b6620000000p-1f, 0x1.21d4340000000p-26f, 0x1.1c73b40000000p-1f, -0x1.9465ce0000000p-27f},
    {0x1.8bc8060000000p-1f, 0x1.62a2e80000000p-26f, 0x1.44cf320000000p-1f, 0x1.4247760000000p-27f},
    {0x1.6a09e60000000p-1f, 0x1.9fcef40000000p-27f, 0x1.6a09e60000000p-1f, 0x1.9fcef40000000p-27f},
    {0x1.44cf320000000p-1f, 0x1.4247760000000p-27f, 0x1.8bc8060000000p-1f, 0x1.62a2e80000000p-26f},
    {0x1.1c73b40000000p-1f, -0x1.9465ce0000000p-27f, 0x1.a9b6620000000p-1f, 0x1.21d4340000000p-26f},
    {0x1.e2b5d40000000p-2f, -0x1.fe42720000000p-28f, 0x1.c38b300000000p-1f, -0x1.cfe84a0000000p-26f},
    {0x1.87de2a0000000p-2f, 0x1.abaa580000000p-28f, 0x1.d906bc0000000p-1f, 0x1.e651a80000000p-26f},
    {0x1.2940620000000p-2f, 0x1.dab3e00000000p-27f, 0x1.e9f4160000000p-1f, -0x1.273a440000000p-26f},
    {0x1.8f8b840000000p-3f, -0x1.cb2cfa0000000p-30f, 0x1.f6297c0000000p-1f, 0x1.feeb960000000p-26f},
    {0x1.917a6c0000000p-4f, -0x1.eb25ea0000000p-31f, 0x1.fd88da0000000p-1f, 0x1.e892920000000p-28f},
    {0.0f, 0.0f, 0x1.0000000000000p+0f, 0.0f},
    {-0x1.917a6c0000000p-4f, 0x1.eb25ea0000000p-31f, 0x1.fd88da0000000p-1f, 0x1.e892920000000p-28f},
    {-0x1.8f8b840000000p-3f, 0x1.cb2cfa0000000p-30f, 0x1.f6297c0000000p-1f, 0x1.feeb960000000p-26f},
    {-0x1.2940620000000p-2f, -0x1.dab3e00000000p-27f, 0x1.e9f4160000000p-1f, -0x1.273a440000000p-26f},
    {-0x1.87de2a0000000p-2f, -0x1.abaa580000000p-28f, 0x1.d906bc0000000p-1f, 0x1.e651a80000000p-26f},
    {-0x1.e2b5d40000000p-2f, 0x1.fe42720000000p-28f, 0x1.c38b300000000p-1f, -0x1.cfe84a0000000p-26f},
    {-0x1.1c73b40000000p-1f, 0x1.9465ce0000000p-27f, 0x1.a9b6620000000p-1f, 0x1.21d4340000000p-26f},
    {-0x1.44cf320000000p-1f, -0x1.4247760000000p-27f, 0x1.8bc8060000000p-1f, 0x1.62a2e80000000p-26f},
    {-0x1.6a09e60000000p-1f, -0x1.9fcef40000000p-27f, 0x1.6a09e60000000p-1f, 0x1.9fcef40000000p-27f},
    {-0x1.8bc8060000000p-1f, -0x1.62a2e80000000p-26f, 0x1.44cf320000000p-1f, 0x1.4247760000000p-27f},
    {-0x1.a9b6620000000p-1f, -0x1.21d4340000000p-26f, 0x1.1c73b40000000p-1f, -0x1.9465ce0000000p-27f},
    {-0x1.c38b300000000p-1f, 0x1.cfe84a0000000p-26f, 0x1.e2b5d40000000p-2f, -0x1.fe42720000000p-28f},
    {-0x1.d906bc0000000p-1f, -0x1.e651a80000000p-26f, 0x1.87de2a0000000p-2f, 0x1.abaa580000000p-28f},
    {-0x1.e9f4160000000p-1f, 0x1.273a440000000p-26f, 0x1.2940620000000p-2f, 0x1.dab3e00000000p-27f},
    {-0x1.f6297c0000000p-1f, -0x1.feeb960000000p-26f, 0x1.8f8b840000000p-3f, -0x1.cb2cfa0000000p-30f},
    {-0x1.fd88da0000000p-1f, -0x1.e892920000000p-28f, 0x1.917a6c0000000p-4f, -0x1.eb25ea0000000p-31f},
    {-0x1.0000000000000p+0f, 0.0f, 0.0f, 0.0f},
    {-0x1.fd88da0000000p-1f, -0x1.e892920000000p-28f, -0x1.917a6c0000000p-4f, 0x1.eb25ea0000000p-31f},
    {-0x1.f6297c0000000p-1f, -0x1.feeb960000000p-26f, -0x1.8f8b840000000p-3f, 0x1.cb2cfa0000000p-30f},
    {-0x1.e9f4160000000p-1f, 0x1.273a440000000p-26f, -0x1.2940620000000p-2f, -0x1.dab3e00000000p-27f},
    {-0x1.d906bc0000000p-1f, -0x1.e651a80000000p-26f, -0x1.87de2a0000000p-2f, -0x1.abaa580000000p-28f},
    {-0x1.c38b300000000p-1f, 0x1.cfe84a0000000p-26f, -0x1.e2b5d40000000p-2f, 0x1.fe42720000000p-28f},
    {-0x1.a9b6620000000p-1f, -0x1.21d4340000000p-26f, -0x1.1c73b40000000p-1f, 0x1.9465ce0000000p-27f},
    {-0x1.8bc8060000000p-1f, -0x1.62a2e80000000p-26f, -0x1.44cf320000000p-1f, -0x1.4247760000000p-27f},
    {-0x1.6a09e60000000p-1f, -0x1.9fcef40000000p-27f, -0x1.6a09e60000000p-1f, -0x1.9fcef40000000p-27f},
    {-0x1.44cf320000000p-1f, -0x1.4247760000000p-27f, -0x1.8bc8060000000p-1f, -0x1.62a2e80000000p-26f},
    {-0x1.1c73b40000000p-1f, 0x1.9465ce0000000p-27f, -0x1.a9b6620000000p-1f, -0x1.21d4340000000p-26f},
    {-0x1.e2b5d40000000p-2f, 0x1.fe42720000000p-28f, -0x1.c38b300000000p-1f, 0x1.cfe84a0000000p-26f},
    {-0x1.87de2a0000000p-2f, -0x1.abaa580000000p-28f, -0x1.d906bc0000000p-1f, -0x1.e651a80000000p-26f},
    {-0x1.2940620000000p-2f, -0x1.dab3e00000000p-27f, -0x1.e9f4160000000p-1f, 0x1.273a440000000p-26f},
    {-0x1.8f8b840000000p-3f, 0x1.cb2cfa0000000p-30f, -0x1.f6297c0000000p-1f, -0x1.feeb960000000p-26f},
    {-0x1.917a6c0000000p-4f, 0x1.eb25ea0000000p-31f, -0x1.fd88da0000000p-1f, -0x1.e892920000000p-28f},
    {0.0f, 0.0f, -0x1.0000000000000p+0f, 0.0f},
    {0x1.917a6c0000000p-4f, -0x1.eb25ea0000000p-31f, -0x1.fd88da0000000p-1f, -0x1.e892920000000p-28f},
    {0x1.8f8b840000000p-3f, -0x1.cb2cfa0000000p-30f, -0x1.f6297c0000000p-1f, -0x1.feeb960000000p-26f},
    {0x1.2940620000000p-2f, 0x1.dab3e00000000p-27f, -0x1.e9f4160000000p-1f, 0x1.273a440000000p-26f},
    {0x1.87de2a0000000p-2f, 0x1.abaa580000000p-28f, -0x1.d906bc0000000p-1f, -0x1.e651a80000000p-26f},
    {0x1.e2b5d40000000p-2f, -0x1.fe42720000000p-28f, -0x1.c38b300000000p-1f, 0x1.cfe84a0000000p-26f},
    {0x1.1c73b40000000p-1f, -0x1.9465ce0000000p-27f, -0x1.a9b6620000000p-1f, -0x1.21d4340000000p-26f},
    {0x1.44cf320000000p-1f, 0x1.4247760000000p-27f, -0x1.8bc8060000000p-1f, -0x1.62a2e80000000p-26f},
    {0x1.6a09e60000000p-1f, 0x1.9fcef40000000p-27f, -0x1.6a09e60000000p-1f, -0x1.9fcef40000000p-27f},
    {0x1.8bc8060000000p-1f, 0x1.62a2e80000000p-26f, -0x1.44cf320000000p-1f, -0x1.4247760000000p-27f},
    {0x1.a9b6620000000p-1f, 0x1.21d4340000000p-26f, -0x1.1c73b40000000p-1f, 0x1.9465ce0000000p-27f},
    {0x1.c38b300000000p-1f, -0x1.cfe84a0000000p-26f, -0x1.e2b5d40000000p-2f, 0x1.fe42720000000p-28f},
    {0x1.d906bc0000000p-1f, 0x1.e651a80000000p-26f, -0x1.87de2a0000000p-2f, -0x1.abaa580000000p-28f},
    {0x1.e9f4160000000p-1f, -0x1.273a440000000p-26f, -0x1.2940620000000p-2f, -0x1.dab3e00000000p-27f},
    {0x1.f6297c0000000p-1f, 0x1.feeb960000000p-26f, -0x1.8f8b840000000p-3f, 0x1.cb2cfa0000000p-30f},
    {0x1.fd88da0000000p-1f, 0x1.e892920000000p-28f, -0x1.917a6c0000000p-4f, 0x1.eb25ea0000000p-31f},
};

// c + cl = cos, s + sl = sin of `fraction` / 2^64 turns.
struct Turn {
    float c, cl, s, sl;
};

// a + b = sum + the returned rest, for |a| >= |b| or a = 0.
__device__ __forceinline__ float quick_sum(float& a, float b) {
    const float s = a + b, rest = b - (s - a);
    a = s;
    return rest;
}

__device__ __forceinline__ Turn turn_of(uint64_t fraction) {
    const uint64_t point = (fraction + (1ULL << 57)) >> 58;
    const int64_t rest = (int64_t)(fraction - (point << 58));  // below 2^57 in magnitude
    const float hi = (float)(int32_t)(rest >> 34);             // at most 2^23: exact
    const float lo = (float)(uint32_t)(((uint64_t)rest & ((1ULL << 34) - 1)) >> 2);
    const float unit = 0x1.921fb6p-28f, unit_rest = -0x1.777a5cp-53f;  // 2 pi 2^-30
    const float d = hi * unit;
    const float dl = fmaf(hi, unit, -d) + fmaf(hi, unit_rest, lo * 0x1.921fb6p-60f);
    const float dd = d * d;
    const float w = fmaf(d * dd, fmaf(dd, 1.0f / 120.0f, -1.0f / 6.0f), dl);                       // sin d - d
    const float u = dd * fmaf(dd, fmaf(dd, -1.0f / 720.0f, 1.0f / 24.0f), -0.5f) - d * dl;         // cos d - 1
    const float4 t = __ldg(&kTurnPoints[point & 63]);
    Turn r;
    // cos: t.x + t.x u - t.z (d + w);  sin: t.z + t.z u + t.x (d + w)
    const float pc = t.z * d, pcl = fmaf(t.z, d, -pc);
    const float ps = t.x * d, psl = fmaf(t.x, d, -ps);
    float c = t.x, cb = -pc, s = t.z, sb = ps;
    if (fabsf(c) < fabsf(cb)) { const float x = c; c = cb; cb = x; }
    if (fabsf(s) < fabsf(sb)) { const float x = s; s = sb; sb = x; }
    const float ce = quick_sum(c, cb), se = quick_sum(s, sb);
    const float ct = ce - pcl + fmaf(t.x, u, t.y) - fmaf(t.z, w, t.w * d);
    const float st = se + psl + fmaf(t.z, u, t.w) + fmaf(t.x, w, t.y * d);
    r.c = c;
    r.cl = quick_sum(r.c, ct);
    r.s = s;
    r.sl = quick_sum(r.s, st);
    return r;
}

// Times m + ml, a factor in two floats.
__device__ __forceinline__ Turn times(const Turn& t, float m, float ml) {
    if (m == 1.0f && ml == 0.0f) return t;
    Turn r;
    r.c = t.c * m;
    r.cl = fmaf(t.c, m, -r.c) + fmaf(t.cl, m, t.c * ml);
    r.s = t.s * m;
    r.sl = fmaf(t.s, m, -r.s) + fmaf(t.sl, m, t.s * ml);
    return r;
}

// a b + c d, rounded once but for about 2^-8 of a last place: both products and
// their sum are kept exactly.  Where that is not finite, the plain sum.
__device__ __forceinline__ float sum_of_products(float a, float b, float bl, float c, float d, float dl) {
    const float p = a * b, pe = fmaf(a, b, -p), q = c * d, qe = fmaf(c, d, -q);
    const float s = p + q, t = s - p;
    const float e = (p - (s - t)) + (q - t);
    const float y = s + (e + (pe + qe) + fmaf(a, bl, c * dl));
    return fabsf(s) <= 0x1p127f ? y : s;
}

}  // namespace
}  // namespace ddg
