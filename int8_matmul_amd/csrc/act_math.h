// Activations of the feed-forward entry points and their slopes, in fp32.
//
//   none      z                     relu       max(z, 0)
//   silu      z s(z)                gelu_tanh  z s(2 sqrt(2/pi) (z + 0.044715 z^3))
//   gelu      z P(z), P the integral of the normal density
// with s(x) = 1 / (1 + exp(-x)).  gelu_tanh is the usual
// (z/2) (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))), as (1 + tanh(y)) / 2 = s(2y);
// so silu and gelu_tanh are one form with an odd cubic in the exponent, and
// none and relu one form with a lower bound.  A call picks one of three code
// paths by a uniform branch.
//
// The normal integral of a negative argument is
//   P(-x) = exp(-x^2 / 2) Q(1 / (1 + 0.3 x)),    x >= 0,
// Q a polynomial of degree 8 without constant term fitted to
// erfcx(x / sqrt(2)) / 2 on [0, 14] for the smallest largest relative error
// (1.7e-7; 4.4e-7 as evaluated in fp32), so the tail keeps its relative
// accuracy; exp, 1/x: one unit in the last place each, plus |x^2/2| units
// from the rounded exponent.  Results are rounded to fp16 next (2^-11), which
// these errors (below 2^-18 for |z| <= 7) do not reach.
#pragma once

#include <hip/hip_runtime.h>

#include "li8_internal.h"

namespace li8 {

// s(x) with exp(-x) = 2^(z (c1 + c3 z^2)): 0 and 1 at the ends, infinities among
// them, NaN for a NaN only.  (z^2 stops at the largest finite number: with silu's c3 =
// 0 an infinite one would be 0 times infinity, from |z| = 1.85e19 on.)
__device__ __forceinline__ float act_sigmoid(float z, const ActParams &p)
{
    const float zz = __builtin_fminf(z * z, 3.402823466e38f);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * (p.c1 + p.c3 * zz)));
}

// The normal integral at z, and e = exp(-z^2 / 2).
__device__ __forceinline__ float act_normal(float z, float &e)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, __builtin_fabsf(z), 1.0f));
    float q = 0.03567490726709366f;
    q = fmaf(q, t, -0.15720361471176147f);
    q = fmaf(q, t, 0.20635436475276947f);
    q = fmaf(q, t, -0.05368437245488167f);
    q = fmaf(q, t, 0.12856197357177734f);
    q = fmaf(q, t, 0.09991339594125748f);
    q = fmaf(q, t, 0.12075397372245789f);
    q = fmaf(q, t, 0.11962930113077164f);
    e = __builtin_amdgcn_exp2f(-0.7213475204444817f * (z * z));
    const float tail = e * (q * t);
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int KIND>
__device__ __forceinline__ float act_value(float z, const ActParams &p)
{
    if constexpr (KIND == 0) {
        return z <= p.lo ? p.lo : z;   // (a NaN stays; no lower bound: lo is one)
    } else if constexpr (KIND == 1) {
        return z * act_sigmoid(z, p);
    } else {
        float e;
        return z * act_normal(z, e);
    }
}

// Value and slope at z.  The slope of relu at 0 is 0.  Kind 1 with
// x = z (a1 + a3 z^2) is z s(x), whose slope is s + z s (1 - s) x'; far out
// s (1 - s) is 0 and x' large, infinite or NaN, so the product is taken as zero
// there rather than 0 times infinity.
template <int KIND>
__device__ __forceinline__ void act_value_slope(float z, const ActParams &p, float &value, float &slope)
{
    if constexpr (KIND == 0) {
        const bool low = z <= p.lo;
        value = low ? p.lo : z;
        slope = low ? 0.0f : 1.0f;
    } else if constexpr (KIND == 1) {
        const float ln2 = 0.6931471805599453f;
        const float s = act_sigmoid(z, p), r = s * (1.0f - s);
        const float x1 = -ln2 * (p.c1 + 3.0f * p.c3 * (z * z));
        value = z * s;
        slope = r == 0.0f ? s : s + z * r * x1;
    } else {
        float e;
        const float n = act_normal(z, e);
        value = z * n;
        slope = e == 0.0f ? n : n + 0.3989422804014327f * (z * e);
    }
}

} // namespace li8
