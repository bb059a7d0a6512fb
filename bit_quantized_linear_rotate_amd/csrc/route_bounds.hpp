// How far the fp32 values that routing by scores compares may be from the true ones, for
// the device code and for a check on the host.  u = 2^-24 is half a last place of 1, V
// the largest of all scores and magnitudes of choice values.
//
// Each operation is off by u of its result, but exp(x) by (1.5 |x| + 2) u (two roundings
// of its argument in base 2, and the power) and the hardware's reciprocal by 2 u.
//   Sigmoid: s = 1 / (1 + exp(-l)) is off by s ((1 - s) (1.5 |l| + 2) + 3) u.  With the
// largest logit at 0 or above that is at most 4.05 u V, else at most (5 + 1.5 |top|) u V
// (it falls with l there).  A bias' sum adds u V, and a difference has two such values:
// (12 + 3 |top|) u V, where 16 + 3 |top| is taken.
//   Softmax: exp(l - top) is off by (2.5 |l - top| + 2) u of itself, 2.05 u of the largest
// at most; the sum by h + nv + 5 (the terms' errors by weight, h <= 19.3 for 1024 experts,
// 10.7 for 32; the additions) and its reciprocal by 1, the same for all scores; a product
// and a bias by 1 each: (nv + 14.1 + h) u V in a difference, where 2 nv + 32 is taken.
//   Sums of two: twice that, and a rounding of each sum, of up to 2 V: 4 u V more.
#pragma once

#include <cmath>
#include <cstdint>

#if defined(__HIPCC__)
#define W4A4_ROUTE_HD __host__ __device__
#else
#define W4A4_ROUTE_HD
#endif

namespace w4a4 {

// Of the difference of two choice values (nv: scores that a lane adds up, top: the
// largest logit).  2^-119: what the hardware's reciprocal rounds to zero.
W4A4_ROUTE_HD inline float route_error(bool sigmoid, int nv, float top, float V)
{
    return fmaf(V, (sigmoid ? 8.0f - 1.5f * fminf(top, 0.0f) : 16.0f + (float)nv) * 0x1p-23f, 0x1p-119f);
}

// Of the difference of two sums of two choice values.
W4A4_ROUTE_HD inline float route_sum_error(float error, float V) { return fmaf(V, 0x1p-22f, 2.0f * error); }

// Values in fixed point, in 2^(32 - bits) - 512 units over their range: two of them this
// many units or less apart may be in either order.  Beside their error, the difference
// from the smallest and the product are off by u of up to 2^(32 - bits) units each, and
// the cut by less than 1; this for both, and one more for apart's own rounding.
W4A4_ROUTE_HD constexpr float route_units(int bits) { return (float)(1u << (32 - bits)) - 512.0f; }
W4A4_ROUTE_HD inline uint32_t route_apart(int bits, float error, float unit)
{
    const float rounding = bits < 8 ? 4.0f * (float)(1u << (8 - bits)) : 4.0f;
    return (uint32_t)fminf(fmaf(error, unit, rounding + 3.0f), 0x1p31f);
}

}  // namespace w4a4
