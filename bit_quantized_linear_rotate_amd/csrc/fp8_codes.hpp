// Device helpers shared by the fp8 quantisers and the gated product's epilogue.
#pragma once

#include "common.hpp"

namespace w4a4 {
namespace {

// What a block's largest magnitude (its fp32 bits, infinity and NaN on top) means for
// its values.  With A = max(absmax, 448 * 2^-126) the scale is A / 448 and a code is
// e4m3(448 y / A): the ratio to the block's largest itself, since y / scale would
// move ties by the scale's own rounding.  `num` * y = 448 y 2^-e with e the exponent
// of A (exact for 16-bit y, at most 896), `den` = A 2^-e in [1, 2): the quotient
// neither overflows nor meets a subnormal divisor whatever A is.
struct Fp8Block {
    float num, den, rden, scale;
    bool bad;
};
__device__ __forceinline__ Fp8Block fp8_block(uint32_t amax)
{
    constexpr uint32_t least = 0x04e00000u;   // 448 * 2^-126
    Fp8Block b;
    b.bad = amax >= 0x7f800000u;
    const uint32_t top = b.bad ? 0x3f800000u : max(amax, least);
    b.num = __uint_as_float(((262u - (top >> 23)) << 23) | 0x600000u);
    b.den = __uint_as_float((top & 0x7fffffu) | 0x3f800000u);
    b.rden = 1.0f / b.den;
    b.scale = b.bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 448.0f;
    return b;
}

// fp32(num y / den): the reciprocal's product, corrected by its exact remainder (a
// rounded division is ten instructions, this is three; where the quotient is
// representable, as on the borders between codes, the correction ends on it).
__device__ __forceinline__ float fp8_ratio(const Fp8Block& b, float y)
{
    const float n = mul_rn(y, b.num), q = mul_rn(n, b.rden);
    return __builtin_fmaf(__builtin_fmaf(-q, b.den, n), b.rden, q);
}

// Four values' codes (nearest, ties to even; the largest is 448 or less by
// construction, so none overflows)
__device__ __forceinline__ uint32_t fp8_codes4(const Fp8Block& b, float v0, float v1, float v2, float v3)
{
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_ratio(b, v0), fp8_ratio(b, v1), 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_ratio(b, v2), fp8_ratio(b, v3), c, true);
    return b.bad ? 0u : (uint32_t)c;
}

}  // namespace
}  // namespace w4a4
