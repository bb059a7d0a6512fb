// Device helpers of the block quantisers (MX4 and fp8): sixteen consecutive values of a
// row per lane, sixteen lanes 256 of them, the fast Walsh-Hadamard transform over
// groups of up to 256 and the largest magnitude.
#pragma once

#include "common.hpp"

namespace w4a4 {
namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));

// the value of the lane whose index differs in bit D (D = 1, 2, 4, 8)
template <int D> __device__ __forceinline__ uint32_t mq_xor(uint32_t v)
{
    if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true);        // quad [1,0,3,2]
    else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(v, 0x4e, 0xf, 0xf, true);   // quad [2,3,0,1]
    else if constexpr (D == 4)                                                             // 7 - i, then quad [3,2,1,0]
        return __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true), 0x1b, 0xf, 0xf, true);
    else return __builtin_amdgcn_mov_dpp(v, 0x128, 0xf, 0xf, true);                        // row rotate by 8
}

template <int D> __device__ __forceinline__ void butterfly_across(float (&v)[16], int lane)
{
    const float s = (lane & D) ? -1.0f : 1.0f;   // upper partner: other - own, lower: own + other
#pragma unroll
    for (int e = 0; e < 16; ++e)
        v[e] = __builtin_fmaf(s, v[e], __uint_as_float(mq_xor<D>(__float_as_uint(v[e]))));
}

// sixteen consecutive values per lane: distances 1, 2, 4, 8 within the lane,
// 16, 32, 64, 128 across lanes
template <int G> __device__ __forceinline__ void rotate16(float (&v)[16], int lane)
{
#pragma unroll
    for (int d = 1; d < 16; d *= 2)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (!(e & d)) {
                const float a = v[e], b = v[e + d];
                v[e] = add_rn(a, b);
                v[e + d] = add_rn(a, -b);
            }
    if constexpr (G >= 32) butterfly_across<1>(v, lane);
    if constexpr (G >= 64) butterfly_across<2>(v, lane);
    if constexpr (G >= 128) butterfly_across<4>(v, lane);
    if constexpr (G >= 256) butterfly_across<8>(v, lane);
}

template <int G> constexpr float inv_sqrt()
{
    // fp32(1 / sqrt(g))
    return G == 16 ? 0.25f : G == 32 ? 0.17677669529663687f : G == 64 ? 0.125f : G == 128 ? 0.08838834764831845f : 0.0625f;
}
// g = 16, 64, 256: 1 / sqrt(g) = 2^-k, an exponent's worth; else 0
template <int G> constexpr int inv_sqrt_exp() { return G == 16 ? 2 : G == 64 ? 3 : G == 256 ? 4 : 0; }

// The fp32 bits of the largest magnitude of sixteen values, infinity and NaN on
// top.  The maximum keeps a NaN wherever it stands (fmaxf would drop it beside a
// number): butterflies of finite values can overflow to infinities and then
// cancel to a NaN in a block that is otherwise finite.
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[16])
{
    float m = __builtin_elementwise_maximum(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
    for (int e = 2; e < 16; e += 2)
        m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(v[e])), fabsf(v[e + 1]));
    return __float_as_uint(m) & 0x7fffffffu;
}

}  // namespace
}  // namespace w4a4
