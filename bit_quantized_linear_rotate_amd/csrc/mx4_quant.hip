// MX4 quantiser (optional Hadamard rotation, block scales, e2m1 codes) and its
// inverse.
//
// Mathematics.  Per row and group of g (if rotated), in fp32:
//   y = H_g (x . sign_in) * fp32(1 / sqrt(g)) . sign_out,
// the fast Walsh-Hadamard transform with butterflies of distance 1, 2, 4, ...
// in that order (the order fixes every rounding, so the result is defined to
// the bit).  Per 32 consecutive y: X = max(floor(log2(absmax)) - 2, -127),
// codes = e2m1(y / 2^X) to nearest, ties to the even code, saturated at 6.  y
// stays in fp32 until the codes are taken: there is no rounding in between.
// A block that holds a NaN or an infinity gets scale byte 255 and codes 0.
//
// Bounds.  x is read once and 17/32 of a byte written per value: memory, until
// g = 128; from there the butterflies and the conversion.  A lane holds sixteen
// consecutive values, sixteen lanes a slab of 256 of a row: butterflies up to
// distance 8 are in registers, the others DPP moves within a row of sixteen
// lanes, a block is two lanes and its scales and codes leave in whole words.
// Measured (hot and cold differ by a tenth): 8192 x 3840 bf16, g = 64 16.9 us =
// 4.7 TB/s (a copy of as many bytes 15.3), unrotated 13.4; 8192 x 10240 fp16,
// g = 256 47 to 51 us = 4.2 TB/s; the way back 14.2 us = 5.6 TB/s; 32 x 3840
// 3.2 and 2.6 us, a launch.
#include "common.hpp"
#include "mx4.hpp"
#include "rotate16.hpp"

namespace w4a4 {

namespace {

// Sixteen lanes hold 256 consecutive k of a row, sixteen per lane (the more a
// lane holds, the fewer butterflies cross lanes, and those cost twice); a
// workgroup takes U * 16 rows of one slab, so its scale bytes lie side by side,
// and every lane has U rows in flight.  VEC: 16-byte loads from contiguous
// aligned rows; else one load per element at any strides.
template <int DT, int G, bool VEC, int U>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(Mx4QuantArgs a)
{
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15;
    const int64_t M = a.M, K = a.K;
    const int64_t slab = blockIdx.y;
    const int64_t k0 = slab * kMxSlab + l16 * 16;
    const int64_t row0 = (int64_t)blockIdx.x * (16 * U) + (tid >> 4);
    const bool in_k = k0 < K;
    constexpr int ESZ = DT == F32 ? 4 : 2, W = 4 * ESZ;   // 32-bit words of a lane's values
    // input signs as sign bits of those words, output signs as those of codes
    uint32_t si[W], so[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < W; ++i) si[i] = 0;
    if constexpr (G > 0) {
        // (the sign bytes are 8-byte aligned)
        const int o = (l16 * 16) & (G - 1);
        auto negative = [&](const int8_t* s, int e) {
            const v2u w = ((const v2u*)(s + o))[e >> 3];
            return (w[(e >> 2) & 1] >> (8 * (e & 3) + 7)) & 1u;
        };
        if (a.sign_in)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if constexpr (DT == F32) si[e] = negative(a.sign_in, e) << 31;
                else si[e >> 1] |= negative(a.sign_in, e) << (15 + 16 * (e & 1));
            }
        if (a.sign_out)
#pragma unroll
            for (int e = 0; e < 16; ++e) so[e >> 3] |= negative(a.sign_out, e) << (3 + 4 * (e & 7));
    }
    uint32_t raw[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + 16 * u;
        const bool in = in_k && row < M;
#pragma unroll
        for (int i = 0; i < W; ++i) raw[u][i] = 0;
        if constexpr (VEC) {
            if (in) {
                const v4u* p = (const v4u*)((const char*)a.x + (row * a.sm + k0) * ESZ);
#pragma unroll
                for (int i = 0; i < ESZ; ++i) {
                    const v4u t = p[i];
#pragma unroll
                    for (int c = 0; c < 4; ++c) raw[u][4 * i + c] = t[c];
                }
            }
        } else if (in) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int64_t at = row * a.sm + (k0 + e) * a.sk;
                if constexpr (DT == F32) raw[u][e] = ((const uint32_t*)a.x)[at];
                else raw[u][e >> 1] |= (uint32_t)((const uint16_t*)a.x)[at] << (16 * (e & 1));
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + 16 * u;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if constexpr (DT == F32) v[e] = __uint_as_float(raw[u][e] ^ si[e]);
            else v[e] = h_to_f32<DT>((uint16_t)((raw[u][e >> 1] ^ si[e >> 1]) >> (16 * (e & 1))));
        }
        if constexpr (G > 0) rotate16<G>(v, lane);
        constexpr int KEXP = inv_sqrt_exp<G>();
        if constexpr (G > 0 && KEXP == 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = mul_rn(v[e], inv_sqrt<G>());
        }
        uint32_t m = amax_bits(v);
        m = max(m, mq_xor<1>(m));
        int k = KEXP;   // y = v * 2^-k
        if constexpr (KEXP > 0) {
            // Near the subnormals the multiplication rounds, so it is done.
            if (__any(m && m < (40u << 23))) {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = mul_rn(v[e], inv_sqrt<G>());
                m = amax_bits(v);
                m = max(m, mq_xor<1>(m));
                k = 0;
            }
        }
        const int ex = (int)(m >> 23);
        const bool bad = ex == 255;
        const int byte = bad ? 255 : ex > 2 + k ? ex - 2 - k : 0;
        const float sc = __uint_as_float((uint32_t)(byte + k) << 23);   // the conversion reads the exponent field only
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            c[p] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[p], v[8 * p + 0], v[8 * p + 1], sc, 0);
            c[p] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[p], v[8 * p + 2], v[8 * p + 3], sc, 1);
            c[p] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[p], v[8 * p + 4], v[8 * p + 5], sc, 2);
            c[p] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[p], v[8 * p + 6], v[8 * p + 7], sc, 3);
            c[p] = bad ? 0u : c[p] ^ so[p];
        }
        if (row < M) {
            if (in_k) *(v2u*)(a.codes + row * (K >> 1) + (k0 >> 1)) = (v2u){c[0], c[1]};
            if (!(lane & 1)) a.scales[(slab * M + row) * 8 + (l16 >> 1)] = (uint8_t)(in_k ? byte : 0);
        }
    }
}

// Eight values per thread: 4 bytes of codes in, 16 or 32 bytes out.  The
// fp32 products are exact; 16-bit outputs round once.
template <int ODT>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int64_t M, int64_t K,
                                                             int64_t pieces, void* __restrict__ out)
{
    const int64_t per_row = K >> 3;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per_row, p = i - row * per_row;
        const uint32_t c = ((const uint32_t*)codes)[i];
        const int64_t blk = p >> 2;
        const uint32_t byte = scales[((blk >> 3) * M + row) * 8 + (blk & 7)];
        // 2^-127 is the subnormal 0x00400000; 255 is NaN
        const float s = __uint_as_float(byte == 255 ? 0x7fc00000u : byte ? byte << 23 : 0x00400000u);
        typedef float f2 __attribute__((ext_vector_type(2)));
        float v[8];
        const f2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0), v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
        const f2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2), v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
        v[0] = mul_rn(v0[0], s); v[1] = mul_rn(v0[1], s); v[2] = mul_rn(v1[0], s); v[3] = mul_rn(v1[1], s);
        v[4] = mul_rn(v2[0], s); v[5] = mul_rn(v2[1], s); v[6] = mul_rn(v3[0], s); v[7] = mul_rn(v3[1], s);
        if constexpr (ODT == F32) {
            v4u* o = (v4u*)out + 2 * i;
            o[0] = (v4u){__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
            o[1] = (v4u){__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
        } else {
            v4u o;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = f32_to_h<ODT>(v[2 * e]) | ((uint32_t)f32_to_h<ODT>(v[2 * e + 1]) << 16);
            ((v4u*)out)[i] = o;
        }
    }
}

template <int DT, int G, bool VEC> hipError_t quantize_u(const Mx4QuantArgs& a, hipStream_t st)
{
    // Two rows in flight per lane once that still leaves a workgroup for
    // every CU several times over; a decode batch spreads over the CUs instead.
    const unsigned slabs = (unsigned)mx4_slabs(a.K);
    if ((a.M + 31) / 32 * slabs >= 1024)
        hipLaunchKernelGGL((mx4_quantize_kernel<DT, G, VEC, 2>), dim3((unsigned)((a.M + 31) / 32), slabs), dim3(256), 0,
                           st, a);
    else
        hipLaunchKernelGGL((mx4_quantize_kernel<DT, G, VEC, 1>), dim3((unsigned)((a.M + 15) / 16), slabs), dim3(256), 0,
                           st, a);
    return hipGetLastError();
}

template <int DT, int G> hipError_t quantize_g(const Mx4QuantArgs& a, hipStream_t st)
{
    const int esz = DT == F32 ? 4 : 2;
    const bool vec = a.sk == 1 && (a.sm * esz) % 16 == 0 && (uintptr_t)a.x % 16 == 0;
    return vec ? quantize_u<DT, G, true>(a, st) : quantize_u<DT, G, false>(a, st);
}

template <int DT> hipError_t quantize_dt(const Mx4QuantArgs& a, hipStream_t st)
{
    switch (a.g) {
    case 0: return quantize_g<DT, 0>(a, st);
    case 16: return quantize_g<DT, 16>(a, st);
    case 32: return quantize_g<DT, 32>(a, st);
    case 64: return quantize_g<DT, 64>(a, st);
    case 128: return quantize_g<DT, 128>(a, st);
    case 256: return quantize_g<DT, 256>(a, st);
    }
    return hipErrorNotSupported;
}

}  // namespace

hipError_t launch_mx4_quantize(const Mx4QuantArgs& a, hipStream_t st)
{
    switch (a.dtype) {
    case F32: return quantize_dt<F32>(a, st);
    case F16: return quantize_dt<F16>(a, st);
    case BF16: return quantize_dt<BF16>(a, st);
    }
    return hipErrorNotSupported;
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* out,
                                 int out_dtype, hipStream_t st)
{
    const int64_t pieces = M * (K >> 3);
    const unsigned grid = (unsigned)((pieces + 255) / 256 < 65536 ? (pieces + 255) / 256 : 65536);
    if (out_dtype == F32)
        hipLaunchKernelGGL(mx4_dequantize_kernel<F32>, dim3(grid), dim3(256), 0, st, codes, scales, M, K, pieces, out);
    else if (out_dtype == F16)
        hipLaunchKernelGGL(mx4_dequantize_kernel<F16>, dim3(grid), dim3(256), 0, st, codes, scales, M, K, pieces, out);
    else
        hipLaunchKernelGGL(mx4_dequantize_kernel<BF16>, dim3(grid), dim3(256), 0, st, codes, scales, M, K, pieces, out);
    return hipGetLastError();
}

}  // namespace w4a4
