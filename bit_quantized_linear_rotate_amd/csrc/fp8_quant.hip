// Block-scaled fp8 quantisers (optional Hadamard rotation, block scales, e4m3
// codes) of activation rows and of weights, and their inverses.
//
// Mathematics.  Per row and group of g (if rotated), in fp32:
//   y = H_g (x . sign_in) * fp32(1 / sqrt(g)) . sign_out,
// the fast Walsh-Hadamard transform with butterflies of distance 1, 2, 4, ...
// in that order (the order fixes every rounding, so the result is defined to
// the bit).  Per block (128 k of a row; of weights 128 rows by 128 k):
//   A = max(absmax, 448 * 2^-126), scale = A / 448, code = e4m3(448 y / A),
// to nearest, ties to the even code.  A block that holds a NaN or an infinity
// gets the scale NaN and codes 0.
//
// Bounds.  Everything is read once and written once (rows: 3 or 5 bytes per value
// and 1/32 for the scale): memory, and from g = 64 on the instructions of the
// butterflies and of the ratios (four per value) beside it.  A lane holds sixteen
// consecutive values of a row, so butterflies up to distance 8 stay in registers and
// its codes leave in 16 bytes; the further ones are DPP moves within sixteen lanes.
// Input signs flip bits of the raw words, output signs those of the codes: eight and
// four instructions instead of three per value (8192 x 10240, g = 256: 61 -> 56 us).
// Measured, hot: rows 8192 x 3840 bf16 15.9 us = 6.0 TB/s, rotated by g = 64 19.5 =
// 4.9; 8192 x 10240 bf16 39 us = 6.5 TB/s, g = 256 56 = 4.5.  Two rows per lane
// instead of one: 38.5 unrotated but 21.5 us at g = 64 (registers), so one.  Weights
// 10240 x 3840: fp32 29.2 us = 6.7 TB/s, g = 64 30.9 = 6.4; bf16 20.1 = 5.9 and
// 25.6 = 4.6.
#include "common.hpp"
#include "fp8.hpp"
#include "fp8_codes.hpp"
#include "rotate16.hpp"

namespace w4a4 {

namespace {

// Where the signs of a lane's sixteen values go: `in` flips those of the raw words,
// `out` those of the codes (a sign commutes with the rounding, and sixteen codes
// are four words).  The sign bytes are 8-byte aligned.
template <int DT> struct Signs {
    static constexpr int W = DT == F32 ? 16 : 8;
    uint32_t in[W], out[4];
    __device__ __forceinline__ void load(const int8_t* sign_in, const int8_t* sign_out, int o)
    {
        auto negative = [&](const int8_t* s, int e) {
            const v2u w = ((const v2u*)(s + o))[e >> 3];
            return (w[(e >> 2) & 1] >> (8 * (e & 3) + 7)) & 1u;
        };
#pragma unroll
        for (int i = 0; i < W; ++i) in[i] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = 0;
        if (sign_in)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if constexpr (DT == F32) in[e] = negative(sign_in, e) << 31;
                else in[e >> 1] |= negative(sign_in, e) << (15 + 16 * (e & 1));
            }
        if (sign_out)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[e] = ((const v2u*)(sign_out + o))[e >> 1][e & 1] & 0x80808080u;
    }
};

// Sixteen consecutive k of one row, as words (VEC: 16-byte loads; else one load per
// element at any stride)
template <int DT, bool VEC, int W> __device__ __forceinline__ void load16(const void* x, int64_t at, int64_t sk, uint32_t (&raw)[W])
{
    constexpr int ESZ = DT == F32 ? 4 : 2;
    if constexpr (VEC) {
        const v4u* p = (const v4u*)((const char*)x + at * ESZ);
#pragma unroll
        for (int i = 0; i < ESZ; ++i) {
            const v4u t = p[i];
#pragma unroll
            for (int c = 0; c < 4; ++c) raw[4 * i + c] = t[c];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if constexpr (DT == F32) raw[e] = ((const uint32_t*)x)[at + e * sk];
            else raw[e >> 1] |= (uint32_t)((const uint16_t*)x)[at + e * sk] << (16 * (e & 1));
        }
    }
}

// The rotated values of sixteen raw ones, but for the output signs
template <int DT, int G, int W>
__device__ __forceinline__ void rotated(const uint32_t (&raw)[W], const Signs<DT>& s, int lane, float (&v)[16])
{
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        if constexpr (DT == F32) v[e] = __uint_as_float(G > 0 ? raw[e] ^ s.in[e] : raw[e]);
        else v[e] = h_to_f32<DT>((uint16_t)((G > 0 ? raw[e >> 1] ^ s.in[e >> 1] : raw[e >> 1]) >> (16 * (e & 1))));
    }
    if constexpr (G > 0) {
        rotate16<G>(v, lane);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = mul_rn(v[e], inv_sqrt<G>());
    }
}

// The codes of sixteen rotated values
template <int DT, int G>
__device__ __forceinline__ v4u codes16(const Fp8Block& b, const Signs<DT>& s, const float (&v)[16])
{
    v4u c;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        c[p] = fp8_codes4(b, v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
        if constexpr (G > 0) c[p] = b.bad ? 0u : c[p] ^ s.out[p];
    }
    return c;
}

// Sixteen lanes hold 256 consecutive k of a row, sixteen per lane; eight lanes
// are a block.  A workgroup takes 16 rows of one pair of blocks.
template <int DT, int G, bool VEC>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(Fp8QuantArgs a)
{
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15;
    const int64_t M = a.M, K = a.K;
    const int64_t k0 = (int64_t)blockIdx.y * 256 + l16 * 16;
    const int64_t row = (int64_t)blockIdx.x * 16 + (tid >> 4);
    const bool in = k0 < K && row < M;
    Signs<DT> s;
    if constexpr (G > 0) s.load(a.sign_in, a.sign_out, (l16 * 16) & (G - 1));
    uint32_t raw[Signs<DT>::W];
#pragma unroll
    for (int i = 0; i < Signs<DT>::W; ++i) raw[i] = 0;
    if (in) load16<DT, VEC>(a.x, row * a.sm + k0 * a.sk, a.sk, raw);
    float v[16];
    rotated<DT, G>(raw, s, lane, v);
    uint32_t m = amax_bits(v);
    m = max(m, mq_xor<1>(m));
    m = max(m, mq_xor<2>(m));
    m = max(m, mq_xor<4>(m));
    const Fp8Block b = fp8_block(m);
    if (in) {
        *(v4u*)(a.codes + row * K + k0) = codes16<DT, G>(b, s, v);
        if (!(l16 & 7)) a.scales[(k0 >> 7) * M + row] = b.scale;
    }
}

// Weights: a workgroup takes 128 rows of two k blocks, R rows per lane, which stay in
// registers while the largest magnitudes of the lanes meet in LDS.  R = 4: with 8 a
// rotated block leaves one wave per SIMD (fp32, g = 64: 34.5 us against 30.9, bf16
// 28.0 against 25.6), with 2 the workgroup of 1024 has too few registers (40 and 25.5).
template <int DT, int G, bool VEC, int R>
__global__ __launch_bounds__(2048 / R) void fp8_quantize_weights_kernel(Fp8QuantArgs a)
{
    constexpr int GROUPS = 128 / R;   // of sixteen lanes
    __shared__ uint32_t top[2][GROUPS];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, grp = tid >> 4;
    const int64_t N = a.M, K = a.K;
    const int64_t nb = blockIdx.x, e = blockIdx.z;
    const int64_t k0 = (int64_t)blockIdx.y * 256 + l16 * 16;
    const bool in_k = k0 < K;
    constexpr int W = Signs<DT>::W;
    Signs<DT> s;
    if constexpr (G > 0) s.load(a.sign_in, a.sign_out, (l16 * 16) & (G - 1));
    uint32_t raw[R][W];
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int64_t row = nb * 128 + GROUPS * u + grp;
#pragma unroll
        for (int i = 0; i < W; ++i) raw[u][i] = 0;
        if (in_k && row < N) load16<DT, VEC>(a.x, e * a.se + row * a.sm + k0 * a.sk, a.sk, raw[u]);
    }
    float v[R][16];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < R; ++u) {
        rotated<DT, G>(raw[u], s, lane, v[u]);
        m = max(m, amax_bits(v[u]));
    }
    m = max(m, mq_xor<1>(m));
    m = max(m, mq_xor<2>(m));
    m = max(m, mq_xor<4>(m));
    if (!(l16 & 7)) top[l16 >> 3][grp] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) m = max(m, top[l16 >> 3][i]);
    const Fp8Block b = fp8_block(m);
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int64_t row = nb * 128 + GROUPS * u + grp;
        if (in_k && row < N) *(v4u*)(a.codes + (e * N + row) * K + k0) = codes16<DT, G>(b, s, v[u]);
    }
    if (grp == 0 && !(l16 & 7) && in_k) a.scales[(e * fp8_blocks(N) + nb) * fp8_blocks(K) + (k0 >> 7)] = b.scale;
}

// Sixteen values per thread: 16 bytes of codes in, 32 or 64 out; code times scale
// in fp32, rounded once more to 16 bits.  Bound by memory: 8192 x 10240 codes to
// bf16 42 us = 6.0 TB/s, to fp32 118 = 3.6 (stores, past what the last-level cache
// holds); of weights 38 = 6.7 and 108 = 3.9.
template <int ODT, bool WEIGHTS>
__global__ __launch_bounds__(256) void fp8_dequantize_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                                                             int64_t rows, int64_t M, int64_t K, int64_t pieces,
                                                             void* __restrict__ out)
{
    const int64_t per_row = K >> 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per_row, kb = (i - row * per_row) >> 3;
        const v4u c = ((const v4u*)codes)[i];
        float s;
        if constexpr (WEIGHTS) {
            const int64_t e = row / M, n = row - e * M;
            s = scales[(e * fp8_blocks(M) + (n >> 7)) * fp8_blocks(K) + kb];
        } else {
            s = scales[kb * rows + row];
        }
        float v[16];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[p], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[p], true);
            v[4 * p + 0] = mul_rn(lo[0], s);
            v[4 * p + 1] = mul_rn(lo[1], s);
            v[4 * p + 2] = mul_rn(hi[0], s);
            v[4 * p + 3] = mul_rn(hi[1], s);
        }
        if constexpr (ODT == F32) {
            v4u* o = (v4u*)out + 4 * i;
#pragma unroll
            for (int p = 0; p < 4; ++p)
                o[p] = (v4u){__float_as_uint(v[4 * p]), __float_as_uint(v[4 * p + 1]), __float_as_uint(v[4 * p + 2]),
                             __float_as_uint(v[4 * p + 3])};
        } else {
            v4u* o = (v4u*)out + 2 * i;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                v4u w;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = f32_to_h<ODT>(v[8 * p + 2 * j]) | ((uint32_t)f32_to_h<ODT>(v[8 * p + 2 * j + 1]) << 16);
                o[p] = w;
            }
        }
    }
}

constexpr int kWeightRows = 4;   // rows per lane of the weights' quantiser

template <int DT, int G, bool VEC> hipError_t quantize_v(const Fp8QuantArgs& a, bool weights, hipStream_t st)
{
    const unsigned pairs = (unsigned)((a.K + 255) / 256);
    if (weights)
        hipLaunchKernelGGL((fp8_quantize_weights_kernel<DT, G, VEC, kWeightRows>),
                           dim3((unsigned)fp8_blocks(a.M), pairs, (unsigned)a.E), dim3(2048 / kWeightRows), 0, st, a);
    else
        hipLaunchKernelGGL((fp8_quantize_kernel<DT, G, VEC>), dim3((unsigned)((a.M + 15) / 16), pairs), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int DT, int G> hipError_t quantize_g(const Fp8QuantArgs& a, bool weights, hipStream_t st)
{
    const int esz = DT == F32 ? 4 : 2;
    const bool vec = a.sk == 1 && (a.sm * esz) % 16 == 0 && (a.se * esz) % 16 == 0 && (uintptr_t)a.x % 16 == 0;
    return vec ? quantize_v<DT, G, true>(a, weights, st) : quantize_v<DT, G, false>(a, weights, st);
}

template <int DT> hipError_t quantize_dt(const Fp8QuantArgs& a, bool weights, hipStream_t st)
{
    switch (a.g) {
    case 0: return quantize_g<DT, 0>(a, weights, st);
    case 16: return quantize_g<DT, 16>(a, weights, st);
    case 32: return quantize_g<DT, 32>(a, weights, st);
    case 64: return quantize_g<DT, 64>(a, weights, st);
    case 128: return quantize_g<DT, 128>(a, weights, st);
    case 256: return quantize_g<DT, 256>(a, weights, st);
    }
    return hipErrorNotSupported;
}

hipError_t quantize(const Fp8QuantArgs& a, bool weights, hipStream_t st)
{
    switch (a.dtype) {
    case F32: return quantize_dt<F32>(a, weights, st);
    case F16: return quantize_dt<F16>(a, weights, st);
    case BF16: return quantize_dt<BF16>(a, weights, st);
    }
    return hipErrorNotSupported;
}

template <int ODT> hipError_t dequantize(const uint8_t* codes, const float* scales, int64_t E, int64_t M, int64_t K, void* out,
                                         hipStream_t st)
{
    const int64_t rows = E ? E * M : M, pieces = rows * (K >> 4);
    const unsigned grid = (unsigned)((pieces + 255) / 256 < 65536 ? (pieces + 255) / 256 : 65536);
    if (E)
        hipLaunchKernelGGL((fp8_dequantize_kernel<ODT, true>), dim3(grid), dim3(256), 0, st, codes, scales, rows, M, K, pieces, out);
    else
        hipLaunchKernelGGL((fp8_dequantize_kernel<ODT, false>), dim3(grid), dim3(256), 0, st, codes, scales, rows, M, K, pieces, out);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, hipStream_t st) { return quantize(a, false, st); }
hipError_t launch_fp8_quantize_weights(const Fp8QuantArgs& a, hipStream_t st) { return quantize(a, true, st); }

hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t E, int64_t M, int64_t K, void* out,
                                 int out_dtype, hipStream_t st)
{
    switch (out_dtype) {
    case F32: return dequantize<F32>(codes, scales, E, M, K, out, st);
    case F16: return dequantize<F16>(codes, scales, E, M, K, out, st);
    case BF16: return dequantize<BF16>(codes, scales, E, M, K, out, st);
    }
    return hipErrorNotSupported;
}

}  // namespace w4a4
