// Device helpers shared by the products grouped by expert (MX4 and fp8): range-checked
// resources and DMA, the rows a workgroup takes, the gate, biases and 16-bit packing.
// `Args` has E, R, offsets, N, bias and bias_dtype (Mx4GemmArgs, Fp8GemmArgs).
#pragma once

#include "common.hpp"

namespace w4a4 {
namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));

constexpr uint32_t kOut = 0x80000000u;   // a lane offset past every resource here

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_rsrc(const void* base, int64_t bytes)
{
    const uint32_t n = bytes > 0x80000000ll ? 0x80000000u : bytes < 0 ? 0u : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)n, 0x00020000);
}

// A pointer that is the same in all lanes, where the compiler cannot tell: its
// resource stays in scalar registers (otherwise each access becomes a loop).
__device__ __forceinline__ const uint8_t* mx_uniform(const uint8_t* p)
{
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return (const uint8_t*)((uint64_t)hi << 32 | lo);
}

// BYTES per lane from the resource (lane offset vo, scalar offset so; nothing
// past its end: zeros) to consecutive LDS bytes
template <int BYTES> __device__ __forceinline__ void mx_dma(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t vo, int so)
{
    using lds_vptr = __attribute__((address_space(3))) void*;
    if constexpr (BYTES == 16)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_vptr)lds, 16, (int)vo, so, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_vptr)lds, 4, (int)vo, so, 0, 0);
}

// ---- which rows a workgroup takes --------------------------------------------
struct MxRows {
    int64_t m0;   // the expert's first (sorted) row
    int rows;     // rows of the expert
    int e;        // expert, -1: none
    int64_t before;   // tiles of the experts before it
};

// offsets[e], kept inside [0, R] whatever the device array holds
template <class Args> __device__ __forceinline__ int64_t mx_offset(const Args& a, int e)
{
    const int64_t o = a.offsets[e];
    return o < 0 ? 0 : o > a.R ? a.R : o;
}

// inclusive sum over the lanes: within rows of sixteen, then across
__device__ __forceinline__ int mx_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast 15, 31
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
    return v;
}

// The expert that has row tile `idx` of the list of all experts' tiles of BM
// rows (BY_TILE; else only count).  Every wave scans the offsets, 64 experts at
// a time.  Returns the number of tiles (of those looked at).
template <int BM, bool BY_TILE, class Args> __device__ __forceinline__ int64_t mx_find(const Args& a, int64_t idx, MxRows& r)
{
    const int lane = threadIdx.x & 63;
    int64_t base = 0;
    r.rows = 0;
    r.e = -1;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + lane;
        int64_t lo = 0, hi = 0;
        if (e < a.E) {
            lo = mx_offset(a, e);
            hi = mx_offset(a, e + 1);
        }
        const int cnt = hi > lo ? (int)(hi - lo) : 0;
        const int cm = (cnt + BM - 1) / BM;
        const int inc = mx_scan(cm);
        const int sum = __builtin_amdgcn_readlane(inc, 63);
        if (BY_TILE && r.e < 0 && idx >= base && idx < base + sum) {
            const unsigned long long hit = __ballot(base + inc > idx);
            const int w = __builtin_ctzll(hit);
            r.e = e0 + w;
            r.before = base + __builtin_amdgcn_readlane(inc, w) - __builtin_amdgcn_readlane(cm, w);
            r.m0 = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)lo, w);
            r.rows = __builtin_amdgcn_readlane(cnt, w);
            return base + sum;
        }
        base += sum;
    }
    return base;
}

// For each lane, row tile and column tile number `tile` of the list of all
// experts' tiles (BM rows by one of tiles_n column tiles): within an expert,
// groups of eight row tiles, row tiles fastest.
template <int BM, class Args>
__device__ __forceinline__ void mx_rows_of(const Args& a, int tile, int tiles_n, int& e, int& m0, int& tn, int& rows)
{
    const int lane = threadIdx.x & 63, row_tile = tile / tiles_n;
    int base = 0;
    e = m0 = tn = rows = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        int lo = 0, hi = 0;
        if (e0 + lane < a.E) {
            lo = (int)mx_offset(a, e0 + lane);
            hi = (int)mx_offset(a, e0 + lane + 1);
        }
        const int cnt = hi > lo ? hi - lo : 0, cm = (cnt + BM - 1) / BM, inc = mx_scan(cm);
        const int sum = __builtin_amdgcn_readlane(inc, 63);
        // the first expert whose tiles reach past row_tile
        const int x = row_tile - base;
        int w = 0;
#pragma unroll
        for (int d = 32; d; d >>= 1)
            if (__builtin_amdgcn_ds_bpermute((w + d - 1) * 4, inc) <= x) w += d;
        w = min(w, 63);
        const int wlo = __builtin_amdgcn_ds_bpermute(w * 4, lo), wcnt = __builtin_amdgcn_ds_bpermute(w * 4, cnt);
        const int wcm = __builtin_amdgcn_ds_bpermute(w * 4, cm), winc = __builtin_amdgcn_ds_bpermute(w * 4, inc);
        if (x >= 0 && x < sum) {
            const int in_e = tile - (base + winc - wcm) * tiles_n, per = 8 * tiles_n, grp = in_e / per;
            const int gm = min(wcm - grp * 8, 8), in_g = in_e - grp * per, m = grp * 8 + in_g % gm;
            e = e0 + w;
            tn = in_g / gm;
            m0 = wlo + m * BM;
            rows = min(wcnt - m * BM, BM);
        }
        base += sum;
    }
}

// silu(g) * u in fp32: g (1 / (1 + exp(-g))) u, rounded to four or eight bits next.  exp is
// 2^(-g log2(e)), whose argument is rounded twice, so off by up to |g| 2^-23 of
// itself; the power and the reciprocal are the hardware's (1 ulp; a rounded
// division is ten instructions a value, 2 us a tile of 256 x 128 results).  In all
// (|g| + 4) 2^-23 of the value.  Where the reciprocal falls below 2^-126 (g < -87)
// it is zero.
__device__ __forceinline__ float mx_gated(float g, float u)
{
    return mul_rn(mul_rn(g, __builtin_amdgcn_rcpf(add_rn(1.0f, __expf(-g)))), u);
}

template <int ODT> __device__ __forceinline__ uint32_t mx_pack2(float lo, float hi)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    if constexpr (ODT == BF16) {
        typedef __bf16 h2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){lo, hi}, h2));
    } else {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){lo, hi}, h2));
    }
}

// The biases of this lane, columns c + 32 nt .. + 15 of the n that start at
// column `first` of expert e's row (zeros from n on).  Loaded all together and
// waited for here: the compiler's own waits would reach into the K loop.
template <int NB, class Args>
__device__ __forceinline__ void mx_bias(const Args& a, int e, int64_t first, int64_t n, int64_t c, float (&bv)[NB][16])
{
    const int dt = a.bias_dtype, esz = dt == F32 ? 4 : 2;
    const uint8_t* p = mx_uniform((const uint8_t*)a.bias + ((int64_t)e * a.N + first) * esz);
    const __amdgpu_buffer_rsrc_t r = mx_rsrc(p, n * esz);
    const int o = (int)(c * esz);
    if (dt == F32) {
#pragma unroll
        for (int i = 0; i < NB * 16; ++i)
            bv[i >> 4][i & 15] = __uint_as_float(
                (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, o + (i >> 4) * 128 + (i & 15) * 4, 0, 0));
        __builtin_amdgcn_s_waitcnt(0x0f70);
        return;
    }
    uint32_t w[NB][8];
    if (((uintptr_t)p | (uintptr_t)(n * 2)) % 16 == 0) {
#pragma unroll
        for (int i = 0; i < NB * 2; ++i) {
            const v4u t = __builtin_bit_cast(
                v4u, __builtin_amdgcn_raw_buffer_load_b128(r, o + (i >> 1) * 64 + (i & 1) * 16, 0, 0));
#pragma unroll
            for (int k = 0; k < 4; ++k) w[i >> 1][(i & 1) * 4 + k] = t[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NB * 8; ++i)
            w[i >> 3][i & 7] =
                (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, o + (i >> 3) * 64 + (i & 7) * 4, 0, 0) |
                (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, o + (i >> 3) * 64 + (i & 7) * 4 + 2, 0, 0) << 16;
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);
#pragma unroll
    for (int i = 0; i < NB * 16; ++i) {
        const uint16_t h = (uint16_t)(w[i >> 4][(i & 15) >> 1] >> (16 * (i & 1)));
        bv[i >> 4][i & 15] = dt == BF16 ? bf16_to_f32(h) : f16_to_f32(h);
    }
}

}  // namespace
}  // namespace w4a4
