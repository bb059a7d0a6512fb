// The MX4 product out[m][n] = sum_k a[m][k] w[n][k] (+ bias[n]) on gfx950's
// scaled f8f6f4 matrix cores, dense and grouped by expert.
//
// Mathematics.  v_mfma_scale_f32_32x32x64_f8f6f4 (16x16x128) multiplies 32 x 64
// by 64 x 32 (16 x 128 by 128 x 16) e2m1 values, each run of 32 k of a row
// times its own power of two, and adds to fp32.  Products of two e2m1 values
// are multiples of 1/4 up to 36, so the sum over a block is exact; sums over
// blocks and steps are fp32.  A lane supplies one row, one block of 32 k and
// that block's scale byte; which block is free as long as both operands agree.
// A step is 256 k, the eight blocks of a scale slab: with 32 x 32 tiles lane
// half h takes the blocks 4h .. 4h + 3, four MFMAs (t = 0 .. 3) whose scales
// are the bytes of one word; with 16 x 16 tiles lane group q takes 2q, 2q + 1.
// The tile kernel uses 32 x 32: one wave per SIMD reaches 8.1 PFLOP/s with it
// and 4.9 with 16 x 16 (registers only, no memory).
#include "common.hpp"
#include "mx4.hpp"

namespace w4a4 {

namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef int v8i __attribute__((ext_vector_type(8)));

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

template <int SB, int SA> __device__ __forceinline__ v4f mx_mfma(v4i w, v4i a, v4f c, uint32_t sw, uint32_t sa)
{
    const v8i w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0}, a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, a8, c, 4, 4, SB, (int)sw, SA, (int)sa);
}

// One 32 x 32 MFMA with byte T of its scale words.  The accumulators are read
// and written in place in accumulation registers (256 of them is all there
// are: any other allocation moves them around), and the instruction stays where
// it is written: the compiler neither moves it across barriers nor sees the
// matrix core's latencies.  s_nop 1: the two wait states between a vector
// instruction's result and an MFMA that reads it (it passes under the MFMA
// before).
typedef float v16f __attribute__((ext_vector_type(16)));
template <int T> __device__ __forceinline__ void mx_mma(v16f& c, const v4i& w, const v4i& a, uint32_t sw, uint32_t sa)
{
#define MX_MMA(sel)                                                                                           \
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 " sel " cbsz:4 blgp:4"   \
                 : "+a"(c)                                                                                    \
                 : "v"(w), "v"(a), "v"(sw), "v"(sa))
    if constexpr (T == 0) MX_MMA("op_sel:[0,0,0] op_sel_hi:[0,0,0]");
    if constexpr (T == 1) MX_MMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
    if constexpr (T == 2) MX_MMA("op_sel:[0,0,0] op_sel_hi:[1,1,0]");
    if constexpr (T == 3) MX_MMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef MX_MMA
}
// Accumulators that start at zero: an MFMA of zeros, in a quarter of the time
// of sixteen register writes each.
__device__ __forceinline__ void mx_clear(v16f (&c)[4])
{
    const v4i z = {0, 0, 0, 0};
#define MX_ZERO(c) "v_mfma_f32_32x32x64_f8f6f4 " c ", %4, %4, 0 cbsz:4 blgp:4\n\t"
    asm volatile("s_nop 1\n\t" MX_ZERO("%0") MX_ZERO("%1") MX_ZERO("%2") MX_ZERO("%3")
                 : "=a"(c[0]), "=a"(c[1]), "=a"(c[2]), "=a"(c[3])
                 : "v"(z));
#undef MX_ZERO
}
// Before accumulators are read by anything but another MFMA:
// the wait states of the last MFMA.
__device__ __forceinline__ void mx_settle(v16f (&c)[4])
{
    asm volatile("s_nop 15\n\ts_nop 15" : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3]));
}

// An accumulator leaves the accumulation registers no earlier than here (the
// compiler would copy all of them out ahead of the epilogue's branches).  It
// still moves them among each other: 240 moves before most of the epilogues of
// 256-row tiles, which are branches of one kernel, and in the grouped one 16
// registers out to scratch and back, once a tile.
__device__ __forceinline__ void mx_here(v16f& c) { asm volatile("" : "+a"(c)); }

// ---- which rows a workgroup takes --------------------------------------------
struct MxRows {
    int64_t m0;   // the expert's first (sorted) row
    int rows;     // rows of the expert
    int e;        // expert, -1: none
    int64_t before;   // tiles of the experts before it
};

// offsets[e], kept inside [0, R] whatever the device array holds
__device__ __forceinline__ int64_t mx_offset(const Mx4GemmArgs& a, int e)
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
template <int BM, bool BY_TILE> __device__ __forceinline__ int64_t mx_find(const Mx4GemmArgs& a, int64_t idx, MxRows& r)
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
template <int BM>
__device__ __forceinline__ void mx_rows_of(const Mx4GemmArgs& a, int tile, int tiles_n, int& e, int& m0, int& tn, int& rows)
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

// Zeros for the sorted rows that no expert owns (before offsets[0] and from
// offsets[E] on), spread over the workgroups that have no tile.
__device__ __forceinline__ void mx_zero_rows(const Mx4GemmArgs& a, int64_t part, int64_t parts)
{
    // number i of these rows' elements, n to a row: one of a row before the
    // first expert's, or one past the last's
    const int64_t first = mx_offset(a, 0), from = max(mx_offset(a, a.E), first), rows = first + a.R - from;
    const int64_t start = part * blockDim.x + threadIdx.x, step = parts * blockDim.x;
    auto at = [&](int64_t i, int64_t n) { return i < first * n ? i : i + (from - first) * n; };
    if (a.out_codes) {
        const int64_t F = a.N / 2, wide = F / 2, slabs = (F + 255) / 256, n = rows * 8;
        for (int64_t i = start; i < rows * wide; i += step) a.out_codes[at(i, wide)] = 0;
        for (int64_t i = start; i < n * slabs; i += step) a.out_scales[i / n * a.R * 8 + at(i % n, 8)] = 0;
    } else {
        const int64_t wide = a.N * (a.out_dtype == F32 ? 2 : 1);
        uint16_t* o = (uint16_t*)a.out;
        for (int64_t i = start; i < rows * wide; i += step) o[at(i, wide)] = 0;
    }
}

// silu(g) * u in fp32: g (1 / (1 + exp(-g))) u, rounded to four bits next.  exp is
// 2^(-g log2(e)), whose argument is rounded twice, so off by up to |g| 2^-23 of
// itself; the power and the reciprocal are the hardware's (1 ulp; a rounded
// division is ten instructions a value, 2 us a tile of 256 x 128 results).  In all
// (|g| + 4) 2^-23 of the value.  Where the reciprocal falls below 2^-126 (g < -87)
// it is zero.
__device__ __forceinline__ float mx_gated(float g, float u)
{
    return mul_rn(mul_rn(g, __builtin_amdgcn_rcpf(add_rn(1.0f, __expf(-g)))), u);
}

// The scale byte of a block whose largest magnitude has fp32 bits m (255:
// NaN or infinity), as the quantiser computes it.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t m)
{
    const uint32_t ex = m >> 23;
    return ex == 255 ? 255u : ex > 2 ? ex - 2 : 0u;
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
template <int NB>
__device__ __forceinline__ void mx_bias(const Mx4GemmArgs& a, int e, int64_t first, int64_t n, int64_t c, float (&bv)[NB][16])
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

// The epilogue of a wave: rows row0 + 32 mt of the tile, sixteen consecutive
// columns from n0 + c0 + 32 nt in this lane, as pieces of 16 bytes (the columns
// of a row need not be aligned to them).  Range-checked buffer stores, so that
// every wave issues the same number of them, 4 MT times two (fp32: four),
// whatever the tile holds; without a branch between them: two per 32 x 32
// outputs cost 0.5 us a tile of 256 rows, in instructions to fetch.  CUT: the
// piece that the matrix's last column cuts goes out a value at a time (all of a
// row that way: 8192 x 3841 outputs, K = 3840: 162 us, so 93, of 3840: 74).
template <int ODT, int MT, bool BIAS, bool CUT>
__device__ __forceinline__ void mx_put(const Mx4GemmArgs& a, v16f (&acc)[MT][4], int64_t m0, int row0, int rows, int64_t n0,
                                       int c0, int e)
{
    constexpr int ESZ = ODT == F32 ? 4 : 2, PIECE = 16 / ESZ, P = 16 / PIECE;
    const int64_t N = a.N;
    const __amdgpu_buffer_rsrc_t ro =
        mx_rsrc(mx_uniform((const uint8_t*)a.out + (m0 * N + n0) * ESZ), ((int64_t)rows * N - n0) * ESZ);
    const uint32_t rstep = (uint32_t)(32 * N * ESZ), off = (uint32_t)((row0 * N + c0) * ESZ);
    const int left = (int)min(N - n0, (int64_t)256) - c0;   // columns from this lane's first (c0 is a multiple of 16)
    float bv[4][16];
    if constexpr (BIAS) mx_bias<4>(a, e, 0, N, n0 + c0, bv);
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        uint32_t at[P];   // (past the resource, and so with any mt rstep, where the piece is not whole)
#pragma unroll
        for (int p = 0; p < P; ++p)
            at[p] = 32 * nt + PIECE * (p + 1) <= left ? off + (32 * nt + PIECE * p) * ESZ : kOut;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float v[16];
            mx_here(acc[mt][nt]);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = acc[mt][nt][i];
            if constexpr (BIAS) {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = add_rn(v[i], bv[nt][i]);
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                v4u w;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (ODT == F32) w[i] = __float_as_uint(v[4 * p + i]);
                    else w[i] = mx_pack2<ODT>(v[8 * p + 2 * i], v[8 * p + 2 * i + 1]);
                }
                __builtin_amdgcn_raw_buffer_store_b128(w, ro, (int)(at[p] + mt * rstep), 0, 0);
            }
            if constexpr (CUT) {
                const int from = left / PIECE * PIECE - 32 * nt, to = left - 32 * nt;   // of these sixteen columns
                if (row0 + 32 * mt < rows && from >= 0 && from < 16) {
                    char* o = (char*)a.out + ((m0 + row0 + 32 * mt) * N + n0 + c0 + 32 * nt) * ESZ;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i >= from && i < to) store_any(ODT, o, i, v[i]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);   // one tile's values at a time
        }
    }
}

template <int ODT, int MT>
__device__ __forceinline__ void mx_epilogue(const Mx4GemmArgs& a, v16f (&acc)[MT][4], int64_t m0, int row0, int rows,
                                            int64_t n0, int c0, int e)
{
    const bool cut = a.N - n0 < 256 && a.N % (ODT == F32 ? 4 : 8);
    if (a.bias) {
        if (cut) mx_put<ODT, MT, true, true>(a, acc, m0, row0, rows, n0, c0, e);
        else mx_put<ODT, MT, true, false>(a, acc, m0, row0, rows, n0, c0, e);
    } else {
        if (cut) mx_put<ODT, MT, false, true>(a, acc, m0, row0, rows, n0, c0, e);
        else mx_put<ODT, MT, false, false>(a, acc, m0, row0, rows, n0, c0, e);
    }
}

// The gated epilogue of a wave: rows row0 + 32 mt of the tile, results 16 h +
// 32 nt .. + 15 of the wave's 64 (columns tn 128 + wn 64 + ...) in this lane:
// gates in accumulator nt, ups in 2 + nt.  Range-checked stores as above: two of
// codes and one of the two blocks' scale bytes per row tile.  On the last tile,
// which may fill half of its slab only, the other half's bytes become zeros.
template <int MT, bool BIAS>
__device__ __forceinline__ void mx_put_gated(const Mx4GemmArgs& a, v16f (&acc)[MT][4], int64_t m0, int row0, int rows, int tn,
                                             bool last, int wn, int h, int e)
{
    const int64_t F = a.N >> 1, R = a.R;
    const int pitch = (int)(F >> 1);
    const __amdgpu_buffer_rsrc_t rc = mx_rsrc(mx_uniform(a.out_codes + m0 * pitch), (int64_t)rows * pitch);
    const __amdgpu_buffer_rsrc_t rs = mx_rsrc(mx_uniform(a.out_scales + ((int64_t)(tn >> 1) * R + m0) * 8), rows * 8);
    const int64_t fw = (int64_t)tn * 128 + wn * 64 + 16 * h;
    const bool in_f[2] = {fw < F, fw + 32 < F};   // F is a multiple of 32, so are the blocks
    float bg[2][16], bu[2][16];
    if constexpr (BIAS) {
        mx_bias<2>(a, e, 0, F, fw, bg);
        mx_bias<2>(a, e, F, F, fw, bu);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const uint32_t row = row0 + 32 * mt, at = row * pitch + (uint32_t)(fw >> 1);
        uint32_t bytes = 0;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            float v[16];
            uint32_t m = 0;
            mx_here(acc[mt][nt]);
            mx_here(acc[mt][2 + nt]);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float g = acc[mt][nt][i], u = acc[mt][2 + nt][i];
                if constexpr (BIAS) {
                    g = add_rn(g, bg[nt][i]);
                    u = add_rn(u, bu[nt][i]);
                }
                v[i] = mx_gated(g, u);
                m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
            }
            // the block's other sixteen: the two halves of the wave exchanged
            const auto both = __builtin_amdgcn_permlane32_swap(m, m, false, false);
            const uint32_t byte = mx_scale_byte(max(both[0], both[1]));
            const float sc = __uint_as_float(byte << 23);
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                c[p] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[p], v[8 * p + 0], v[8 * p + 1], sc, 0);
                c[p] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[p], v[8 * p + 2], v[8 * p + 3], sc, 1);
                c[p] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[p], v[8 * p + 4], v[8 * p + 5], sc, 2);
                c[p] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[p], v[8 * p + 6], v[8 * p + 7], sc, 3);
                if (byte == 255) c[p] = 0;
            }
            __builtin_amdgcn_raw_buffer_store_b64((v2u){c[0], c[1]}, rc, (int)(in_f[nt] ? at + 16 * nt : kOut), 0, 0);
            bytes |= (in_f[nt] ? byte : 0u) << (8 * nt);
            __builtin_amdgcn_sched_barrier(0);   // one block's values at a time
        }
        const int so = h == 0 ? (int)(row * 8 + (tn & 1) * 4 + wn * 2) : (int)kOut;
        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bytes, rs, so, 0, 0);
        if (last && !(tn & 1)) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)0, rs, so | 4, 0, 0);
    }
}

// ---- the tile kernel ---------------------------------------------------------
// BM x 256 outputs per workgroup of four waves (2 x 2, each BM/2 x 128), K in
// steps of 256; one workgroup per CU, which takes tiles in turn.
//   * A step's codes (128 bytes a row) and scales (8 bytes a row) go global ->
//     LDS by DMA into one of two or three slots, as many steps ahead of their
//     use and, at a tile's end, into the next tiles' steps.  16-byte chunk c of a row sits at
//     c ^ swizzle(row): a ds_read_b128 serves sixteen lanes a cycle (lanes
//     {0-3, 12-15} of one group of sixteen and {4-11} of its neighbour), and
//     these then hit sixteen different 16-byte bank groups.
//   * A step is four quarters (t).  While one quarter's MFMAs run from
//     registers, the fragments of the next are read from LDS.  Before the last
//     quarter the waves wait for the next step's DMA and meet: then nobody
//     reads this step's slot any more, and the DMA furthest ahead goes out
//     into it, half in this quarter and half in the next step's first.
//     Reads, DMA and addresses are dealt out between the MFMAs, whose 32
//     cycles each hide them.
//   * The MFMA takes the weights as first operand, and MFMA row c of a column
//     tile is column 16 ((c >> 2) & 1) + 4 (c >> 3) + (c & 3), so a lane ends
//     with sixteen consecutive columns of one row.
//   * Gated: a wave's 128 columns are 64 gates and the 64 ups that belong to
//     them, so gate, up and the block of 32 results (two lane halves) meet in
//     registers: silu, product, block scale and codes are the epilogue, and
//     the 2 x 16-bit intermediate is never written.
// Bounds (sizes are rows x K x columns).  8192 x 8192 x 8192 246 us = 4.5
// PFLOP/s: the steps of 256-row tiles run at 5.8, the matrix core's rate with
// random codes (the card is then at its power limit; zeros go at 9.6), the rest
// is a tile's end, whose outputs leave in a burst of all CUs.  8192 x 10240 x
// 3840 153 us; 8192 x 3840 x 3840 68 us: 55 without the epilogue, 6 for its
// conversion, 8 for its stores.  Tiles of 128 and 64 rows read more LDS per MFMA
// (a row's step goes at 0.73 and 0.55 of the rate) and are for outputs too few
// to fill the CUs with larger ones: 16396 rows of 32 experts x 3840 x 2560 127
// us; 333 x 5376 x 7168 in fp32 24 us, 168 tiles for 256 CUs.  Gated: 32768 x 3840
// x 2560 183 us.
// Storing a tile's outputs between the next tile's MFMAs, with two sets of
// accumulators, was slower: the compiler moves them between registers.
template <int BM, bool GROUPED, bool GATED>
__global__ __launch_bounds__(256, 1) void mx4_tile_kernel(Mx4GemmArgs a, int tiles_m, int tiles_n)
{
    constexpr int MT = BM / 64, NT = 4;       // 32 x 32 tiles per wave
    // a slot: codes and scales of both operands (256 bytes more for the scale
    // DMA of waves that have no rows, so that all issue the same)
    constexpr int AB = BM * 128, BB = 256 * 128, SAB = BM * 8, SBB = 256 * 8;
    constexpr int SLOT = AB + BB + SAB + SBB + (BM == 64 ? 256 : 0);
    constexpr int SLOTS = BM == 256 ? 2 : 3;  // what LDS holds
    constexpr int AI = BM / 32;               // A DMA instructions per wave (8 rows each)
    constexpr int SAI = BM == 256 ? 2 : 1;    // of A's scales (32 rows each)
    constexpr int DMAS = AI + 8 + SAI + 2;    // all of a step's, per wave
    constexpr int PUTS = GATED ? 3 * MT : 8 * MT;   // stores of an epilogue, at least
    __shared__ __align__(16) uint8_t smem[SLOTS * SLOT];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int j = lane & 31, h = lane >> 5;
    const int wm = wave & 1, wn = wave >> 1;
    const int64_t K = a.K, N = a.N, pitch = K >> 1;
    const int nsteps = (int)((K + 255) / 256);
    const int kblocks = (int)(K >> 5);
    const int64_t F = N >> 1;   // gated: number of results

    // ---- tiles: this workgroup takes number blockIdx.x, + gridDim.x, ...
    struct Tile {
        int m0, rows, tn, e;   // rows 0: none
    };
    int ntiles;
    if constexpr (GROUPED) {
        MxRows r;
        ntiles = (int)mx_find<BM, false>(a, 0, r) * tiles_n;
        mx_zero_rows(a, blockIdx.x, gridDim.x);
    } else {
        ntiles = tiles_m * tiles_n;
    }
    // Lane i of every wave holds the workgroup's i-th tile of a batch of 64:
    // looking tiles up one at a time, in the K loop, cost 5 us a tile.
    Tile mine;
    auto fill = [&](int batch) {
        mine = Tile{0, 0, 0, 0};
        const int64_t at = blockIdx.x + (int64_t)(batch * 64 + lane) * gridDim.x;
        const bool have = at < ntiles;
        // each XCD (workgroup index modulo 8; the grid is a multiple of 8 or
        // the tiles are its first) takes a contiguous range
        const int t = have ? (int)at : 0, q8 = ntiles >> 3, r8 = ntiles & 7, xcd = t & 7;
        const int tile = xcd * q8 + min(xcd, r8) + (t >> 3);
        if constexpr (GROUPED) {
            mx_rows_of<BM>(a, tile, tiles_n, mine.e, mine.m0, mine.tn, mine.rows);
            if (!have) mine.rows = 0;
        } else {
            // groups of four row tiles: an XCD's 32 concurrent tiles span 4 x 8 blocks
            const int per = 4 * tiles_n, grp = tile / per, gm = min(tiles_m - grp * 4, 4), in_g = tile - grp * per;
            mine.m0 = (grp * 4 + in_g % gm) * BM;
            mine.tn = in_g / gm;
            mine.rows = have ? (int)min(a.M - mine.m0, (int64_t)BM) : 0;
        }
    };
    auto tile_of = [&](int i) {
        if (i && !(i & 63)) fill(i >> 6);
        const int l = i & 63;
        return Tile{__builtin_amdgcn_readlane(mine.m0, l), __builtin_amdgcn_readlane(mine.rows, l),
                    __builtin_amdgcn_readlane(mine.tn, l), __builtin_amdgcn_readlane(mine.e, l)};
    };

    // ---- DMA: wave w moves rows [w BM/4, (w + 1) BM/4) of A and 64 weight columns
    const int l8 = lane >> 3, ar0 = wave * (BM / 4);
    // chunk of this lane (bits 1 and 2 of the row decide; bit 3, for columns
    // bit 4, is the instruction's and turns it into its partner ^ 4)
    const int ch = (lane & 7) ^ (l8 >> 1);
    const bool gather = GROUPED && a.rows != nullptr;
    // Every resource is 2^31 bytes long: a lane that has nothing to read (a row
    // or column past the tile's, no tile, a chunk past K) has an offset past
    // that and gets zeros.
    const int slab_a = (int)(a.M * 8), slab_b = (int)(N * 8);   // bytes of a scale slab
    uint32_t avo[AI], bvo[8], savo[SAI], sbvo[2];   // lane offsets of codes and scales
    __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
    auto set_dma = [&](const Tile& t) {
        // the source row of tile row i, or none
        auto src_row = [&](int i) -> int64_t {
            if (i >= t.rows) return -1;
            if (!gather) return i;
            const int64_t s = a.rows[(int64_t)t.m0 + i];
            return s >= 0 && s < a.M ? s : -1;
        };
#pragma unroll
        for (int i = 0; i < AI; ++i) {
            const int64_t s = src_row(ar0 + 8 * i + l8);
            avo[i] = s < 0 ? kOut : (uint32_t)(s * pitch + (ch ^ ((i & 1) * 4)) * 16);
        }
        // scales: 32 rows per instruction, two words each
#pragma unroll
        for (int i = 0; i < SAI; ++i) {
            const int r0 = wave * 32 * SAI + i * 32;
            const int64_t s = r0 < BM ? src_row(r0 + (lane >> 1)) : -1;
            savo[i] = s < 0 ? kOut : (uint32_t)(s * 8 + (lane & 1) * 4);
        }
        ra = mx_rsrc(mx_uniform(gather ? a.a : a.a + (int64_t)t.m0 * pitch), kOut);
        rsa = mx_rsrc(mx_uniform(gather ? a.sa : a.sa + (int64_t)t.m0 * 8), kOut);
        // the wave's 64 weight columns (gated: even waves gates, odd waves ups)
        const int64_t col0 = GATED ? (int64_t)t.tn * 128 + (wave >> 1) * 64 : (int64_t)t.tn * 256 + wave * 64;
        const int64_t ncols = t.rows == 0 ? 0 : GATED ? F : N;
        const int left = (int)(ncols - col0 < 0 ? 0 : ncols - col0 > 64 ? 64 : ncols - col0);
        const int64_t wcol = left == 0 ? 0 : GATED ? (wave & 1) * F + col0 : col0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            bvo[i] = 8 * i + l8 < left ? (uint32_t)((8 * i + l8) * pitch + (ch ^ ((i & 2) * 2)) * 16) : kOut;
#pragma unroll
        for (int i = 0; i < 2; ++i) sbvo[i] = 32 * i + (lane >> 1) < left ? lane * 4u + i * 256u : kOut;
        rb = mx_rsrc(mx_uniform(a.b + ((int64_t)t.e * N + wcol) * pitch), kOut);
        rsb = mx_rsrc(mx_uniform(a.sb + ((int64_t)t.e * nsteps * N + wcol) * 8), kOut);
    };

    // The DMA of one step, an instruction at a time: `Dma` holds what its
    // instructions share.
    struct Dma {
        int ko, soa, sob;    // offsets of the step in a row of codes and in the scales
        uint32_t t0, t1;     // kOut where the chunk, its partner lies past K
    };
    auto dma_chunks = [&](Dma& d, int s) {
        d.t0 = s * 8 < kblocks - ch ? 0u : kOut;
        d.t1 = s * 8 < kblocks - (ch ^ 4) ? 0u : kOut;
    };
    auto dma_offsets = [&](Dma& d, int s) {
        d.ko = s * 128;
        d.soa = s * slab_a;
        d.sob = s * slab_b;
    };
    auto dma = [&](const Dma& d, int sl, int n) {
        if (n < AI) {
            mx_dma<16>(ra, smem + sl + (ar0 + 8 * n) * 128, avo[n < AI ? n : 0] | ((n & 1) ? d.t1 : d.t0), d.ko);
        } else if (n < AI + 8) {
            const int i = n - AI;
            mx_dma<16>(rb, smem + sl + AB + (wave * 64 + 8 * i) * 128, bvo[i & 7] | ((i & 2) ? d.t1 : d.t0), d.ko);
        } else if (n < AI + 8 + SAI) {
            const int i = n - AI - 8, r0 = wave * 32 * SAI + i * 32;
            mx_dma<4>(rsa, smem + sl + AB + BB + (r0 < BM ? r0 * 8 : SAB + SBB), savo[i < SAI ? i : 0], d.soa);
        } else {
            const int i = n - AI - 8 - SAI;
            mx_dma<4>(rsb, smem + sl + AB + BB + SAB + (wave * 64 + i * 32) * 8, sbvo[i & 1], d.sob);
        }
    };
    // The steps of all tiles form one sequence; the DMA runs SLOTS steps, so up
    // to as many tiles, ahead of the MFMAs.
    fill(0);
    Tile cur = tile_of(0), q0{0, 0, 0, 0}, q1 = q0, q2 = q0;
    if (cur.rows == 0) return;
    int t_dma = 0, s_dma = 0, ahead = 0;
    set_dma(cur);
    auto advance = [&]() {
        if (++s_dma < nsteps) return;
        s_dma = 0;
        const Tile t = tile_of(++t_dma);
        set_dma(t);
        // (by value: a choice of addresses would put the queue in memory)
        auto put = [&](Tile& q, bool here) {
            q.m0 = here ? t.m0 : q.m0;
            q.rows = here ? t.rows : q.rows;
            q.tn = here ? t.tn : q.tn;
            q.e = here ? t.e : q.e;
        };
        put(q0, ahead == 0);
        put(q1, ahead == 1);
        if constexpr (SLOTS == 3) put(q2, ahead == 2);
        ++ahead;
    };

    // ---- fragments: row tile mt is rows arow + 32 mt, column tile nt columns
    // bcol + 32 nt, chunk 4h + t
    const int arow = wm * (BM / 2) + j, asw = (j >> 1) & 7;
    const int bc_ = 16 * ((j >> 2) & 1) + 4 * (j >> 3) + (j & 3), bcol = wn * 128 + bc_;
    const int bsw = ((bc_ >> 1) & 3) | (((bc_ >> 4) & 1) << 2);
    const int ao = arow * 128 + ((4 * h) ^ asw) * 16, bo = AB + bcol * 128 + ((4 * h) ^ bsw) * 16;
    const int so_a = AB + BB + arow * 8 + 4 * h, so_b = AB + BB + SAB + bcol * 8 + 4 * h;
    v4i fa[2][MT], fb[2][NT];            // fragments of two quarters
    uint32_t fsa[MT], fsb[NT], nsa[MT], nsb[NT];   // scale words of this step and the next
    constexpr int FR = MT + NT;
    constexpr int NM = MT * NT, NR = NM < FR ? NM : FR;   // MFMAs of a quarter; the first NR are followed by reads
    auto read = [&](int sl, int t, int i) {
        if (i < NT) fb[t & 1][i] = *(const v4i*)(smem + ((sl + bo) ^ (t * 16)) + i * 32 * 128);
        else fa[t & 1][i - NT] = *(const v4i*)(smem + ((sl + ao) ^ (t * 16)) + (i - NT) * 32 * 128);
    };
    auto read_scale = [&](int sl, int i) {
        if (i < NT) nsb[i] = *(const uint32_t*)(smem + sl + so_b + i * 32 * 8);
        else nsa[i - NT] = *(const uint32_t*)(smem + sl + so_a + (i - NT) * 32 * 8);
    };
    // the fragments that follow MFMA k of a quarter: of quarter t of a slot
    auto reads_at = [&](int sl, int t, int k, bool scales) {
        if (k >= NR) return;
#pragma unroll
        for (int i = k * FR / NR; i < (k + 1) * FR / NR; ++i) {
            read(sl, t, i);
            if (scales) read_scale(sl, i);
        }
    };
    auto take_scales = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i) fsb[i] = nsb[i];
#pragma unroll
        for (int i = 0; i < MT; ++i) fsa[i] = nsa[i];
    };

#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        Dma d;
        dma_chunks(d, s_dma);
        dma_offsets(d, s_dma);
#pragma unroll
        for (int n = 0; n < DMAS; ++n) dma(d, s * SLOT, n);
        if (s + 1 < SLOTS) advance();
    }
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((SLOTS - 1) * DMAS) : "memory");   // the first step has landed
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < FR; ++i) {
        read(0, 0, i);
        read_scale(0, i);
    }
    const int row0 = wm * (BM / 2) + j;    // this lane's row (+ 32 mt), and of the
    const int c0 = wn * 128 + 16 * h;      // columns sixteen from c0 + 32 nt
    constexpr int D1 = DMAS / 2;           // DMA instructions of the last quarter; the others follow
    int sl = 0, stores = 0;                // stores: steps in which the last epilogue's may be in flight
    Dma d;
    for (;;) {
        v16f acc[MT][NT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) mx_clear(acc[mt]);
        // the first quarter of the tile's first step (its DMA went out before
        // the last epilogue)
        take_scales();
#pragma unroll
        for (int k = 0; k < NM; ++k) {
            mx_mma<0>(acc[k / NT][k % NT], fb[0][k % NT], fa[0][k / NT], fsb[k % NT], fsa[k / NT]);
            reads_at(sl, 1, k, false);
            __builtin_amdgcn_sched_barrier(0);
        }
        for (int s = 0;;) {
            const int nx = sl == (SLOTS - 1) * SLOT ? 0 : sl + SLOT;
#pragma unroll
            for (int k = 0; k < NM; ++k) {
                mx_mma<1>(acc[k / NT][k % NT], fb[1][k % NT], fa[1][k / NT], fsb[k % NT], fsa[k / NT]);
                reads_at(sl, 2, k, false);
                if (k == NM / 2) advance();
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int k = 0; k < NM; ++k) {
                mx_mma<2>(acc[k / NT][k % NT], fb[0][k % NT], fa[0][k / NT], fsb[k % NT], fsa[k / NT]);
                reads_at(sl, 3, k, false);
                if (k == NM / 2) dma_chunks(d, s_dma);
                if (k == NM * 3 / 4) dma_offsets(d, s_dma);
                __builtin_amdgcn_sched_barrier(0);
            }
            // The next step has landed, and this one is read.  Still in flight
            // may be the DMA of the steps after the next and, in a tile's first
            // SLOTS - 1 steps, the stores of the tile before, which went out
            // after it.
            asm volatile("s_waitcnt lgkmcnt(0)\n\t"
                         "s_cmp_lt_i32 %0, 1\n\t"
                         "s_cbranch_scc1 1f\n\t"
                         "s_waitcnt vmcnt(%1)\n\t"
                         "s_branch 2f\n"
                         "1:\n\t"
                         "s_waitcnt vmcnt(%2)\n"
                         "2:" ::"s"(__builtin_amdgcn_readfirstlane(stores)), "n"((SLOTS - 2) * DMAS + PUTS),
                         "n"((SLOTS - 2) * DMAS)
                         : "memory", "scc");
            --stores;
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < NM; ++k) {
                mx_mma<3>(acc[k / NT][k % NT], fb[1][k % NT], fa[1][k / NT], fsb[k % NT], fsa[k / NT]);
                reads_at(nx, 0, k, true);   // (past the last step: of a slot's older contents, unused)
#pragma unroll
                for (int i = k * D1 / NM; i < (k + 1) * D1 / NM; ++i) dma(d, sl, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (++s == nsteps) break;
            take_scales();
#pragma unroll
            for (int k = 0; k < NM; ++k) {
                mx_mma<0>(acc[k / NT][k % NT], fb[0][k % NT], fa[0][k / NT], fsb[k % NT], fsa[k / NT]);
                reads_at(nx, 1, k, false);
#pragma unroll
                for (int i = D1 + k * (DMAS - D1) / NM; i < D1 + (k + 1) * (DMAS - D1) / NM; ++i) dma(d, sl, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            sl = nx;
        }
#pragma unroll
        for (int i = D1; i < DMAS; ++i) dma(d, sl, i);
        sl = sl == (SLOTS - 1) * SLOT ? 0 : sl + SLOT;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) mx_settle(acc[mt]);

        // ---- epilogue
        if constexpr (GATED) {
            const bool last = cur.tn == tiles_n - 1;
            if (a.bias) mx_put_gated<MT, true>(a, acc, cur.m0, row0, cur.rows, cur.tn, last, wn, h, cur.e);
            else mx_put_gated<MT, false>(a, acc, cur.m0, row0, cur.rows, cur.tn, last, wn, h, cur.e);
        } else {
            const int64_t n0 = (int64_t)cur.tn * 256;
            if (a.out_dtype == BF16) mx_epilogue<BF16, MT>(a, acc, cur.m0, row0, cur.rows, n0, c0, cur.e);
            else if (a.out_dtype == F16) mx_epilogue<F16, MT>(a, acc, cur.m0, row0, cur.rows, n0, c0, cur.e);
            else mx_epilogue<F32, MT>(a, acc, cur.m0, row0, cur.rows, n0, c0, cur.e);
        }
        stores = SLOTS - 1;
        cur = q0;
        q0 = q1;
        if constexpr (SLOTS == 3) q1 = q2;
        --ahead;
        if (cur.rows == 0) break;
    }
}

// ---- the skinny kernel -------------------------------------------------------
// Few rows: the weights are the cost, read once, straight into registers.  A
// workgroup of eight waves takes 16 MT rows.  KW of its waves share the K
// steps of one group of 16 NT columns (gated, NT = 4: 32 gates and their 32
// ups, one block of results); 8 / KW groups lie side by side.  The waves'
// partial sums meet in LDS and are added in wave order.
// Bound by the weights' bytes and, up to a few megabytes of them, by latency:
// 3840 x 3840 weights (7.8 MB) with one row 4.2 us, 10240 x 10240 (56 MB) 14.9 to
// 15.6 us = 3.7 TB/s; 64 rows 27.4 to 28.4 us, each column group reading the rows again.
constexpr int kSkinnyWaves = 8;
template <int MT, int NT, int KW, bool GROUPED, bool GATED>
__global__ __launch_bounds__(512) void mx4_skinny_kernel(Mx4GemmArgs a)
{
    static_assert(!GATED || NT == 4, "a block of gates and its ups");
    constexpr int W = kSkinnyWaves, CG = W / KW;
    constexpr int COLS = GATED ? 32 : 16 * NT;   // results of a column group
    __shared__ float part[W][MT][NT][16][17];    // [wave][row tile][column tile][row][column]
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int kw = wave % KW, cg = wave / KW;
    const int j = lane & 15, q = lane >> 4;
    const int64_t K = a.K, N = a.N, F = N >> 1, pitch = K >> 1;
    const int64_t n = GATED ? F : N;             // results of a row
    const int nsteps = (int)((K + 255) / 256);
    int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    int rows, e = 0;
    if constexpr (GROUPED) {
        MxRows r;
        const int64_t total = mx_find<16 * MT, true>(a, blockIdx.y, r);
        if (r.e < 0) {
            mx_zero_rows(a, (int64_t)(blockIdx.y - total) * gridDim.x + blockIdx.x, (int64_t)(gridDim.y - total) * gridDim.x);
            return;
        }
        const int m = (int)(blockIdx.y - r.before);
        e = r.e;
        m0 = r.m0 + (int64_t)m * (16 * MT);
        rows = min(r.rows - m * 16 * MT, 16 * MT);
    } else {
        rows = (int)min(a.M - m0, (int64_t)(16 * MT));
    }
    const uint8_t* wb = a.b + (int64_t)e * N * pitch;
    const uint8_t* wsb = a.sb + (int64_t)e * nsteps * N * 8;
    const int kblocks = (int)(K >> 5);
    const int64_t first = ((int64_t)blockIdx.x * CG + cg) * COLS;   // the group's first result
    // this lane's weight columns and rows (clamped: what they give is not stored)
    int64_t col[NT], src[MT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int64_t c = first + (GATED ? (nt & 1) : nt) * 16 + j;
        col[nt] = (c < n ? c : n - 1) + (GATED ? (nt >> 1) * F : 0);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int i = 16 * mt + j;
        int64_t s = m0 + (i < rows ? i : rows - 1);
        bool ok = true;
        if (GROUPED && a.rows) {
            s = a.rows[s];
            ok = s >= 0 && s < a.M;
        }
        src[mt] = ok ? s : -1;
    }
    v4f acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = (v4f){0.f, 0.f, 0.f, 0.f};
    constexpr int U = NT * MT > 4 ? 1 : 2;     // steps in flight
    for (int s0 = kw; s0 < nsteps; s0 += KW * U) {
        v4i fb[U][NT][2], fa[U][MT][2];
        uint32_t sb[U][NT], sa[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + KW * u;
            const bool in = s < nsteps;
            const int b0 = s * 8 + 2 * q;        // this lane's two blocks
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const v4i* p = (const v4i*)(wb + col[nt] * pitch) + b0;
                fb[u][nt][0] = in && b0 < kblocks ? p[0] : (v4i){0, 0, 0, 0};
                fb[u][nt][1] = in && b0 + 1 < kblocks ? p[1] : (v4i){0, 0, 0, 0};
                sb[u][nt] = in ? *(const uint16_t*)(wsb + ((int64_t)s * N + col[nt]) * 8 + 2 * q) : 0;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const bool ok = in && src[mt] >= 0;
                const v4i* p = (const v4i*)(a.a + src[mt] * pitch) + b0;
                fa[u][mt][0] = ok && b0 < kblocks ? p[0] : (v4i){0, 0, 0, 0};
                fa[u][mt][1] = ok && b0 + 1 < kblocks ? p[1] : (v4i){0, 0, 0, 0};
                sa[u][mt] = ok ? *(const uint16_t*)(a.sa + ((int64_t)s * a.M + src[mt]) * 8 + 2 * q) : 0;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    acc[mt][nt] = mx_mfma<0, 0>(fb[u][nt][0], fa[u][mt][0], acc[mt][nt], sb[u][nt], sa[u][mt]);
                    acc[mt][nt] = mx_mfma<1, 1>(fb[u][nt][1], fa[u][mt][1], acc[mt][nt], sb[u][nt], sa[u][mt]);
                }
    }
    // lane (j, q): row j of the row tile, columns 4q .. 4q + 3 of the column tile
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) part[wave][mt][nt][j][4 * q + r] = acc[mt][nt][r];
    __syncthreads();
    const int waves = nsteps < KW ? nsteps : KW;   // those that had a step
    auto sum = [&](int g, int mt, int nt, int row, int c) {
        float v = part[g * KW][mt][nt][row][c];
        for (int w = 1; w < waves; ++w) v = add_rn(v, part[g * KW + w][mt][nt][row][c]);
        return v;
    };
    if constexpr (GATED) {
        // a half wave takes the 32 results of one row of one group
        const int c = tid & 31;
        const int64_t R = a.R;
        for (int i = tid >> 5; i < 16 * MT * CG; i += 16) {
            const int row = i % (16 * MT), g_ = i / (16 * MT), mt = row >> 4;
            const int64_t f = ((int64_t)blockIdx.x * CG + g_) * 32 + c;
            if (f >= F || row >= rows) continue;   // (whole half waves)
            float g = sum(g_, mt, c >> 4, row & 15, c & 15), u = sum(g_, mt, 2 + (c >> 4), row & 15, c & 15);
            if (a.bias) {
                g = add_rn(g, load_any_f32(a.bias_dtype, a.bias, (int64_t)e * N + f));
                u = add_rn(u, load_any_f32(a.bias_dtype, a.bias, (int64_t)e * N + F + f));
            }
            const float v = mx_gated(g, u);
            uint32_t m = __float_as_uint(v) & 0x7fffffffu;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
            const uint32_t byte = mx_scale_byte(m);
            const float hi = __shfl_down(v, 1);
            uint32_t cc = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v, hi, __uint_as_float(byte << 23), 0);
            if (byte == 255) cc = 0;
            if (!(c & 1)) a.out_codes[((m0 + row) * F + f) / 2] = (uint8_t)cc;
            if (c == 0) {
                const int64_t blk = f >> 5;
                uint8_t* o = a.out_scales + ((blk >> 3) * R + m0 + row) * 8;
                o[blk & 7] = (uint8_t)byte;
                // the last block also clears what is left of its slab
                if (blk == (F >> 5) - 1)
                    for (int b = (int)(blk & 7) + 1; b < 8; ++b) o[b] = 0;
            }
        }
    } else {
        constexpr int WG = CG * COLS;
        for (int i = tid; i < 16 * MT * WG; i += 512) {
            const int row = i / WG, c = i % WG, g = c / COLS, nt = (c % COLS) >> 4;
            const int64_t nn = (int64_t)blockIdx.x * WG + c;
            if (nn < N && row < rows) {
                float v = sum(g, row >> 4, nt, row & 15, c & 15);
                if (a.bias) v = add_rn(v, load_any_f32(a.bias_dtype, a.bias, (int64_t)e * N + nn));
                store_any(a.out_dtype, a.out, (m0 + row) * N + nn, v);
            }
        }
    }
}

// One workgroup per CU (LDS holds one), which takes tiles in turn.
constexpr int64_t kTileGrid = 256;

template <int BM> hipError_t launch_tile(const Mx4GemmArgs& a, hipStream_t st)
{
    const bool gated = a.out_codes != nullptr;
    const int64_t tn = gated ? (a.N / 2 + 127) / 128 : (a.N + 255) / 256;
    // (grouped: at most this many, the device knows)
    const int64_t tm = a.E ? a.R / BM + (a.E < a.R ? a.E : a.R) : (a.M + BM - 1) / BM;
    const unsigned grid = (unsigned)(tm * tn < kTileGrid ? tm * tn : kTileGrid);
    if (!a.E)
        hipLaunchKernelGGL((mx4_tile_kernel<BM, false, false>), dim3(grid), dim3(256), 0, st, a, (int)tm, (int)tn);
    else if (gated)
        hipLaunchKernelGGL((mx4_tile_kernel<BM, true, true>), dim3(grid), dim3(256), 0, st, a, 0, (int)tn);
    else
        hipLaunchKernelGGL((mx4_tile_kernel<BM, true, false>), dim3(grid), dim3(256), 0, st, a, 0, (int)tn);
    return hipGetLastError();
}

int skinny_rows(const Mx4GemmArgs& a)
{
    const int64_t rows = a.E ? (a.R + a.E - 1) / a.E : a.M;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// 64 columns a group: a single pass of more than 16 rows whose groups of 32
// would be more than the CUs; the rows are read half as often (10240 x 10240
// weights, 32 and 64 rows: 19.9 and 27.4 us against 23.8 and 34.5; with several
// passes or shorter K nothing or a loss: 128 rows 51.6 : 49.1, K = 1280 64 rows
// 13.5 : 10.5).
bool skinny_wide(const Mx4GemmArgs& a) { return !a.E && a.M > 16 && a.M <= 64 && a.K > 1792 && a.N > 32 * 256; }

template <int MT, int NT, int KW, bool GATED, bool GROUPED = true> hipError_t launch_skinny_w(const Mx4GemmArgs& a, hipStream_t st)
{
    constexpr int COLS = (GATED ? 32 : 16 * NT) * (kSkinnyWaves / KW);
    const int64_t n = GATED ? a.N / 2 : a.N;
    const unsigned tn = (unsigned)((n + COLS - 1) / COLS);
    if (GROUPED && a.E) {
        if constexpr (GROUPED) {
            const unsigned tm = (unsigned)(a.R / (16 * MT) + (a.E < a.R ? a.E : a.R) + 1);
            hipLaunchKernelGGL((mx4_skinny_kernel<MT, NT, KW, true, GATED>), dim3(tn, tm), dim3(512), 0, st, a);
        }
    } else if constexpr (!GATED) {
        hipLaunchKernelGGL((mx4_skinny_kernel<MT, NT, KW, false, false>), dim3(tn, (unsigned)((a.M + 16 * MT - 1) / (16 * MT))),
                           dim3(512), 0, st, a);
    }
    return hipGetLastError();
}

template <int MT> hipError_t launch_skinny(const Mx4GemmArgs& a, hipStream_t st)
{
    // half the waves per column group where K has few steps for eight of them
    const bool deep = a.K > 1792;
    if (a.out_codes) return deep ? launch_skinny_w<MT, 4, 8, true>(a, st) : launch_skinny_w<MT, 4, 4, true>(a, st);
    // 32 columns a group once 16 would make more workgroups than the CUs hold
    if constexpr (MT > 1)
        if (skinny_wide(a)) return launch_skinny_w<MT, 4, 8, false, false>(a, st);
    const bool narrow = !a.E && (a.N + 15) / 16 * ((a.M + 16 * MT - 1) / (16 * MT)) <= 512;
    if (narrow) return deep ? launch_skinny_w<MT, 1, 8, false>(a, st) : launch_skinny_w<MT, 1, 4, false>(a, st);
    return deep ? launch_skinny_w<MT, 2, 8, false>(a, st) : launch_skinny_w<MT, 2, 4, false>(a, st);
}

}  // namespace

namespace {

// Estimated microseconds of each kernel.  Tiles: the 256 workgroups take them
// in rounds; a step (256 k) of a 64, 128, 256 row tile measured 0.66, 1.0,
// 1.46 us with all CUs busy, and a tile's beginning and end 3.7, 4.2, 9.4 us
// (16384 x 2560 outputs at K = 3840 and 7680: 136 and 235, 96 and 171, 95 and
// 161 us; at other shapes the choice can be wrong: 768 rows of each of 8 experts
// of 3840 x 2560 take tiles of 64 rows, 54 us where 128 and 256 take 42 and 40).
// Skinny: 2.5 us, then weights at 5 TB/s and, for each column group,
// the rows again at 6 TB/s (10240 x 10240 weights with 1, 16, 32, 64 rows:
// 14.9, 18.3, 19.9, 27.4 us).  The groups' sizes are on the device: all are
// taken to have the mean, and to fill half of their last tile.
double tile_us(const Mx4GemmArgs& a, int bm, double step, double ends)
{
    const double tn = a.out_codes ? (double)((a.N / 2 + 127) / 128) : (double)((a.N + 255) / 256);
    double tm = (double)((a.M + bm - 1) / bm);
    if (a.E) {
        const double groups = (double)(a.E < a.R ? a.E : a.R);
        tm = (double)a.R / bm + 0.5 * groups;
        if (tm < groups * 0.7) tm = groups * 0.7;
    }
    // (a single group's estimate of less than a tile is still a tile: 3840 x 96
    // weights of one expert and one row 13.9 us so, 5.1 with the skinny kernel)
    const double rounds = tm * tn < 1 ? 1 : (double)(int64_t)((tm * tn + 255) / 256);
    return rounds * ((double)((a.K + 255) / 256) * step + ends);
}

double skinny_us(const Mx4GemmArgs& a)
{
    const int rows = skinny_rows(a);
    double passes = (double)((a.M + rows - 1) / rows);
    if (a.E) {
        const double groups = (double)(a.E < a.R ? a.E : a.R);
        passes = (double)a.R / rows + 0.5 * groups;
        if (passes < groups * 0.7) passes = groups * 0.7;
    }
    const double weights = (double)a.N * (double)a.K * 17 / 32 * 1e-6;   // MB
    return 2.5 + passes * weights * (1 / 5.0 + (double)rows / (a.out_codes || skinny_wide(a) ? 64 : 32) / 6.0);
}

}  // namespace

int mx4_gemm_path(const Mx4GemmArgs& a)
{
    const double t[4] = {skinny_us(a), tile_us(a, 64, 0.66, 3.7), tile_us(a, 128, 1.0, 4.2), tile_us(a, 256, 1.46, 9.4)};
    const int64_t rows = a.E ? (a.R + a.E - 1) / a.E : a.M;
    // Tiles of 256 rows are two steps ahead in their weights, the others three:
    // not enough where a group's weights serve a few tiles only.  Ragged groups
    // of 32 experts of 3840 x 2560 with a mean of 384, 512, 768, 1024, 1536 rows:
    // 94, 116, 169, 220, 325 us with 128 rows a tile, 97, 134, 178, 222, 313 with
    // 256; of 16 of 7680 x 2560 93, 101, 164, 201, 285 and 101, 111, 171, 182,
    // 261.  (Gated with 768 rows 156 : 144, and equal groups can go the other way:
    // 768 rows 167 : 152, 512 104 : 111.)
    const int last = a.E && rows < 1024 ? kMx4Tile128 : kMx4Tile256;
    int best = kMx4Tile64;
    for (int i = kMx4Tile128; i <= last; ++i)
        if (t[i] < t[best]) best = i;
    // A tile's outputs are addressed with 31 bits: rows of 8 MB and more are the
    // skinny kernel's.
    if (a.N * (a.out_codes ? 1 : a.out_dtype == F32 ? 4 : 2) >= (int64_t)1 << 23) return kMx4Skinny;
    // (past 128 rows a weight column would be read three times and more)
    return rows <= 128 && t[kMx4Skinny] < t[best] ? kMx4Skinny : best;
}

hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, hipStream_t st)
{
    switch (mx4_gemm_path(a)) {
    case kMx4Tile256: return launch_tile<256>(a, st);
    case kMx4Tile128: return launch_tile<128>(a, st);
    case kMx4Tile64: return launch_tile<64>(a, st);
    }
    const int rows = skinny_rows(a);
    return rows == 16 ? launch_skinny<1>(a, st) : rows == 32 ? launch_skinny<2>(a, st) : launch_skinny<4>(a, st);
}

}  // namespace w4a4
