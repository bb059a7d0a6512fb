// The block-scaled fp8 product
//   out[m][n] = sum_b sa[b][m] sw[n / 128][b] (sum_{k in block b} a[m][k] w[n][k]) (+ bias[n])
// on gfx950's f8f6f4 matrix cores, dense and grouped by expert.
//
// Mathematics.  v_mfma_f32_16x16x128_f8f6f4 multiplies 16 x 128 by 128 x 16 e4m3
// values: one block of k.  It starts from zero, and its fp32 result joins the
// accumulators with one fma per output, times the product of the two scales.  The
// weights are the first operand, so a lane (j, q) ends with columns 4q .. 4q + 3 of
// one row j of a 16 x 16 tile, and a single factor serves all of a row's columns
// that share a weight block.  A lane supplies 32 k of one row; which 32 is free as
// long as both operands agree.
//
// Precision.  The fp8 matrix core adds the products of eight neighbouring k in fixed
// point, 2^-13 of the largest of them the last place (measured: a product of 2^-14
// beside one of 1 is lost inside such a group, kept outside it), and the groups in
// fp32.  That is 1.4e-5 of the outputs (rms, rows of equal spread), 3.5e-5 where one
// channel in fifty is 20 times the others and 6.4e-5 where one in 128 is 400 times, since
// the last place follows the largest of eight.  Rounding to bf16 is 1.66e-3 and to fp16
// 2.08e-4, so with it an output is 0.2% at most and 0.2%, 1.4% and 5% further off than
// rounding alone: such outputs take the fp8 core.  Where the output is fp32 it would be
// the largest error of all, and in a gated product it would move one code in two thousand
// over a border (an error of its own of 1e-3 where the codes are the result).  Those
// products (Fp8GemmArgs::half) convert the codes (exactly) to fp16, whose matrix core
// (16x16x32, half the rate) adds in fp32: outputs are 6e-8, 1.0e-7 and 1.6e-7 off at K =
// 1280, 3840 and 10240, where rounding to fp32 alone is 2.5e-8.
#include <type_traits>

#include "common.hpp"
#include "fp8.hpp"
#include "fp8_codes.hpp"
#include "grouped.hpp"

namespace w4a4 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

// 16 x 16 outputs of one block of 128 k, from zero
__device__ __forceinline__ v4f fp8_mfma(v8i w, v8i a)
{
    const v4f z = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, z, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v8i join(v4i lo, v4i hi)
{
    return (v8i){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// The lane's 32 codes as fp16, four operands of the 16x16x32 instruction
typedef int v16i __attribute__((ext_vector_type(16)));
__device__ __forceinline__ v16i fp8_to_f16(v8i c)
{
    // (written out: a loop over the elements would put the fragments in memory)
#define FP8_F16(i) __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[(i) >> 1], 1.0f, (i) & 1))
    return (v16i){FP8_F16(0), FP8_F16(1), FP8_F16(2), FP8_F16(3), FP8_F16(4), FP8_F16(5), FP8_F16(6), FP8_F16(7),
                  FP8_F16(8), FP8_F16(9), FP8_F16(10), FP8_F16(11), FP8_F16(12), FP8_F16(13), FP8_F16(14), FP8_F16(15)};
#undef FP8_F16
}
__device__ __forceinline__ v4f f16_mfma(v16i w, v16i a)
{
#define FP8_QUARTER(v, t) __builtin_bit_cast(v8h, __builtin_shufflevector(v, v, 4 * t, 4 * t + 1, 4 * t + 2, 4 * t + 3))
    v4f d = {0.f, 0.f, 0.f, 0.f};
    d = __builtin_amdgcn_mfma_f32_16x16x32_f16(FP8_QUARTER(w, 0), FP8_QUARTER(a, 0), d, 0, 0, 0);
    d = __builtin_amdgcn_mfma_f32_16x16x32_f16(FP8_QUARTER(w, 1), FP8_QUARTER(a, 1), d, 0, 0, 0);
    d = __builtin_amdgcn_mfma_f32_16x16x32_f16(FP8_QUARTER(w, 2), FP8_QUARTER(a, 2), d, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(FP8_QUARTER(w, 3), FP8_QUARTER(a, 3), d, 0, 0, 0);
#undef FP8_QUARTER
}

// Zeros for the sorted rows that no expert owns (before offsets[0] and from
// offsets[E] on), spread over all workgroups, each before its first tile.
__device__ __forceinline__ void fp8_zero_rows(const Fp8GemmArgs& a, int64_t part, int64_t parts)
{
    const int64_t first = mx_offset(a, 0), from = max(mx_offset(a, a.E), first), rows = first + a.R - from;
    const int64_t start = part * blockDim.x + threadIdx.x, step = parts * blockDim.x;
    auto at = [&](int64_t i, int64_t n) { return i < first * n ? i : i + (from - first) * n; };
    if (a.out_codes) {
        const int64_t F = a.N / 2, blocks = F / kFp8Block;
        for (int64_t i = start; i < rows * F; i += step) a.out_codes[at(i, F)] = 0;
        for (int64_t i = start; i < rows * blocks; i += step) a.out_scales[i / rows * a.R + at(i % rows, 1)] = 0.0f;
    } else {
        const int64_t wide = a.N * (a.out_dtype == F32 ? 2 : 1);
        uint16_t* o = (uint16_t*)a.out;
        for (int64_t i = start; i < rows * wide; i += step) o[at(i, wide)] = 0;
    }
}

// ---- the skinny kernel -------------------------------------------------------
// Few rows, dense: the weights are the cost, read once, straight into registers.  A
// workgroup of eight waves takes 16 MT rows; KW of its waves share the K steps of one
// group of 16 NT columns, 8 / KW groups lie side by side.  Partial sums meet in LDS
// and are added in wave order.  The matrix cores wait for memory here, so all types
// take the fp16 products.
// Bound by the weights' bytes and, up to a few megabytes of them, by latency: 3840 x
// 3840 weights with one row 5.0 us, 10240 x 10240 (105 MB) 21 us = 5 TB/s, with 32 rows
// 44 us, each column group reading the rows again.
// (Grouped by expert, 64-row tiles are as fast or faster from one row an expert on: 32
// experts of 3840 x 2560, a mean of 1, 4, 16 rows: 24, 62, 68 us where this kernel's
// grouped form took 24, 62, 89.)
constexpr int kSkinnyWaves = 8;
template <int MT, int NT, int KW> __global__ __launch_bounds__(512) void fp8_skinny_kernel(Fp8GemmArgs a)
{
    constexpr int W = kSkinnyWaves, CG = W / KW, COLS = 16 * NT;
    __shared__ float part[W][MT][NT][16][17];    // [wave][row tile][column tile][row][column]
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int kw = wave % KW, cg = wave / KW;
    const int j = lane & 15, q = lane >> 4;
    const int64_t K = a.K, N = a.N;
    const int nsteps = (int)fp8_blocks(K);
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    const int rows = (int)min(a.M - m0, (int64_t)(16 * MT));
    const int64_t first = ((int64_t)blockIdx.x * CG + cg) * COLS;   // the group's first column
    // this lane's weight columns and rows (clamped: what they give is not stored)
    int64_t col[NT], src[MT];
    const float* ws[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int64_t c = first + nt * 16;
        col[nt] = min(c + j, N - 1);
        ws[nt] = a.sb + min(c, N - 1) / kFp8Block * nsteps;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) src[mt] = m0 + min(16 * mt + j, rows - 1);
    v4f acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = (v4f){0.f, 0.f, 0.f, 0.f};
    constexpr int U = NT * MT > 4 ? 1 : 2;     // steps in flight
    for (int s0 = kw; s0 < nsteps; s0 += KW * U) {
        v4i fb[U][NT][2], fa[U][MT][2];
        float sw[U][NT], sa[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + KW * u;
            const bool in = s < nsteps;
            const int64_t k = (int64_t)s * kFp8Block + 32 * q;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint8_t* p = a.b + col[nt] * K + k;
                fb[u][nt][0] = in && k < K ? *(const v4i*)p : (v4i){0, 0, 0, 0};
                fb[u][nt][1] = in && k + 16 < K ? *(const v4i*)(p + 16) : (v4i){0, 0, 0, 0};
                sw[u][nt] = in ? ws[nt][s] : 0.0f;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const uint8_t* p = a.a + src[mt] * K + k;
                fa[u][mt][0] = in && k < K ? *(const v4i*)p : (v4i){0, 0, 0, 0};
                fa[u][mt][1] = in && k + 16 < K ? *(const v4i*)(p + 16) : (v4i){0, 0, 0, 0};
                sa[u][mt] = in ? a.sa[(int64_t)s * a.M + src[mt]] : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const v4f p = f16_mfma(fp8_to_f16(join(fb[u][nt][0], fb[u][nt][1])), fp8_to_f16(join(fa[u][mt][0], fa[u][mt][1])));
                    const float f = mul_rn(sa[u][mt], sw[u][nt]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[mt][nt][r] = __builtin_fmaf(p[r], f, acc[mt][nt][r]);
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
    constexpr int WG = CG * COLS;
    for (int i = tid; i < 16 * MT * WG; i += 512) {
        const int row = i / WG, c = i % WG, g = c / COLS, nt = (c % COLS) >> 4, mt = row >> 4;
        const int64_t nn = (int64_t)blockIdx.x * WG + c;
        if (nn < N && row < rows) {
            float v = part[g * KW][mt][nt][row & 15][c & 15];
            for (int w = 1; w < waves; ++w) v = add_rn(v, part[g * KW + w][mt][nt][row & 15][c & 15]);
            if (a.bias) v = add_rn(v, load_any_f32(a.bias_dtype, a.bias, nn));
            store_any(a.out_dtype, a.out, (m0 + row) * N + nn, v);
        }
    }
}

// ---- the tile kernel ---------------------------------------------------------
// The epilogue of a wave: rows row0 + 16 mt of the tile, columns n0 + c0 .. + 7 and
// n0 + c0 + 32 .. + 39 in this lane, as pieces of 16 bytes (four lanes: 64 bytes of a
// row; the columns of a row need not be aligned to them).  Range-checked buffer stores,
// so that every wave issues the same number of them whatever the tile holds.  CUT: the
// piece that the matrix's last column cuts goes out a value at a time.
template <int ODT, int MT, bool BIAS, bool CUT>
__device__ __forceinline__ void fp8_put(const Fp8GemmArgs& a, const v4f (&acc)[MT][4], int64_t m0, int row0, int rows,
                                        int64_t n0, int c0, int e)
{
    constexpr int ESZ = ODT == F32 ? 4 : 2, PIECE = 16 / ESZ, P = 16 / PIECE;
    const int64_t N = a.N;
    const __amdgpu_buffer_rsrc_t ro =
        mx_rsrc(mx_uniform((const uint8_t*)a.out + (m0 * N + n0) * ESZ), ((int64_t)rows * N - n0) * ESZ);
    const uint32_t rstep = (uint32_t)(16 * N * ESZ), off = (uint32_t)((row0 * N + c0) * ESZ);
    const int left = (int)min(N - n0, (int64_t)256) - c0;   // columns from this lane's first
    auto col = [](int i) { return i < 8 ? i : i + 24; };    // of value i
    float bv[2][16];
    if constexpr (BIAS) mx_bias<2>(a, e, 0, N, n0 + c0, bv);   // (columns c0 .. + 15 and c0 + 32 .. + 47)
    uint32_t at[P];   // (past the resource, and so with any mt rstep, where the piece is not whole)
#pragma unroll
    for (int p = 0; p < P; ++p) at[p] = col(PIECE * p) + PIECE <= left ? off + col(PIECE * p) * ESZ : kOut;
    v4f b4[4];
    if constexpr (BIAS) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            b4[i] = (v4f){bv[i >> 1][4 * (i & 1)], bv[i >> 1][4 * (i & 1) + 1], bv[i >> 1][4 * (i & 1) + 2], bv[i >> 1][4 * (i & 1) + 3]};
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        auto plus = [&](v4f x, int i) {
            if constexpr (BIAS) x = (v4f){add_rn(x[0], b4[i][0]), add_rn(x[1], b4[i][1]), add_rn(x[2], b4[i][2]), add_rn(x[3], b4[i][3])};
            return x;
        };
        v4f c0_ = plus(acc[mt][0], 0), c1_ = plus(acc[mt][1], 1), c2_ = plus(acc[mt][2], 2), c3_ = plus(acc[mt][3], 3);
        // (values from here on: a choice among their addresses would put all in memory)
        asm volatile("" : "+v"(c0_), "+v"(c1_), "+v"(c2_), "+v"(c3_));
        auto four = [&](int i) { return i == 0 ? c0_ : i == 1 ? c1_ : i == 2 ? c2_ : c3_; };
#pragma unroll
        for (int p = 0; p < P; ++p) {
            v4u w;
            if constexpr (ODT == F32) {
                w = __builtin_bit_cast(v4u, four(p & 3));
            } else {
                const v4f x = four(2 * (p & 1)), y = four(2 * (p & 1) + 1);
                w = (v4u){mx_pack2<ODT>(x[0], x[1]), mx_pack2<ODT>(x[2], x[3]), mx_pack2<ODT>(y[0], y[1]), mx_pack2<ODT>(y[2], y[3])};
            }
            // not temporal: the outputs would drive operands out of the L2 (32 experts'
            // 32768 rows, K 1280, N 3840: 210 -> 201 us; the dense products the same)
            __builtin_amdgcn_raw_buffer_store_b128(w, ro, (int)(at[p] + mt * rstep), 0, 2);
        }
        if constexpr (CUT) {
            if (row0 + 16 * mt < rows) {
                char* o = (char*)a.out + ((m0 + row0 + 16 * mt) * N + n0 + c0) * ESZ;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (col(i) < left && col(i / PIECE * PIECE) + PIECE > left) store_any(ODT, o, col(i), four(i >> 2)[i & 3]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);   // one row tile's values at a time
    }
}

template <int ODT, int MT>
__device__ __forceinline__ void fp8_epilogue(const Fp8GemmArgs& a, const v4f (&acc)[MT][4], int64_t m0, int row0, int rows,
                                             int64_t n0, int c0, int e)
{
    const bool cut = a.N - n0 < 256 && a.N % (ODT == F32 ? 4 : 8);
    if (a.bias) {
        if (cut) fp8_put<ODT, MT, true, true>(a, acc, m0, row0, rows, n0, c0, e);
        else fp8_put<ODT, MT, true, false>(a, acc, m0, row0, rows, n0, c0, e);
    } else {
        if (cut) fp8_put<ODT, MT, false, true>(a, acc, m0, row0, rows, n0, c0, e);
        else fp8_put<ODT, MT, false, false>(a, acc, m0, row0, rows, n0, c0, e);
    }
}

// The gated epilogue of a wave: rows row0 + 16 mt of the tile, results 8 q .. + 7 of
// the wave's 32 in this lane, gates in accumulators 0 and 1, ups in 2 and 3.  Four
// waves make a block of 128 results, whose largest magnitude they find in LDS (top:
// [wm][wn][row]); the stores are range-checked.
template <int BM, bool BIAS>
__device__ __forceinline__ void fp8_put_gated(const Fp8GemmArgs& a, v4f (&acc)[BM / 32][4], int64_t m0, int rows, int tn,
                                              int wm, int wn, int j, int q, int e, uint32_t* top)
{
    constexpr int MT = BM / 32;
    const int64_t F = a.N >> 1;
    const int row0 = wm * (BM / 2) + j;
    const int64_t f = (int64_t)tn * kFp8Block + wn * 32 + 8 * q;   // the lane's first result
    const __amdgpu_buffer_rsrc_t rc = mx_rsrc(mx_uniform(a.out_codes + m0 * F), (int64_t)rows * F);
    const __amdgpu_buffer_rsrc_t rs = mx_rsrc(mx_uniform((const uint8_t*)(a.out_scales + (int64_t)tn * a.R + m0)), rows * 4);
    float bg[1][16], bu[1][16];
    if constexpr (BIAS) {
        mx_bias<1>(a, e, 0, F, f, bg);
        mx_bias<1>(a, e, F, F, f, bu);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        uint32_t m = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v4f g = acc[mt][h], u = acc[mt][2 + h];
            asm volatile("" : "+v"(g), "+v"(u));
            if constexpr (BIAS) {
                g = (v4f){add_rn(g[0], bg[0][4 * h]), add_rn(g[1], bg[0][4 * h + 1]), add_rn(g[2], bg[0][4 * h + 2]), add_rn(g[3], bg[0][4 * h + 3])};
                u = (v4f){add_rn(u[0], bu[0][4 * h]), add_rn(u[1], bu[0][4 * h + 1]), add_rn(u[2], bu[0][4 * h + 2]), add_rn(u[3], bu[0][4 * h + 3])};
            }
            const v4f v = {mx_gated(g[0], u[0]), mx_gated(g[1], u[1]), mx_gated(g[2], u[2]), mx_gated(g[3], u[3])};
            acc[mt][h] = v;
#pragma unroll
            for (int r = 0; r < 4; ++r) m = max(m, __float_as_uint(v[r]) & 0x7fffffffu);
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (q == 0) top[(wm * 4 + wn) * (BM / 2) + 16 * mt + j] = m;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        uint32_t m = top[wm * 4 * (BM / 2) + 16 * mt + j];
#pragma unroll
        for (int w = 1; w < 4; ++w) m = max(m, top[(wm * 4 + w) * (BM / 2) + 16 * mt + j]);
        const Fp8Block b = fp8_block(m);
        v2u c;
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = fp8_codes4(b, acc[mt][i][0], acc[mt][i][1], acc[mt][i][2], acc[mt][i][3]);
        const uint32_t row = (uint32_t)(row0 + 16 * mt);
        __builtin_amdgcn_raw_buffer_store_b64(c, rc, (int)(row * (uint32_t)F + (uint32_t)f), 0, 0);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(b.scale), rs, wn == 0 && q == 0 ? (int)(row * 4) : (int)kOut, 0, 0);
    }
}

// BM x 256 outputs per workgroup of eight waves (2 x 4, each BM/2 x 64, two to a
// SIMD: with one wave the matrix core would wait for the fmas that read its results),
// K in steps of 128, a scale block; one workgroup per CU, which takes tiles in turn.
//   * A step's codes (128 bytes a row) go global -> LDS by DMA into one of two or three
//     slots, its scales into one more slot of their own, and at a tile's end those of
//     the next tiles' steps.  16-byte chunk c of LDS row r sits at c ^ ((r >> 1) & 7): a
//     ds_read_b128 serves sixteen lanes a cycle (lanes {0-3, 12-15} of one group of
//     sixteen and {4-11} of its neighbour), and these then hit sixteen different
//     16-byte bank groups.
//   * A wave holds all its weight fragments of a step (four column tiles) and walks
//     the row tiles, whose fragments are read one tile ahead.  Before every fourth row
//     tile the waves wait for what the next two need and meet: then nobody reads the
//     last two's rows any more (before the second: nor the weights), and the DMA of the
//     step that takes this slot next goes out into them.  So LDS holds nearly two steps
//     in flight (refilled a whole slot at a time, one: 8192 x 8192 x 8192 of zeros, where
//     power does not matter, ran at 2.9 PFLOP/s, waiting for DMA).  The next step's
//     weight fragments replace this one's as the last MFMAs let go of them.
//   * An MFMA's result joins the accumulators three MFMAs later.
//   * LDS row 16 nt + i of a wave's 64 columns is column 32 (nt >> 1) + 8 (i >> 2) +
//     4 (nt & 1) + (i & 3), so a lane ends with twice eight consecutive columns of one
//     row, 64 bytes of it in four lanes.  Gated: with 32 gates (nt = 0, 1) and the 32
//     ups that belong to them, eight of each in a lane.
// Measured: 8192 x 8192 x 8192 452 to 490 us by the card = 2.2 to 2.4 PFLOP/s, of zeros
// 380: the power limit (in registers alone, an MFMA of random codes with its four fmas
// takes 17.9 ns a SIMD, of zeros 14.9).  8192 x 3840 x 3840 115 us = 2.1 PFLOP/s, the
// matrix cores busy 57% of the time: 480 tiles for 256 CUs, two rounds, and a tile's
// stores, 11.5 us with its beginning, which the next tile's products do not overlap.
// Grouped, 32768 rows of 32 experts, K 1280, N 3840: 201 us in 16 bits, 260 in fp32 (503
// MB of stores from ten steps a tile: 40 us less without them).
// fp16 products: 8192 x 8192 x 8192 in fp32 920 to 1010 us = 1.1 to 1.2 PFLOP/s, zeros
// 845, gated 32768 x 3840 x 2560 598 = 1.08, the matrix cores busy half the time (a bf16
// product of the library: 1.46 to 1.49).  Of 1010 us a quarter of the MFMAs is worth
// 143, the conversions nothing (1010 without them): the rest is what a step of 128 rows
// costs beside its MFMAs.  Fragments converted one product ahead, two column tiles'
// MFMAs in turn, and the next step's weights read half a step earlier (at a second
// meeting) gave the same time to 7% more.
template <int BM, bool GROUPED, bool GATED, bool HALF>
__global__ __launch_bounds__(512, 2) void fp8_tile_kernel(Fp8GemmArgs a, int tiles_m, int tiles_n)
{
    constexpr int MT = BM / 32, NT = 4, G = GATED ? 2 : 1;
    constexpr int AB = BM * 128, SLOT = AB + 256 * 128;   // a slot: codes of both operands
    constexpr int SLOTS = BM == 256 ? 2 : 3;  // what LDS holds
    // a scale slot: of the rows, of the two weight blocks, and room for the DMA of
    // waves that have no scales, so that all issue the same
    constexpr int SA = BM * 4, SSLOT = SA + 512, S0 = SLOTS * SLOT, SEND = S0 + (SLOTS + 1) * SSLOT;
    // A step's DMA goes out in NP groups, group k before the last of row tiles PH k ..
    // PH (k + 1) - 1: their rows, and with the first one the weights and scales.
    constexpr int PH = MT < 4 ? MT : 4, NP = MT / PH;
    constexpr int AG = PH / 2, G0 = AG + 5, D = G0 + (NP - 1) * AG;   // instructions per wave: of a group's rows, in all
    constexpr int PUTS = 2 * MT;              // stores of an epilogue, at least
    // (one array: with several the compiler waits for all DMA before every read)
    constexpr int TILES = SEND, TOP = TILES + 2048;
    __shared__ __align__(16) uint8_t smem[TOP + (GATED ? 2 * 4 * (BM / 2) * 4 : 0)];
    v4i* const tiles = (v4i*)(smem + TILES);

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int j = lane & 15, q = lane >> 4;
    const int wm = wave >> 2, wn = wave & 3;   // (a SIMD's two waves: one of each half of the rows)
    const int64_t K = a.K, N = a.N;
    const int nsteps = (int)fp8_blocks(K);
    const int chunks = (int)(K >> 4);
    const int64_t F = N >> 1;   // gated: number of results

    // ---- tiles: this workgroup takes number blockIdx.x, + gridDim.x, ...
    struct Tile {
        int m0, rows, tn, e;   // rows 0: none
    };
    int ntiles;
    if constexpr (GROUPED) {
        MxRows r;
        ntiles = (int)mx_find<BM, false>(a, 0, r) * tiles_n;
        fp8_zero_rows(a, blockIdx.x, gridDim.x);
    } else {
        ntiles = tiles_m * tiles_n;
    }
    // The workgroup's tiles lie in LDS, two batches of 64: looking one up where it is
    // needed, in the K loop, would take registers and time that the MFMAs want.  Wave 0
    // fills a batch.
    auto fill = [&](int batch) {
        if (wave != 0) return;
        Tile mine{0, 0, 0, 0};
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
        tiles[(batch & 1) * 64 + lane] = (v4i){mine.m0, mine.rows, mine.tn, mine.e};
    };
    auto tile_of = [&](int i) {
        const v4i v = tiles[i & 127];
        return Tile{__builtin_amdgcn_readfirstlane(v[0]), __builtin_amdgcn_readfirstlane(v[1]),
                    __builtin_amdgcn_readfirstlane(v[2]), __builtin_amdgcn_readfirstlane(v[3])};
    };

    // ---- DMA: wave w moves 8 rows of A at a time, LDS rows (w >> 2) BM/2 + 32 i +
    // 8 (w & 3) + ..., and 32 weight columns
    const int ar0 = (wave >> 2) * (BM / 2) + 8 * (wave & 3), ahalf = wave & 1;
    const int ch = (lane & 7) ^ (lane >> 4);   // chunk of this lane; bit 2 of the LDS row's half turns it into ch ^ 4
    const bool gather = GROUPED && a.rows != nullptr;
    // Every resource is 2^31 bytes long: a lane that has nothing to read (a row
    // or column past the tile's, no tile, a chunk past K) has an offset past
    // that and gets zeros.
    uint32_t avo[MT / 2], bvo[4], svo;   // lane offsets of codes and scales
    int sstep = 0;                   // bytes from a step's scales to the next's
    __amdgpu_buffer_rsrc_t ra, rb, rs;
    // (the lane index, made anew: what depends on it would otherwise be kept in
    // registers from tile to tile)
    auto fresh = [&]() {
        int l = threadIdx.x & 63;
        asm volatile("" : "+v"(l));
        return l;
    };
    auto set_dma = [&](const Tile& t) {
        const int lane = fresh(), l8 = lane >> 3, ch = (lane & 7) ^ (lane >> 4);
        // the source row of tile row i, or none
        auto src_row = [&](int i) -> int {
            if (i >= t.rows) return -1;
            if (!gather) return i;
            const int s = a.rows[(int64_t)t.m0 + i];
            return s >= 0 && s < a.M ? s : -1;
        };
#pragma unroll
        for (int i = 0; i < MT / 2; ++i) {
            const int s = src_row(ar0 + 32 * i + l8);
            avo[i] = s < 0 ? kOut : (uint32_t)s * (uint32_t)K + (ch ^ (ahalf * 4)) * 16;
        }
        ra = mx_rsrc(mx_uniform(gather ? a.a : a.a + (int64_t)t.m0 * K), kOut);
        // LDS rows 32 wave + 8 i + l8: column tile nt, row idx of it
        const int64_t ncols = t.rows == 0 ? 0 : GATED ? F : N;
        const int64_t col0 = (int64_t)t.tn * (GATED ? 128 : 256);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int nt = (wave & 1) * 2 + (i >> 1), idx = (i & 1) * 8 + l8;
            const int c = (GATED ? (wave >> 1) * 32 : (wave >> 1) * 64 + 32 * (nt >> 1)) + 8 * (idx >> 2) + 4 * (nt & 1) + (idx & 3);
            bvo[i] = col0 + c < ncols ? (uint32_t)(c * (uint32_t)K + (ch ^ ((i & 1) * 4)) * 16) : kOut;
        }
        const int64_t brow = (int64_t)t.e * N + col0 + (GATED && (wave & 1) ? F : 0);
        rb = mx_rsrc(mx_uniform(a.b + (t.rows ? brow : 0) * K), kOut);
        // scales: of 64 rows, or of the two weight blocks
        if (wave < BM / 64) {
            const int s = src_row(wave * 64 + lane);
            svo = s < 0 ? kOut : (uint32_t)s * 4;
            rs = mx_rsrc(mx_uniform((const uint8_t*)(gather ? a.sa : a.sa + t.m0)), kOut);
            sstep = (int)(a.M * 4);
        } else {
            const int64_t blocks = fp8_blocks(N), nb = GATED ? t.tn : 2 * t.tn, up = GATED ? F / kFp8Block : 1;
            const bool have = wave == BM / 64 && lane < 2 && t.rows != 0 && nb + lane * up < blocks;
            svo = have ? (uint32_t)(lane * up * nsteps * 4) : kOut;
            rs = mx_rsrc(mx_uniform((const uint8_t*)(a.sb + ((int64_t)t.e * blocks + (t.rows ? nb : 0)) * nsteps)), kOut);
            sstep = 4;
        }
    };
    // the scale DMA's place in a scale slot
    const int sdst = S0 + (wave < BM / 64 ? wave * 256 : wave == BM / 64 ? SA : SA + 256);

    // The DMA of one step, an instruction at a time: `Dma` holds what its
    // instructions share.
    struct Dma {
        int ko, so;          // offsets of the step in a row of codes and in the scales
        uint32_t t0, t1;     // kOut where the chunk, its partner lies past K
    };
    auto dma_of = [&](Dma& d, int s) {
        d.t0 = s * 8 < chunks - ch ? 0u : kOut;
        d.t1 = s * 8 < chunks - (ch ^ 4) ? 0u : kOut;
        d.ko = s * 128;
        d.so = __builtin_amdgcn_readfirstlane(s * sstep);
    };
    // instruction n of group k, into slot sl and scale slot ssl
    auto dma = [&](const Dma& d, int sl, int ssl, int k, int n) {
        if (n < AG) {
            const int i = k * AG + n;
            mx_dma<16>(ra, smem + sl + (ar0 + 32 * i) * 128, avo[i] | (ahalf ? d.t1 : d.t0), d.ko);
        } else if (n == AG) {
            mx_dma<4>(rs, smem + ssl + sdst, svo, d.so);
        } else {
            const int i = n - AG - 1;
            mx_dma<16>(rb, smem + sl + AB + (wave * 32 + 8 * i) * 128, bvo[i & 3] | ((i & 1) ? d.t1 : d.t0), d.ko);
        }
    };
    // The steps of all tiles form one sequence; the DMA runs SLOTS steps, so up
    // to as many tiles, ahead of the MFMAs.
    fill(0);
    __syncthreads();
    Tile cur = tile_of(0);
    if (cur.rows == 0) return;
    int t_cur = 0, t_dma = 0, s_dma = 0;
    set_dma(cur);
    auto advance = [&]() {
        if (++s_dma < nsteps) return;
        s_dma = 0;
        set_dma(tile_of(++t_dma));
    };

    // ---- fragments: LDS rows ao + 16 mt and bo + 16 nt, chunks q and q + 4
    const int sw = (q ^ ((j >> 1) & 7)) * 16;
    const int ao = (wm * (BM / 2) + j) * 128 + sw, bo = AB + (wn * 64 + j) * 128 + sw;
    const int sao = S0 + (wm * (BM / 2) + j) * 4, sbo = S0 + SA + (GATED ? 0 : (wn >> 1) * 4);
    v8i fa[2], fb[NT];
    float sa[2], sb[G];
    // (base: a lane's address in a slot, off: the row tile's, which is an immediate)
    auto read = [&](v8i& f, int base, int off) {
        const v4i lo = *(const v4i*)(smem + base + off), hi = *(const v4i*)(smem + (base ^ 64) + off);
        f = join(lo, hi);
    };
    // row tile mt of a slot: its fragment and scales
    auto read_a = [&](int sl, int ssl, int mt) {
        read(fa[mt & 1], sl + ao, mt * 16 * 128);
        sa[mt & 1] = *(const float*)(smem + ssl + sao + mt * 64);
    };
    auto read_sb = [&](int ssl) {
#pragma unroll
        for (int i = 0; i < G; ++i) sb[i] = *(const float*)(smem + ssl + sbo + 4 * i);
    };

    Dma d;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        dma_of(d, s_dma);
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int n = 0; n < (k ? AG : G0); ++n) dma(d, s * SLOT, s * SSLOT, k, n);
        if (s + 1 < SLOTS) advance();
    }
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(SLOTS * D - G0) : "memory");   // the first group has landed
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int n = 0; n < NT; ++n) read(fb[n], bo, n * 16 * 128);
    read_a(0, 0, 0);
    read_sb(0);
    int sl = 0, ssl = 0;                   // this step's slots
    int stores = 0;                        // meetings at which the last epilogue's stores may be in flight
    for (;;) {
        v4f acc[MT][NT], tmp[4];
        float f[2][G];                     // factors of a row tile, and of the one before
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[mt][n] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) tmp[i] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < G; ++g) f[1][g] = 0.0f;
        // result i of a step joins its accumulators
        auto join_in = [&](int i) {
            const v4f t = tmp[i & 3];
            v4f c = acc[i >> 2][i & 3];
            const float x = f[(i >> 2) & 1][GATED ? (i & 3) >> 1 : 0];
            c = (v4f){__builtin_fmaf(t[0], x, c[0]), __builtin_fmaf(t[1], x, c[1]), __builtin_fmaf(t[2], x, c[2]),
                      __builtin_fmaf(t[3], x, c[3])};
            asm volatile("" : "+v"(c));   // here, not behind the next branch
            acc[i >> 2][i & 3] = c;
        };
        // all steps of a tile; LIVE: with the arithmetic
        auto steps = [&](auto live) {
            constexpr bool LIVE = decltype(live)::value;
#pragma clang loop unroll(disable)
            for (int s = 0; s < nsteps; ++s) {
                const int nx = sl == (SLOTS - 1) * SLOT ? 0 : sl + SLOT;
                const int snx = ssl == SLOTS * SSLOT ? 0 : ssl + SSLOT, spv = ssl == 0 ? SLOTS * SSLOT : ssl - SSLOT;
                v16i hb[HALF ? NT : 1], ha;
                if constexpr (HALF && LIVE) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) hb[n] = fp8_to_f16(fb[n]);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (m % PH == PH - 1) {
                        // What the next PH row tiles need has landed, and the last are read.  Still in flight may be all groups sent since and, until
                        // they are those that followed them, the stores of the tile before.
                        constexpr int kAll = SLOTS * D;
                        const int k = m / PH;
                        const int n0 = kAll - (k == 0 ? G0 : AG) - ((k + 1) % NP == 0 ? G0 : AG);
                        asm volatile("s_waitcnt lgkmcnt(0)\n\t"
                                     "s_cmp_lt_i32 %0, 1\n\t"
                                     "s_cbranch_scc1 1f\n\t"
                                     "s_waitcnt vmcnt(%1)\n\t"
                                     "s_branch 2f\n"
                                     "1:\n\t"
                                     "s_waitcnt vmcnt(%2)\n"
                                     "2:" ::"s"(__builtin_amdgcn_readfirstlane(stores)), "n"(n0 + PUTS), "n"(n0)
                                     : "memory", "scc");
                        --stores;
                        __builtin_amdgcn_s_barrier();
                        asm volatile("" ::: "memory");
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if constexpr (HALF && LIVE) ha = fp8_to_f16(fa[m & 1]);
#pragma unroll
                    for (int g = 0; g < G; ++g) f[m & 1][g] = mul_rn(sa[m & 1], sb[g]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int i = m * NT + n;
                        if constexpr (!LIVE) (void)0;
                        else if constexpr (HALF) tmp[i & 3] = f16_mfma(hb[n], ha);
                        else tmp[i & 3] = fp8_mfma(fb[n], fa[m & 1]);
                        if (m < MT - 1) {
                            if (n == 0) read_a(sl, ssl, m + 1);
                        } else {
                            // (past the last step: of a slot's older contents, unused)
                            if (n == 0) read_a(nx, snx, 0);
                            read(fb[n], nx + bo, n * 16 * 128);
                            if (n == NT - 1) read_sb(snx);
                        }
                        if (m % PH == PH - 1) {
                            const int size = m / PH == 0 ? G0 : AG;
#pragma unroll
                            for (int x = n * size / NT; x < (n + 1) * size / NT; ++x) dma(d, sl, spv, m / PH, x);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                        if constexpr (LIVE) join_in(i >= 3 ? i - 3 : MT * NT - 3 + i);
                        if (m == 0 && n == 2) {
                            advance();
                            dma_of(d, s_dma);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                sl = nx;
                ssl = snx;
            }
        };
        // Few rows: where a wave's are all past the tile's it only moves data, and leaves
        // its SIMD to the wave of the other half (32 experts of 3840 x 2560 with two rows
        // each, gated: 75 -> 66 us).
        if constexpr (HALF && BM == 64) {
            if (wm * (BM / 2) < cur.rows) steps(std::true_type{});
            else steps(std::false_type{});
        } else {
            steps(std::true_type{});
        }
#pragma unroll
        for (int i = MT * NT - 3; i < MT * NT; ++i) join_in(i);

        // ---- epilogue
        const int l = fresh(), j = l & 15, q = l >> 4, row0 = wm * (BM / 2) + j;
        if constexpr (GATED) {
            if (a.bias) fp8_put_gated<BM, true>(a, acc, cur.m0, cur.rows, cur.tn, wm, wn, j, q, cur.e, (uint32_t*)(smem + TOP));
            else fp8_put_gated<BM, false>(a, acc, cur.m0, cur.rows, cur.tn, wm, wn, j, q, cur.e, (uint32_t*)(smem + TOP));
        } else {
            const int64_t n0 = (int64_t)cur.tn * 256;
            const int c0 = wn * 64 + 8 * q;
            if (HALF || a.out_dtype == F32) fp8_epilogue<F32, MT>(a, acc, cur.m0, row0, cur.rows, n0, c0, cur.e);
            else if (a.out_dtype == BF16) fp8_epilogue<BF16, MT>(a, acc, cur.m0, row0, cur.rows, n0, c0, cur.e);
            else fp8_epilogue<F16, MT>(a, acc, cur.m0, row0, cur.rows, n0, c0, cur.e);
        }
        stores = SLOTS * NP - 1;
        // (the other batch is read from 29 tiles on at the earliest, many barriers later)
        if ((++t_cur & 63) == 32) fill((t_cur >> 6) + 1);
        cur = tile_of(t_cur);
        if (cur.rows == 0) break;
    }
}

int skinny_rows(const Fp8GemmArgs& a) { return a.M <= 16 ? 16 : a.M <= 32 ? 32 : 64; }

// 32 columns a group once 16 would make more workgroups than the CUs hold: the rows
// are read half as often.
int skinny_cols(const Fp8GemmArgs& a)
{
    return (a.N + 15) / 16 * ((a.M + skinny_rows(a) - 1) / skinny_rows(a)) <= 512 ? 16 : 32;
}

template <int MT, int NT, int KW> hipError_t launch_skinny_w(const Fp8GemmArgs& a, hipStream_t st)
{
    constexpr int COLS = 16 * NT * (kSkinnyWaves / KW);
    hipLaunchKernelGGL((fp8_skinny_kernel<MT, NT, KW>), dim3((unsigned)((a.N + COLS - 1) / COLS), (unsigned)((a.M + 16 * MT - 1) / (16 * MT))),
                       dim3(512), 0, st, a);
    return hipGetLastError();
}

template <int MT> hipError_t launch_skinny(const Fp8GemmArgs& a, hipStream_t st)
{
    // half the waves per column group where K has few steps for eight of them
    const bool deep = a.K > 1024;
    if (skinny_cols(a) == 16) return deep ? launch_skinny_w<MT, 1, 8>(a, st) : launch_skinny_w<MT, 1, 4>(a, st);
    return deep ? launch_skinny_w<MT, 2, 8>(a, st) : launch_skinny_w<MT, 2, 4>(a, st);
}

// One workgroup per CU (LDS holds one), which takes tiles in turn.
constexpr int64_t kTileGrid = 256;

template <int BM, bool HALF> hipError_t launch_tile(const Fp8GemmArgs& a, hipStream_t st)
{
    const bool gated = a.out_codes != nullptr;
    const int64_t tn = gated ? a.N / 2 / kFp8Block : (a.N + 255) / 256;
    // (grouped: at most this many, the device knows)
    const int64_t tm = a.E ? a.R / BM + (a.E < a.R ? a.E : a.R) : (a.M + BM - 1) / BM;
    const unsigned grid = (unsigned)(tm * tn < kTileGrid ? tm * tn : kTileGrid);
    if (!a.E)
        hipLaunchKernelGGL((fp8_tile_kernel<BM, false, false, HALF>), dim3(grid), dim3(512), 0, st, a, (int)tm, (int)tn);
    else if (!gated)
        hipLaunchKernelGGL((fp8_tile_kernel<BM, true, false, HALF>), dim3(grid), dim3(512), 0, st, a, 0, (int)tn);
    else if constexpr (HALF)
        hipLaunchKernelGGL((fp8_tile_kernel<BM, true, true, true>), dim3(grid), dim3(512), 0, st, a, 0, (int)tn);
    else
        return hipErrorNotSupported;   // (gated products are fp16 ones)
    return hipGetLastError();
}

// Estimated microseconds of each kernel.  Tiles: the 256 workgroups take them in
// rounds; a step of a 64, 128, 256 row tile measured 0.63, 0.95, 1.63 us with all CUs
// busy, a tile's beginning and end 4.3, 7.8, 11.5 (1024, 2048, 4096 rows of 4096
// outputs at K = 1280 and 3840: 13.2 and 25.6, 18.9 and 39.0, 28.4 and 63.9 us); with
// fp16 products a step of 64, 128 rows 1.15, 1.74 (256 rows would not fit the registers).
// Skinny: the weights, and for each column group the rows again, at 5 TB/s (10240 x
// 10240 weights with 1, 16, 32, 64 rows: 21, 30, 44, 65 us; with 64-row tiles 46).
// The groups' sizes are on the device: all are taken to have the mean, and to fill
// half of their last tile (ragged groups of 32 experts of 3840 x 2560 with a mean of
// 128, 256, 512, 1024 rows: 115, 158, 276, 500 us with 64 rows a tile, 89, 158, 233, 404
// with 128, 119, 134, 228, 361 with 256; gated, fp16 products: 145, 213, 384, 722 and 113,
// 217, 323, 598; with a mean of 64 rows 78 and 111).
double tile_us(const Fp8GemmArgs& a, int bm, double step, double ends)
{
    const double tn = a.out_codes ? (double)(a.N / 2 / kFp8Block) : (double)((a.N + 255) / 256);
    double tm = (double)((a.M + bm - 1) / bm);
    if (a.E) {
        const double groups = (double)(a.E < a.R ? a.E : a.R);
        tm = (double)a.R / bm + 0.5 * groups;
    }
    const double rounds = tm * tn < 1 ? 1 : (double)(int64_t)((tm * tn + 255) / 256);
    return 2.5 + rounds * ((double)fp8_blocks(a.K) * step + ends);
}

double skinny_us(const Fp8GemmArgs& a)
{
    const double weights = (double)a.N * (double)a.K * 1e-6;   // MB
    return 2.5 + (weights * (double)((a.M + skinny_rows(a) - 1) / skinny_rows(a)) + weights * (double)a.M / skinny_cols(a)) / 5.0;
}

}  // namespace

int fp8_gemm_path(const Fp8GemmArgs& a)
{
    const double t[4] = {skinny_us(a), tile_us(a, 64, a.half ? 1.15 : 0.63, 4.3), tile_us(a, 128, a.half ? 1.74 : 0.95, 7.8), tile_us(a, 256, 1.63, 11.5)};
    int best = kFp8Tile64;
    for (int i = kFp8Tile128; i <= (a.half ? kFp8Tile128 : kFp8Tile256); ++i)
        if (t[i] < t[best]) best = i;
    if (a.E) return best;
    // A tile's outputs are addressed with 31 bits: rows of 8 MB and more are the
    // skinny kernel's.
    if (a.N * (a.out_dtype == F32 ? 4 : 2) >= kFp8MaxRowBytes) return kFp8Skinny;
    // (past 128 rows the weights would be read three times and more)
    return a.M <= 128 && t[kFp8Skinny] < t[best] ? kFp8Skinny : best;
}

hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t st)
{
    switch (fp8_gemm_path(a)) {
    case kFp8Tile256: return launch_tile<256, false>(a, st);
    case kFp8Tile128: return a.half ? launch_tile<128, true>(a, st) : launch_tile<128, false>(a, st);
    case kFp8Tile64: return a.half ? launch_tile<64, true>(a, st) : launch_tile<64, false>(a, st);
    }
    const int rows = skinny_rows(a);
    return rows == 16 ? launch_skinny<1>(a, st) : rows == 32 ? launch_skinny<2>(a, st) : launch_skinny<4>(a, st);
}

}  // namespace w4a4
