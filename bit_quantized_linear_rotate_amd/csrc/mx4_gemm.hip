// The MX4 product out[m][n] = sum_k a[m][k] w[n][k] (+ bias[n]) on gfx950's
// scaled f8f6f4 matrix cores, dense and grouped by expert.
//
// Mathematics.  v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 by
// 128 x 16 e2m1 values, each run of 32 k of a row times its own power of two,
// and adds to fp32.  Products of two e2m1 values are multiples of 1/4 up to
// 36, so the sum over a block is exact; sums over blocks and steps are fp32.
// Lane (j, q) (j = lane & 15, q = lane >> 4) supplies row j, one block of 32 k
// and that block's scale byte.  Which 32 k lane group q holds is free as long
// as both operands agree: here a step of 256 k gives group q the blocks 2q and
// 2q + 1, two MFMAs (t = 0, 1) whose scales are bytes t of one 16-bit word.
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

// ---- which rows a workgroup takes --------------------------------------------
struct MxRows {
    int64_t m0;   // first (sorted) row
    int rows;     // rows of the tile, 0: none
    int e;        // expert
    int m, cm;    // tile of the expert, and how many it has
    int64_t before;   // tiles of the experts before it
};

// offsets[e], kept inside [0, R] whatever the device array holds
__device__ __forceinline__ int64_t mx_offset(const Mx4GemmArgs& a, int e)
{
    const int64_t o = a.offsets[e];
    return o < 0 ? 0 : o > a.R ? a.R : o;
}

// The row tile `idx` of the list of all experts' tiles of BM rows (idx < 0:
// only count).  Every wave scans the offsets, 64 experts at a time.  Returns
// the number of tiles.
template <int BM, bool BY_TILE> __device__ __forceinline__ int64_t mx_find(const Mx4GemmArgs& a, int64_t idx, int64_t per,
                                                                         MxRows& r)
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
        int inc = cm;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int v = __shfl_up(inc, d);
            if (lane >= d) inc += v;
        }
        const int sum = __builtin_amdgcn_readlane(inc, 63);
        if (BY_TILE && r.e < 0 && idx >= base * per && idx < (base + sum) * per) {
            const unsigned long long hit = __ballot((base + inc) * per > idx);
            const int w = __builtin_ctzll(hit);
            r.e = e0 + w;
            r.cm = __builtin_amdgcn_readlane(cm, w);
            r.before = base + __builtin_amdgcn_readlane(inc, w) - r.cm;
            r.m0 = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)lo, w);
            r.rows = __builtin_amdgcn_readlane(cnt, w);   // of the expert; the caller picks the tile
            return base + sum;
        }
        base += sum;
    }
    return base;
}

// Zeros for the sorted rows that no expert owns (from offsets[E] on), spread
// over the workgroups that have no tile.
__device__ __forceinline__ void mx_zero_rows(const Mx4GemmArgs& a, int64_t part, int64_t parts)
{
    const int64_t from = mx_offset(a, a.E);
    if (a.out_codes) {
        const int64_t F = a.N / 2, wide = F / 2;
        for (int64_t i = from * wide + part * blockDim.x + threadIdx.x; i < a.R * wide; i += parts * blockDim.x)
            a.out_codes[i] = 0;
        const int64_t slabs = (F + 255) / 256, n = (a.R - from) * 8;
        for (int64_t i = part * blockDim.x + threadIdx.x; i < n * slabs; i += parts * blockDim.x)
            a.out_scales[(i / n * a.R + from) * 8 + i % n] = 0;
    } else {
        const int esz = a.out_dtype == F32 ? 4 : 2;
        uint16_t* o = (uint16_t*)a.out;
        const int64_t end = a.R * a.N * (esz / 2);
        for (int64_t i = from * a.N * (esz / 2) + part * blockDim.x + threadIdx.x; i < end; i += parts * blockDim.x)
            o[i] = 0;
    }
}

// silu(g) * u in fp32: g / (1 + exp(-g)) * u
__device__ __forceinline__ float mx_gated(float g, float u)
{
    return mul_rn(g / add_rn(1.0f, __expf(-g)), u);
}

// The scale byte of a block whose largest magnitude has fp32 bits m (255:
// NaN or infinity), as the quantiser computes it.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t m)
{
    const uint32_t ex = m >> 23;
    return ex == 255 ? 255u : ex > 2 ? ex - 2 : 0u;
}

__device__ __forceinline__ uint32_t mx_pack2(int odt, float lo, float hi)
{
    return odt == BF16 ? (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16)
                       : (uint32_t)f32_to_f16(lo) | ((uint32_t)f32_to_f16(hi) << 16);
}

// Sixteen consecutive outputs of one row, from column c on (those below N).
// vec: rows are 16-byte aligned, so a 16-byte piece is all in or all out.
__device__ __forceinline__ void mx_store16(const Mx4GemmArgs& a, int64_t row, int64_t c, bool vec, const float (&v)[16])
{
    const int esz = a.out_dtype == F32 ? 4 : 2;
    char* o = (char*)a.out + (row * a.N + c) * esz;
    if (!vec) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (c + i < a.N) store_any(a.out_dtype, o, i, v[i]);
    } else if (a.out_dtype == F32) {
#pragma unroll
        for (int h = 0; h < 4; ++h)
            if (c + 4 * h < a.N) ((v4f*)o)[h] = (v4f){v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (c + 8 * h < a.N)
                ((v4u*)o)[h] = (v4u){mx_pack2(a.out_dtype, v[8 * h], v[8 * h + 1]),
                                     mx_pack2(a.out_dtype, v[8 * h + 2], v[8 * h + 3]),
                                     mx_pack2(a.out_dtype, v[8 * h + 4], v[8 * h + 5]),
                                     mx_pack2(a.out_dtype, v[8 * h + 6], v[8 * h + 7])};
    }
}

// ---- the tile kernel ---------------------------------------------------------
// BM x 256 outputs per workgroup of four waves (2 x 2, each BM/2 x 128), K in
// steps of 256.
//   * A step's codes (128 bytes a row) and scales (8 bytes a row) go global ->
//     LDS by DMA into one of two slots.  16-byte chunk c of a row sits at
//     c ^ swizzle(row), so that the sixteen lanes of every ds_read_b128 cycle
//     (lanes j in {0-3, 12-15} of one 16-lane group and {4-11} of its
//     neighbour) hit sixteen different 16-byte bank groups.
//   * A step is two halves (t = 0, 1).  While half t's MFMAs run from
//     registers, the fragments of the next half are read from LDS.  Between
//     the halves the waves wait for the next step's DMA and meet; then nobody
//     reads this step's slot any more, and the DMA of the step after the next
//     goes out into it, a whole step ahead of its use.
//   * The MFMA takes the weights as first operand, and the weight columns of
//     four neighbouring column tiles are interleaved (tile nt, MFMA row c is
//     column 16 (c >> 2) + 4 nt + (c & 3) of 64), so a lane ends with sixteen
//     consecutive columns of one row.
//   * Gated: a wave's 128 columns are 64 gates and the 64 ups that belong to
//     them, so gate, up and the block of 32 results (two neighbouring lane
//     groups) meet in registers: silu, product, block scale and codes are the
//     epilogue, and the 2 x 16-bit intermediate is never written.
template <int BM, bool GROUPED, bool GATED>
__global__ __launch_bounds__(256, 1) void mx4_tile_kernel(Mx4GemmArgs a, int tiles_m, int tiles_n)
{
    constexpr int MT = BM / 32, NT = 8;
    constexpr int AB = BM * 128, BB = 256 * 128, SAB = BM * 8, SBB = 256 * 8;
    constexpr int SLOT = AB + BB + SAB + SBB;
    constexpr int AI = BM / 32;               // A DMA instructions per wave (8 rows each)
    __shared__ __align__(16) uint8_t smem[2 * SLOT];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int j = lane & 15, q = lane >> 4;
    const int wm = wave & 1, wn = wave >> 1;
    const int64_t K = a.K, N = a.N, pitch = K >> 1;
    const int nsteps = (int)((K + 255) / 256);

    // ---- the tile
    int64_t m0;
    int rows, tn, e = 0;
    if constexpr (GROUPED) {
        MxRows r;
        const int64_t total = mx_find<BM, false>(a, 0, 1, r) * tiles_n;
        const int64_t t = blockIdx.x;
        if (t >= total) {
            mx_zero_rows(a, t - total, gridDim.x - total);
            return;
        }
        // each XCD (workgroup index modulo 8) takes a contiguous range
        const int64_t q8 = total >> 3, r8 = total & 7, xcd = t & 7;
        const int64_t tile = xcd * q8 + (xcd < r8 ? xcd : r8) + (t >> 3);
        mx_find<BM, true>(a, tile, tiles_n, r);
        // within an expert: groups of eight row tiles, row tiles fastest
        const int in_e = (int)(tile - r.before * tiles_n);
        const int per = 8 * tiles_n, grp = in_e / per, gm = min(r.cm - grp * 8, 8), in_g = in_e - grp * per;
        const int m = grp * 8 + in_g % gm;
        tn = in_g / gm;
        e = r.e;
        m0 = r.m0 + (int64_t)m * BM;
        rows = min(r.rows - m * BM, BM);
    } else {
        const int total = tiles_m * tiles_n, t = blockIdx.x;
        const int q8 = total >> 3, r8 = total & 7, xcd = t & 7;
        const int tile = xcd * q8 + min(xcd, r8) + (t >> 3);
        // groups of four row tiles: an XCD's 32 concurrent tiles span 4 x 8 blocks
        const int per = 4 * tiles_n, grp = tile / per, gm = min(tiles_m - grp * 4, 4), in_g = tile - grp * per;
        m0 = (int64_t)(grp * 4 + in_g % gm) * BM;
        tn = in_g / gm;
        rows = (int)min(a.M - m0, (int64_t)BM);
    }
    const int64_t F = N >> 1;   // gated: number of results
    const uint8_t* wb = a.b + (int64_t)e * N * pitch;
    const uint8_t* wsb = a.sb + (int64_t)e * nsteps * N * 8;

    // ---- DMA: wave w moves rows [w BM/4, (w + 1) BM/4) of A and 64 weight columns
    const int l8 = lane >> 3, c8 = lane & 7;
    const int ar0 = wave * (BM / 4);
    const int ca = c8 ^ ((((l8 >> 1) & 1) << 2) | ((l8 >> 2) & 1));
    const int cb0 = c8 ^ (((l8 >> 1) & 1) << 2);
    const bool gather = GROUPED && a.rows != nullptr;
    const uint8_t* abase = gather ? a.a : a.a + m0 * pitch;
    const uint8_t* sabase = gather ? a.sa : a.sa + m0 * 8;
    const int64_t arows = gather ? a.M : rows;      // rows behind the resource
    const int64_t srows = a.M;                      // rows of a scale slab
    // the source row of tile row i, or one past the resource
    auto src_row = [&](int i) -> int64_t {
        if (!gather) return i;
        if (i >= rows) return -1;
        const int64_t s = a.rows[m0 + i];
        return s >= 0 && s < a.M ? s : -1;
    };
    uint32_t avo[AI], savo[2];
#pragma unroll
    for (int i = 0; i < AI; ++i) {
        const int64_t s = src_row(ar0 + 8 * i + l8);
        avo[i] = s < 0 ? kOut : (uint32_t)(s * pitch + ca * 16);
    }
    // scales: 32 rows per 64-lane instruction; BM / 32 instructions in all
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r0 = BM == 256 ? wave * 64 + i * 32 : wave * 32;
        const int64_t s = src_row(r0 + (lane >> 1));
        savo[i] = s < 0 || r0 >= BM ? kOut : (uint32_t)(s * 8 + (lane & 1) * 4);
    }
    const __amdgpu_buffer_rsrc_t ra = mx_rsrc(abase, arows * pitch);
    // the wave's 64 weight columns (gated: even waves gates, odd waves ups)
    const int64_t col0 = GATED ? (int64_t)tn * 128 + (wave >> 1) * 64 : (int64_t)tn * 256 + wave * 64;
    const int64_t ncols = GATED ? F : N, wcol = GATED ? (wave & 1) * F + col0 : col0;
    const int64_t left = ncols - col0 < 0 ? 0 : ncols - col0 > 64 ? 64 : ncols - col0;
    const __amdgpu_buffer_rsrc_t rb = mx_rsrc(wb + (left ? wcol : 0) * pitch, left * pitch);
    const uint32_t bvo = (uint32_t)(l8 * pitch), bstep = (uint32_t)(8 * pitch);
    const uint8_t* sbcol = wsb + (left ? wcol : 0) * 8;
    const int kblocks = (int)(K >> 5);

    auto issue = [&](int s) {
        uint8_t* sl = smem + (s & 1) * SLOT;
        const int ko = s * 128;
        // chunks past K read zeros (offset past the resource)
        const uint32_t ta = s * 8 + ca < kblocks ? 0u : kOut;
        const uint32_t tb0 = (s * 8 + cb0 < kblocks ? cb0 * 16u : kOut) + bvo;
        const uint32_t tb1 = (s * 8 + (cb0 ^ 1) < kblocks ? (cb0 ^ 1) * 16u : kOut) + bvo;
#pragma unroll
        for (int i = 0; i < AI; ++i)
            mx_dma<16>(ra, sl + (ar0 + 8 * i) * 128, avo[i] | ta, ko);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mx_dma<16>(rb, sl + AB + (wave * 64 + 8 * i) * 128, ((i >> 2) ? tb1 : tb0) + i * bstep, ko);
        const __amdgpu_buffer_rsrc_t rsa = mx_rsrc(sabase + s * srows * 8, arows * 8);
        const __amdgpu_buffer_rsrc_t rsb = mx_rsrc(sbcol + s * N * 8, left * 8);
        if constexpr (BM == 256) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                mx_dma<4>(rsa, sl + AB + BB + (wave * 64 + i * 32) * 8, savo[i], 0);
        } else if (wave * 32 < BM) {
            mx_dma<4>(rsa, sl + AB + BB + wave * 32 * 8, savo[0], 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            mx_dma<4>(rsb, sl + AB + BB + SAB + (wave * 64 + i * 32) * 8, lane * 4 + i * 256, 0);
    };

    // ---- fragments
    const int arow = wm * (BM / 2) + j, asw = (((j >> 1) & 1) << 2) | ((j >> 2) & 1);
    const int bcol = wn * 128 + 16 * (j >> 2) + (j & 3), bsw = (((j >> 1) & 1) << 2) | ((j >> 3) & 1);
    const int ao = arow * 128, bo = AB + bcol * 128;
    const int ac = ((2 * q) ^ asw) * 16, bc = ((2 * q) ^ bsw) * 16;
    const int so_a = AB + BB + arow * 8 + 2 * q, so_b = AB + BB + SAB + bcol * 8 + 2 * q;
    v4i fa[2][MT], fb[2][NT];
    uint32_t fsa[MT], fsb[NT];
    v4f acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = (v4f){0.f, 0.f, 0.f, 0.f};
    auto read = [&](int slot, int t, v4i (&xa)[MT], v4i (&xb)[NT]) {
        const uint8_t* sl = smem + slot * SLOT;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            xb[nt] = *(const v4i*)(sl + bo + ((nt >> 2) * 64 + (nt & 3) * 4) * 128 + (bc ^ (t * 16)));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) xa[mt] = *(const v4i*)(sl + ao + mt * 16 * 128 + (ac ^ (t * 16)));
    };
    auto read_scales = [&](int slot, uint32_t (&xa)[MT], uint32_t (&xb)[NT]) {
        const uint8_t* sl = smem + slot * SLOT;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            xb[nt] = *(const uint16_t*)(sl + so_b + ((nt >> 2) * 64 + (nt & 3) * 4) * 8);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) xa[mt] = *(const uint16_t*)(sl + so_a + mt * 16 * 8);
    };

    issue(0);
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (nsteps > 1) issue(1);
    read(0, 0, fa[0], fb[0]);
    read_scales(0, fsa, fsb);

    for (int s = 0; s < nsteps; ++s) {
        // ---- half 0: read half 1 of this step
        read(s & 1, 1, fa[1], fb[1]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                acc[mt][nt] = mx_mfma<0, 0>(fb[0][nt], fa[0][mt], acc[mt][nt], fsb[nt], fsa[mt]);
#pragma unroll
        for (int i = 0; i < MT + NT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, MT * NT / (MT + NT), 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0): the next step has landed, this one is read
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        // ---- half 1: DMA of the step after the next, read half 0 of the next
        // (past the last step: of a slot that holds an older step, unused)
        if (s + 2 < nsteps) issue(s + 2);
        uint32_t nsa[MT], nsb[NT];
        read((s & 1) ^ 1, 0, fa[0], fb[0]);
        read_scales((s & 1) ^ 1, nsa, nsb);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                acc[mt][nt] = mx_mfma<1, 1>(fb[1][nt], fa[1][mt], acc[mt][nt], fsb[nt], fsa[mt]);
#pragma unroll
        for (int i = 0; i < MT + NT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, MT * NT / (MT + NT), 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) fsb[nt] = nsb[nt];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) fsa[mt] = nsa[mt];
    }

    // ---- epilogue: lane (j, q) holds row wm BM/2 + 16 mt + j, and of each
    // half u of the wave's 128 columns the sixteen from 16 q
    if constexpr (GATED) {
        const int64_t f0 = (int64_t)tn * 128 + wn * 64 + 16 * q;
        const bool in_f = f0 < F;     // F is a multiple of 32, so are the blocks
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int row = wm * (BM / 2) + 16 * mt + j;
            float v[16];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float g = acc[mt][i >> 2][i & 3], u = acc[mt][4 + (i >> 2)][i & 3];
                if (a.bias && in_f) {
                    g = add_rn(g, load_any_f32(a.bias_dtype, a.bias, (int64_t)e * N + f0 + i));
                    u = add_rn(u, load_any_f32(a.bias_dtype, a.bias, (int64_t)e * N + F + f0 + i));
                }
                v[i] = mx_gated(g, u);
                m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
            }
            m = max(m, (uint32_t)__builtin_amdgcn_ds_swizzle((int)m, 0x401f));   // the block's other sixteen
            const uint32_t byte = mx_scale_byte(m);
            const float sc = __uint_as_float(byte << 23);
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                c[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[h], v[8 * h + 0], v[8 * h + 1], sc, 0);
                c[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[h], v[8 * h + 2], v[8 * h + 3], sc, 1);
                c[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[h], v[8 * h + 4], v[8 * h + 5], sc, 2);
                c[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[h], v[8 * h + 6], v[8 * h + 7], sc, 3);
                if (byte == 255) c[h] = 0;
            }
            if (row < rows) {
                const int64_t R = GROUPED ? a.R : a.M;
                if (in_f) *(v2u*)(a.out_codes + ((m0 + row) * F + f0) / 2) = (v2u){c[0], c[1]};
                // one lane per block writes its scale; columns past F, up to
                // the end of the slab (which a last tile may fill only half),
                // get zeros
                if (!(q & 1)) {
                    uint8_t* o = a.out_scales + ((f0 >> 8) * R + m0 + row) * 8 + ((f0 >> 5) & 7);
                    o[0] = (uint8_t)(in_f ? byte : 0u);
                    if (tn == tiles_n - 1 && !(tn & 1)) o[4] = 0;
                }
            }
            __builtin_amdgcn_sched_barrier(0);   // one row tile's values at a time
        }
    } else {
        const int esz = a.out_dtype == F32 ? 4 : 2;
        const bool vec = (N * esz) % 16 == 0 && (uintptr_t)a.out % 16 == 0;
        // sixteen consecutive columns of one row: half u of the wave's 128
        const int64_t c0 = (int64_t)tn * 256 + wn * 128 + 16 * q;
        float bv[2][16];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int64_t c = c0 + 64 * (i >> 4) + (i & 15);
            bv[i >> 4][i & 15] = a.bias && c < N ? load_any_f32(a.bias_dtype, a.bias, (int64_t)e * N + c) : 0.0f;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int row = wm * (BM / 2) + 16 * mt + j;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    v[i] = acc[mt][4 * u + (i >> 2)][i & 3];
                    if (a.bias) v[i] = add_rn(v[i], bv[u][i]);
                }
                if (row < rows) mx_store16(a, m0 + row, c0 + 64 * u, vec, v);
                __builtin_amdgcn_sched_barrier(0);   // one row tile's values at a time
            }
        }
    }
}

// ---- the skinny kernel -------------------------------------------------------
// Few rows: the weights are the cost, read once, straight into registers.  A
// workgroup of eight waves takes 16 MT rows and 16 columns (gated: 32 gates
// and their 32 ups, one block of results); the waves share the K steps and
// their partial sums meet in LDS, added in wave order.
constexpr int kSkinnyWaves = 8;
template <int MT, bool GROUPED, bool GATED>
__global__ __launch_bounds__(512) void mx4_skinny_kernel(Mx4GemmArgs a)
{
    constexpr int NT = GATED ? 4 : 1, W = kSkinnyWaves;
    __shared__ float part[W][MT][NT][16][17];   // [wave][row tile][column tile][row][column]
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int j = lane & 15, q = lane >> 4;
    const int64_t K = a.K, N = a.N, F = N >> 1, pitch = K >> 1;
    const int nsteps = (int)((K + 255) / 256);
    int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    int rows, e = 0;
    if constexpr (GROUPED) {
        MxRows r;
        const int64_t total = mx_find<16 * MT, true>(a, blockIdx.y, 1, r);
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
    // this lane's weight columns and rows (clamped: what they give is not stored)
    int64_t col[NT], src[MT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int64_t c = GATED ? (int64_t)blockIdx.x * 32 + (nt & 1) * 16 + j : (int64_t)blockIdx.x * 16 + j;
        const int64_t n = GATED ? F : N;
        col[nt] = (c < n ? c : n - 1) + (nt >> 1) * F;
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
    constexpr int U = GATED ? 1 : 2;     // steps in flight
    for (int s0 = wave; s0 < nsteps; s0 += W * U) {
        v4i fb[U][NT][2], fa[U][MT][2];
        uint32_t sb[U][NT], sa[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + W * u;
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
    const int waves = nsteps < W ? nsteps : W;
    auto sum = [&](int mt, int nt, int row, int c) {
        float v = part[0][mt][nt][row][c];
        for (int w = 1; w < waves; ++w) v = add_rn(v, part[w][mt][nt][row][c]);
        return v;
    };
    if constexpr (GATED) {
        // a half wave takes the 32 results of one row
        const int c = tid & 31;
        const int64_t f = (int64_t)blockIdx.x * 32 + c, R = GROUPED ? a.R : a.M;
        for (int row = tid >> 5; row < 16 * MT; row += 16) {
            const int mt = row >> 4;
            float g = sum(mt, c >> 4, row & 15, c & 15), u = sum(mt, 2 + (c >> 4), row & 15, c & 15);
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
            if (row < rows) {
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
        }
    } else {
        for (int i = tid; i < MT * 256; i += 512) {
            const int mt = i >> 8, row = (i >> 4) & 15, c = i & 15;
            const int64_t n = (int64_t)blockIdx.x * 16 + c;
            float v = sum(mt, 0, row, c);
            if (n < N && 16 * mt + row < rows) {
                if (a.bias) v = add_rn(v, load_any_f32(a.bias_dtype, a.bias, (int64_t)e * N + n));
                store_any(a.out_dtype, a.out, (m0 + 16 * mt + row) * N + n, v);
            }
        }
    }
}

template <int BM> hipError_t launch_tile(const Mx4GemmArgs& a, hipStream_t st)
{
    const bool gated = a.out_codes != nullptr;
    const int64_t tn = gated ? (a.N / 2 + 127) / 128 : (a.N + 255) / 256;
    if (a.E) {
        const int64_t tm = a.R / BM + (a.E < a.R ? a.E : a.R) + 1;
        if (gated)
            hipLaunchKernelGGL((mx4_tile_kernel<BM, true, true>), dim3((unsigned)(tm * tn)), dim3(256), 0, st, a, 0, (int)tn);
        else
            hipLaunchKernelGGL((mx4_tile_kernel<BM, true, false>), dim3((unsigned)(tm * tn)), dim3(256), 0, st, a, 0, (int)tn);
    } else {
        const int64_t tm = (a.M + BM - 1) / BM;
        hipLaunchKernelGGL((mx4_tile_kernel<BM, false, false>), dim3((unsigned)(tm * tn)), dim3(256), 0, st, a, (int)tm, (int)tn);
    }
    return hipGetLastError();
}

template <int MT> hipError_t launch_skinny(const Mx4GemmArgs& a, hipStream_t st)
{
    const bool gated = a.out_codes != nullptr;
    const unsigned tn = (unsigned)(gated ? a.N / 64 : (a.N + 15) / 16);
    if (a.E) {
        const unsigned tm = (unsigned)(a.R / (16 * MT) + (a.E < a.R ? a.E : a.R) + 1);
        if (gated)
            hipLaunchKernelGGL((mx4_skinny_kernel<MT, true, true>), dim3(tn, tm), dim3(512), 0, st, a);
        else
            hipLaunchKernelGGL((mx4_skinny_kernel<MT, true, false>), dim3(tn, tm), dim3(512), 0, st, a);
    } else {
        hipLaunchKernelGGL((mx4_skinny_kernel<MT, false, false>), dim3(tn, (unsigned)((a.M + 16 * MT - 1) / (16 * MT))),
                           dim3(512), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace

int mx4_gemm_path(const Mx4GemmArgs& a)
{
    // rows a weight tile meets: all of them, or an expert's share
    const int64_t rows = a.E ? (a.R + a.E - 1) / a.E : a.M;
    if (rows <= 64) return kMx4Skinny;
    if (rows <= 128) return kMx4Tile64;
    if (rows <= 512) return kMx4Tile128;
    return kMx4Tile256;
}

hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, hipStream_t st)
{
    switch (mx4_gemm_path(a)) {
    case kMx4Tile256: return launch_tile<256>(a, st);
    case kMx4Tile128: return launch_tile<128>(a, st);
    case kMx4Tile64: return launch_tile<64>(a, st);
    }
    const int64_t rows = a.E ? (a.R + a.E - 1) / a.E : a.M;
    return rows <= 16 ? launch_skinny<1>(a, st) : launch_skinny<2>(a, st);
}

}  // namespace w4a4
