// Routing rows to experts and combining the experts' results.
//
// Routing.  Per token, k rounds of "largest logit, lowest index" over the E
// logits by sixteen lanes (64 for many experts or choices); weights are
// exp(l - max) over their sum (over the chosen or over all experts).  The
// (token, choice) slots are then sorted by expert with a stable counting sort,
// so the order is a function of the logits alone: chunks of tokens count their
// slots per expert, and every chunk adds up the counts before it to place its
// own.  Counts are integers: the order in which they are added does not matter.
//
// Bounds.  A few megabytes: the launches, and the k dependent rounds of a maximum
// over lanes (8192 tokens of 128 experts, 1, 2, 4 and 8 choices: 4.8, 5.3, 6.0,
// 8.0 us, so 0.45 us a round; the sort 5.3 to 5.9).  One chunk (up to 64 tokens)
// is one launch, more are two, since the sort needs all chunks' counts.  Measured: 32 tokens of 32 experts, 4
// choices 3.8 us; 8192 of 128, 8 choices 8.7 + 6.4 us; 8192 of 32, 4 choices
// 4.9 + 6.6 us.
#include "common.hpp"
#include "mx4.hpp"

namespace w4a4 {

namespace {

constexpr int kChunkTokens = 64;    // at least; 128 chunks at most
constexpr int kMaxChunks = 128;

// reductions over the L lanes of a token (16: a DPP row; 64: the wave), the
// result in every lane
template <int CTRL> __device__ __forceinline__ uint32_t dpp0(uint32_t v)
{
    return __builtin_amdgcn_update_dpp(0u, v, CTRL, 0xf, 0xf, false);   // 0 where there is no source
}
template <int L> __device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    if constexpr (L == 16) {
        v = max(v, dpp0<0x128>(v));   // row_ror 8, 4, 2, 1
        v = max(v, dpp0<0x124>(v));
        v = max(v, dpp0<0x122>(v));
        return max(v, dpp0<0x121>(v));
    }
    v = max(v, dpp0<0x111>(v));   // row_shr 1, 2, 4, 8
    v = max(v, dpp0<0x112>(v));
    v = max(v, dpp0<0x114>(v));
    v = max(v, dpp0<0x118>(v));
    v = max(v, dpp0<0x142>(v));   // row_bcast 15, 31
    v = max(v, dpp0<0x143>(v));
    return __builtin_amdgcn_readlane(v, 63);
}
template <int L> __device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int d = 1; d < L; d *= 2) v = add_rn(v, __shfl_xor(v, d));
    return v;
}

// Larger key = larger logit; 0 for what is never taken (-inf, NaN)
__device__ __forceinline__ uint32_t route_key(float v)
{
    const uint32_t b = __float_as_uint(v);
    if (!(v > -__builtin_inff())) return 0;
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// One token by L lanes, NV logits each: choice r ends in lane r of them
// (expert -1: none; t past the last token: nothing is live)
template <int DT, int L, int NV> __device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, bool live, int lane,
                                                                             int& expert, float& weight)
{
    float val[NV];
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * L + lane;
        // (+ 0: both zeros are the same logit)
        val[i] = live && e < a.E ? add_rn(load_as_f32<DT>(a.logits, t * a.stride + e), 0.0f) : -__builtin_inff();
        key[i] = route_key(val[i]);
    }
    expert = -1;
    float mine = 0.0f, top = 0.0f;
    for (int r = 0; r < a.k; ++r) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) best = max(best, key[i]);
        best = lanes_max<L>(best);
        if (L == 64 && best == 0) break;   // nothing is left
        uint32_t idx = 0;       // ~index, so that the lowest index is the largest
#pragma unroll
        for (int i = 0; i < NV; ++i) idx = max(idx, key[i] == best ? ~(uint32_t)(i * L + lane) : 0u);
        idx = ~lanes_max<L>(idx);
        const float v = __uint_as_float((best & 0x80000000u) ? best & 0x7fffffffu : ~best);
        if (best != 0) {
            if (r == 0) top = v;
            if (lane == r) {
                expert = (int)idx;
                mine = v;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (idx == (uint32_t)(i * L + lane)) key[i] = 0;
    }
    const float e = expert >= 0 ? expf(mine - top) : 0.0f;
    float part = e;
    if (!a.renormalize) {
        part = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (val[i] > -__builtin_inff()) part = add_rn(part, expf(val[i] - top));
    }
    const float total = lanes_sum<L>(part);
    weight = expert >= 0 ? e / total : 0.0f;
}

// the slots [from, to) of a chunk, whose first rows per expert are in base[]
__device__ __forceinline__ void place_slots(const RouteArgs& a, int64_t from, int64_t to, int* base)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
    for (int64_t s0 = from; s0 < to; s0 += blockDim.x) {
        const int64_t s = s0 + tid;
        const int e = s < to ? a.experts[s] : -1;
        // lanes with the same expert
        unsigned long long peers = __ballot(e >= 0);
        for (int b = 0; (1 << b) < a.E; ++b) {
            const unsigned long long one = __ballot((e >> b) & 1);
            peers &= ((e >> b) & 1) ? one : ~one;
        }
        const int rank = __popcll(peers & ((1ull << lane) - 1));
        const int busy = (int)min((to - s0 + 63) / 64, (int64_t)waves);
        for (int w = 0; w < busy; ++w) {   // waves in order: the sort is stable
            if (wave == w && e >= 0) {
                const int p = base[e] + rank;
                a.pos[s] = p;
                a.rows[p] = (int)(s / a.k);
            }
            __builtin_amdgcn_wave_barrier();
            if (wave == w && e >= 0 && rank == 0) base[e] += __popcll(peers);
            __syncthreads();
        }
        if (s < to && e < 0) a.pos[s] = -1;
    }
}

// exclusive prefix sum of tot[0 .. E) into off[0 .. E] by wave 0
__device__ __forceinline__ void scan_experts(const int* tot, int* off, int E)
{
    const int tid = threadIdx.x;
    if (tid < 64) {
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int v = e0 + tid < E ? tot[e0 + tid] : 0;
            int inc = v;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int o = __shfl_up(inc, d);
                if (tid >= d) inc += o;
            }
            if (e0 + tid < E) off[e0 + tid] = carry + inc - v;
            carry += __builtin_amdgcn_readlane(inc, 63);
        }
        if (tid == 0) off[E] = carry;
    }
}

// top-k of a chunk's tokens and the chunk's slots per expert.  ONE: the only
// chunk, which then sorts its own slots.
template <int DT, int L, int NV, bool ONE> __global__ __launch_bounds__(1024) void route_kernel(RouteArgs a, int64_t chunk)
{
    __shared__ int cnt[kRouteMaxExperts], off[kRouteMaxExperts + 1];
    const int tid = threadIdx.x, lane = tid & (L - 1);
    for (int e = tid; e < a.E; e += 1024) cnt[e] = 0;
    __syncthreads();
    const int64_t t0 = blockIdx.x * chunk, t1 = min(t0 + chunk, a.T);
    // (all lanes of a wave stay in the loop: lanes read one another)
    for (int64_t tw = t0 + (tid >> 6) * (64 / L); tw < t1; tw += 1024 / L) {
        const int64_t t = tw + ((tid & 63) / L);
        int e;
        float w;
        route_token<DT, L, NV>(a, t, t < t1, lane, e, w);
        if (lane < a.k && t < t1) {
            a.weights[t * a.k + lane] = w;
            a.experts[t * a.k + lane] = e;
            if (e >= 0) atomicAdd(&cnt[e], 1);
        }
    }
    __syncthreads();
    if constexpr (ONE) {
        scan_experts(cnt, off, a.E);
        __syncthreads();
        const int total = off[a.E];
        for (int e = tid; e <= a.E; e += 1024) a.offsets[e] = off[e];
        for (int64_t i = total + tid; i < a.T * a.k; i += 1024) a.rows[i] = -1;
        __syncthreads();
        place_slots(a, 0, a.T * a.k, off);
    } else {
        for (int e = tid; e < a.E; e += 1024) a.hist[(int64_t)blockIdx.x * a.E + e] = cnt[e];
    }
}

constexpr int kSortThreads = 512;
__global__ __launch_bounds__(kSortThreads) void route_sort_kernel(RouteArgs a, int64_t chunk, int chunks)
{
    __shared__ int tot[kRouteMaxExperts], pre[kRouteMaxExperts], off[kRouteMaxExperts + 1];
    const int tid = threadIdx.x;
    for (int e = tid; e < a.E; e += kSortThreads) tot[e] = pre[e] = 0;
    __syncthreads();
    // counts of all chunks and of those before this one; with few experts
    // several groups of threads share the chunks
    const int width = a.E >= kSortThreads ? kSortThreads : a.E, groups = kSortThreads / width, grp = tid / width;
    if (grp < groups)
        for (int e = tid - grp * width; e < a.E; e += width) {
            int all = 0, before = 0;
#pragma unroll 16
            for (int c = grp; c < chunks; c += groups) {
                const int v = a.hist[(int64_t)c * a.E + e];
                all += v;
                before += c < (int)blockIdx.x ? v : 0;
            }
            atomicAdd(&tot[e], all);
            atomicAdd(&pre[e], before);
        }
    __syncthreads();
    scan_experts(tot, off, a.E);
    __syncthreads();
    const int total = off[a.E];
    if (blockIdx.x == 0)
        for (int e = tid; e <= a.E; e += kSortThreads) a.offsets[e] = off[e];
    for (int64_t i = total + (int64_t)blockIdx.x * kSortThreads + tid; i < a.T * a.k; i += (int64_t)gridDim.x * kSortThreads) a.rows[i] = -1;
    __syncthreads();
    for (int e = tid; e < a.E; e += kSortThreads) off[e] += pre[e];
    __syncthreads();
    const int64_t t0 = blockIdx.x * chunk, t1 = min(t0 + chunk, a.T);
    place_slots(a, t0 * a.k, t1 * a.k, off);
}

template <int DT, int L, int NV> hipError_t route_nv(const RouteArgs& a, hipStream_t st)
{
    const int64_t chunks = route_chunks(a.T), chunk = (a.T + chunks - 1) / chunks;
    if (chunks == 1) {
        hipLaunchKernelGGL((route_kernel<DT, L, NV, true>), dim3(1), dim3(1024), 0, st, a, chunk);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((route_kernel<DT, L, NV, false>), dim3((unsigned)chunks), dim3(1024), 0, st, a, chunk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(route_sort_kernel, dim3((unsigned)chunks), dim3(kSortThreads), 0, st, a, chunk, (int)chunks);
    return hipGetLastError();
}

template <int DT> hipError_t route_dt(const RouteArgs& a, hipStream_t st)
{
    // Four tokens a wave while sixteen lanes hold the logits and the choices
    // (8192 tokens, 128 experts, 8 choices: 15.2 us with a wave per token).
    if (a.E <= 256 && a.k <= 16)
        return a.E <= 32 ? route_nv<DT, 16, 2>(a, st) : a.E <= 64 ? route_nv<DT, 16, 4>(a, st)
               : a.E <= 128 ? route_nv<DT, 16, 8>(a, st) : route_nv<DT, 16, 16>(a, st);
    return a.E <= 256 ? route_nv<DT, 64, 4>(a, st) : route_nv<DT, 64, 16>(a, st);
}

// Combining: out[t] = sum_j w[t][j] y[pos[t][j]] in fp32, j in order, rounded
// once.  8 (fp32: 4) columns per thread, one token per workgroup row.  Bound by
// memory, y being read once: 8192 tokens of 4 rows of 3840 bf16 (315 MB) 58.6
// us = 5.4 TB/s, a copy's rate.
// (In the expert layer y is in the layer's 16-bit type unless the caller asks
// for fp32: a second rounding next to the output's, 2^-9 of a value, where its
// four-bit operands are 2^-4 off.  In fp32 the layer's largest array is twice as
// large: 504 MB more to move at 8192 tokens, 441 us then 584; with 16 no change.)
template <int DT, int ODT, bool VEC> __global__ __launch_bounds__(256) void combine_kernel(CombineArgs a)
{
    constexpr int V = VEC ? (DT == F32 ? 4 : 8) : 1;
    typedef unsigned v4u __attribute__((ext_vector_type(4)));
    typedef unsigned v2u __attribute__((ext_vector_type(2)));
    const int64_t pieces = (a.N + V - 1) / V;
    const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (n >= pieces) return;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll 4
        for (int c = 0; c < a.k; ++c) {
            const int p = a.pos[t * a.k + c];
            const float w = a.weights[t * a.k + c];
            if (p < 0 || p >= a.R) continue;
            if constexpr (VEC) {
                const v4u v = ((const v4u*)a.y)[p * pieces + n];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float f = DT == F32 ? __uint_as_float(v[i & 3])
                                              : h_to_f32<DT == F32 ? BF16 : DT>((uint16_t)(v[(i >> 1) & 3] >> (16 * (i & 1))));
                    acc[i] = __builtin_fmaf(w, f, acc[i]);
                }
            } else {
                acc[0] = __builtin_fmaf(w, load_as_f32<DT>(a.y, p * a.N + n), acc[0]);
            }
        }
        if constexpr (!VEC) {
            store_any(ODT, a.out, t * a.N + n, acc[0]);
        } else if constexpr (ODT == F32) {
            ((v4u*)a.out)[t * pieces + n] = (v4u){__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                                                  __float_as_uint(acc[3])};
        } else if constexpr (DT == F32) {
            ((v2u*)a.out)[t * pieces + n] = (v2u){f32_to_h<ODT>(acc[0]) | ((uint32_t)f32_to_h<ODT>(acc[1]) << 16),
                                                  f32_to_h<ODT>(acc[2]) | ((uint32_t)f32_to_h<ODT>(acc[3]) << 16)};
        } else {
            v4u o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = f32_to_h<ODT>(acc[2 * i]) | ((uint32_t)f32_to_h<ODT>(acc[2 * i + 1]) << 16);
            ((v4u*)a.out)[t * pieces + n] = o;
        }
    }
}

template <int DT, int ODT> hipError_t combine_dt(const CombineArgs& a, hipStream_t st)
{
    const int v = DT == F32 ? 4 : 8;
    const bool vec = a.N % v == 0 && (uintptr_t)a.y % 16 == 0 && (uintptr_t)a.out % 16 == 0;
    const int64_t pieces = vec ? a.N / v : a.N;
    const dim3 grid((unsigned)((pieces + 255) / 256), (unsigned)(a.T < 65535 ? a.T : 65535));
    if (vec)
        hipLaunchKernelGGL((combine_kernel<DT, ODT, true>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((combine_kernel<DT, ODT, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace

int64_t route_chunks(int64_t T)
{
    const int64_t c = (T + kChunkTokens - 1) / kChunkTokens;
    if (c <= kMaxChunks) return c > 1 ? c : 1;
    const int64_t chunk = (T + kMaxChunks - 1) / kMaxChunks;
    return (T + chunk - 1) / chunk;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t st)
{
    switch (a.dtype) {
    case F32: return route_dt<F32>(a, st);
    case F16: return route_dt<F16>(a, st);
    case BF16: return route_dt<BF16>(a, st);
    }
    return hipErrorNotSupported;
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t st)
{
    if (a.dtype == F32) {
        switch (a.out_dtype) {
        case F32: return combine_dt<F32, F32>(a, st);
        case F16: return combine_dt<F32, F16>(a, st);
        case BF16: return combine_dt<F32, BF16>(a, st);
        }
    } else if (a.dtype == a.out_dtype) {
        switch (a.dtype) {
        case F16: return combine_dt<F16, F16>(a, st);
        case BF16: return combine_dt<BF16, BF16>(a, st);
        }
    }
    return hipErrorNotSupported;
}

}  // namespace w4a4
