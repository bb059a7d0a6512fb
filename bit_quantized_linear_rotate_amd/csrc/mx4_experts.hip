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
#include <type_traits>

#include "common.hpp"
#include "mx4.hpp"
#include "route_bounds.hpp"

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

// The end of a chunk whose slots per expert are counted.  ONE: the only chunk,
// which then sorts its own slots.
template <bool ONE> __device__ __forceinline__ void route_chunk_done(const RouteArgs& a, int* cnt, int* off)
{
    const int tid = threadIdx.x, threads = blockDim.x;
    if constexpr (ONE) {
        scan_experts(cnt, off, a.E);
        __syncthreads();
        const int total = off[a.E];
        for (int e = tid; e <= a.E; e += threads) a.offsets[e] = off[e];
        for (int64_t i = total + tid; i < a.T * a.k; i += threads) a.rows[i] = -1;
        __syncthreads();
        place_slots(a, 0, a.T * a.k, off);
    } else {
        for (int e = tid; e < a.E; e += threads) a.hist[(int64_t)blockIdx.x * a.E + e] = cnt[e];
    }
}

// top-k of a chunk's tokens and the chunk's slots per expert.
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
    route_chunk_done<ONE>(a, cnt, off);
}

// ---- routing by scores -------------------------------------------------------
// The choice is that of double precision: in fp32 the rounding of a score would
// decide between experts whose choice values differ by a few parts in 2^24, which a
// batch of some thousand tokens holds.  A token is first chosen in fp32, by sixteen
// lanes; where two values that the choice compares lie within the error of that, a
// wave chooses it again in double precision.  Without a bias the scores' order is the
// logits', and (unless groups are ranked by sums) nothing is in doubt.  The weights
// are computed in double precision, a choice to a lane.
// Bounds.  The logits are 8 MB at the most; what counts are the k dependent rounds
// over lanes, the exponentials, and fetching the code (every variant on sizes is its
// own kernel, straight through).  Measured: 32 tokens of 128 experts, 8 choices,
// softmax 8.0 us with the sort (in double precision throughout 11.4); 8192 tokens of
// 256, 8 choices, 4 of 8 groups by their two largest, sigmoid and bias 31 us (64), and the sort
// 7.4; of 32 experts, 4 choices, 4 groups 13.8; 16 tokens of those 10.1 with the sort.

// the value of the lane whose index differs in bits D, for the lanes of one token
template <int L> __device__ __forceinline__ double lanes_max64(double v)
{
#pragma unroll
    for (int d = 1; d < L; d *= 2) v = fmax(v, __shfl_xor(v, d));
    return v;
}
template <int L> __device__ __forceinline__ double lanes_sum64(double v)
{
#pragma unroll
    for (int d = 1; d < L; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// The lane (of the wave) with the token's largest v, the lowest of several; -1 where
// every v is -inf
template <int L> __device__ __forceinline__ int first_best(double v, double& best)
{
    best = lanes_max64<L>(v);
    const unsigned long long hit = __ballot(v == best && best > -__builtin_inf());
    const int base = L == 64 ? 0 : (threadIdx.x & 63) & ~(L - 1);
    const unsigned long long mine = L == 64 ? hit : (hit >> base) & ((1ull << (L & 63)) - 1);
    return mine ? base + __builtin_ctzll(mine) : -1;
}

// One token by L lanes, NV consecutive experts each: choice r ends in lane r.  worth:
// this token's E choice values in LDS (GROUPS only).
template <int L, int NV, bool GROUPS>
__device__ __forceinline__ void route_scored_token(const RouteScoredArgs& a, int64_t t, bool live, int lane, double* worth,
                                                   int& expert, float& weight)
{
    const double none = -__builtin_inf();
    const int e0 = lane * NV;
    double score[NV], val[NV];
    float logit[NV], top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = e0 + i;
        // (+ 0: both zeros are the same logit; a NaN is no logit)
        const float l = live && e < a.E ? add_rn(load_any_f32(a.dtype, a.logits, t * a.stride + e), 0.0f) : -__builtin_inff();
        logit[i] = l > -__builtin_inff() ? l : -__builtin_inff();
        val[i] = (double)logit[i];
        top = fmaxf(top, logit[i]);
    }
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NV; ++i) score[i] = val[i] > none ? 1.0 / (1.0 + exp(-val[i])) : 0.0;
    } else {
        const double m = lanes_max64<L>((double)top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // (equal to the largest, which may be infinite: 1)
            score[i] = val[i] > none ? (val[i] == m ? 1.0 : exp(val[i] - m)) : 0.0;
            sum += score[i];
        }
        sum = lanes_sum64<L>(sum);
        const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i) score[i] *= inv;
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const double v = score[i] + (double)a.bias[min(e0 + i, a.E - 1)];
            val[i] = val[i] > none && v > none ? v : none;
        }
    }
    if constexpr (GROUPS) {
        const int size = a.E / a.groups;
#pragma unroll
        for (int i = 0; i < NV; ++i)   // (without a bias the largest is known by its logit)
            if (e0 + i < a.E) worth[e0 + i] = val[i] > none && !a.bias && a.group_best == 2 ? score[i] : val[i];
        __threadfence_block();
        __builtin_amdgcn_wave_barrier();
        constexpr int GN = kRouteMaxGroups / L;   // groups of a lane, neighbours
        const int gn = (a.groups + L - 1) / L;
        double of[GN];
#pragma unroll
        for (int i = 0; i < GN; ++i) {
            const int g = lane * gn + i;
            of[i] = none;
            if (i < gn && g < a.groups) {
                double m1 = none, m2 = none;
                for (int x = 0; x < size; ++x) {
                    const double v = worth[g * size + x];
                    m2 = fmax(m2, fmin(m1, v));
                    m1 = fmax(m1, v);
                }
                of[i] = a.group_best == 2 && m2 > none ? m1 + m2 : m1;
            }
        }
        __builtin_amdgcn_wave_barrier();
        unsigned long long kept = 0;
        for (int r = 0; r < a.top_groups; ++r) {
            double mine = of[0], best;
#pragma unroll
            for (int i = 1; i < GN; ++i) mine = fmax(mine, of[i]);
            const int from = first_best<L>(mine, best);
            int g = 0;
#pragma unroll
            for (int i = GN - 1; i >= 0; --i)
                if (of[i] == best) g = i;
            if (lane == (from & (L - 1)) && from >= 0) {
#pragma unroll
                for (int i = 0; i < GN; ++i)
                    if (i == g) of[i] = none;
            }
            g = __shfl(lane * gn + g, from < 0 ? 0 : from);
            if (from >= 0) kept |= 1ull << g;
        }
        int g = e0 / size, left = (g + 1) * size - e0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (left == 0) {
                ++g;
                left = size;
            }
            --left;
            if (!((kept >> (g & 63)) & 1)) val[i] = none;
        }
    }
    expert = -1;
    double mine = 0.0;
    for (int r = 0; r < a.k; ++r) {
        double m = val[0], best;
#pragma unroll
        for (int i = 1; i < NV; ++i) m = fmax(m, val[i]);
        const int from = first_best<L>(m, best);
        int at = 0;
        double s = score[0];
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
            if (val[i] == best) {
                at = i;
                s = score[i];
            }
        const bool won = from >= 0 && lane == (from & (L - 1));
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (won && i == at) val[i] = none;
        const int src = from < 0 ? 0 : from, e = __shfl(e0 + at, src);
        s = __shfl(s, src);
        if (from >= 0 && lane == r) {
            expert = e;
            mine = s;
        }
    }
    if (a.renormalize) {
        const double sum = lanes_sum64<L>(mine);
        mine = sum > 0.0 ? mine / sum : 0.0;
    }
    weight = (float)(mine * (double)a.scale);
}

template <int L> __device__ __forceinline__ float lanes_maxf(float v)
{
    auto step = [&](auto ctrl) {
        const int b = __float_as_int(v);
        v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, decltype(ctrl)::value, 0xf, 0xf, false)));
    };
    if constexpr (L == 16) {
        step(std::integral_constant<int, 0x128>());   // row_ror 8, 4, 2, 1
        step(std::integral_constant<int, 0x124>());
        step(std::integral_constant<int, 0x122>());
        step(std::integral_constant<int, 0x121>());
        return v;
    }
    step(std::integral_constant<int, 0x111>());   // row_shr 1, 2, 4, 8
    step(std::integral_constant<int, 0x112>());
    step(std::integral_constant<int, 0x114>());
    step(std::integral_constant<int, 0x118>());
    step(std::integral_constant<int, 0x142>());   // row_bcast 15, 31
    step(std::integral_constant<int, 0x143>());
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Keys of N values per lane, of which the largest over L lanes tells the largest value
// and its index (i L + lane), the lower of equals: the index in the last BITS bits,
// above it the value.  16-bit values (exact) fit as they are; others in fixed point
// between the token's smallest and largest.  Then values `apart` units and less from
// one another may be in either order (error: of their difference).
template <int L, int N, int BITS> struct Ranked {
    uint32_t key[N];
    uint32_t apart = 0;
    bool exact;
    __device__ __forceinline__ void set(const float (&v)[N], bool exact_, float error, int lane)
    {
        constexpr uint32_t low = (1u << BITS) - 1;
        const float none = -__builtin_inff();
        exact = exact_;
        float lo = __builtin_inff(), hi = none;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            hi = fmaxf(hi, v[i]);
            lo = fminf(lo, v[i] > none ? v[i] : lo);
        }
        hi = lanes_maxf<L>(hi);
        lo = -lanes_maxf<L>(-lo);
        const float range = add_rn(hi, -lo);
        float unit = route_units(BITS) / range;
        if (!exact && hi > none) {
            // (a range of zero or infinity: nothing is told apart)
            if (!(unit < 0x1p120f && unit > 0.0f)) unit = 0.0f;
            apart = route_apart(BITS, error, unit);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t b = __float_as_uint(v[i]), order = (b & 0x80000000u) ? ~b : b | 0x80000000u;
            const uint32_t at = low - (uint32_t)(i * L + lane);
            const uint32_t fixed = ((uint32_t)mul_rn(add_rn(v[i], -lo), unit) + 1) << BITS;
            key[i] = v[i] > none ? (exact ? order & ~low : fixed) | at : 0;
        }
    }
    // The next largest's key, 0: none.
    __device__ __forceinline__ uint32_t next()
    {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < N; ++i) best = max(best, key[i]);
        best = lanes_max<L>(best);
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = key[i] == best ? 0 : key[i];
        return best;
    }
    static __device__ __forceinline__ int index(uint32_t k)
    {
        constexpr uint32_t low = (1u << BITS) - 1;
        return k ? (int)(low - (k & low)) : -1;
    }
    // whether the later of two keys may belong before the earlier one
    __device__ __forceinline__ bool doubt(uint32_t earlier, uint32_t later) const
    {
        return !exact && later && (earlier >> BITS) - (later >> BITS) <= apart;
    }
};

// One token in fp32 by L lanes, NV consecutive experts each: choice r ends in lane r
// (worth: its E values in LDS, sixteen and a gap each time, GROUPS only).
// unsure: two values that decide who is chosen lie within their error (route_bounds.hpp).
template <int DT, int L, int NV, bool GROUPS>
__device__ __forceinline__ void route_quick_token(const RouteScoredArgs& a, int64_t t, bool live, int lane, float* worth,
                                                  int& expert, float& weight, bool& unsure)
{
    const float none = -__builtin_inff();
    // (made anew for every token: kept from one to the next, what depends on it would
    // fill registers and a page of instructions ahead of the loop)
    asm volatile("" : "+v"(lane));
    float val[NV], top = none;
#pragma unroll
    for (int i = 0; i < NV; ++i) val[i] = load_as_f32<DT>(a.logits, (live ? t * a.stride : 0) + min(i * L + lane, a.E - 1));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        // (+ 0: both zeros are the same logit; a NaN is no logit)
        val[i] = add_rn(val[i], 0.0f);
        val[i] = live && i * L + lane < a.E && val[i] > none ? val[i] : none;
        top = fmaxf(top, val[i]);
    }
    top = lanes_maxf<L>(top);
    // scores, where the choice needs them; the sum of the softmax in double precision
    // where the candidates' values or the weights need it
    const bool sums = GROUPS && a.group_best == 2, scored = a.bias || sums;
    float score[NV], error = 0.0f, sum_error = 0.0f;   // of a difference of choice values, of sums of two
    double total = 0.0;
    if (!a.sigmoid && (a.bias || !a.renormalize)) {
        // (a loop over memory: exp NV times over would fill the instruction cache)
#pragma clang loop unroll(disable)
        for (int i = 0; i < NV; ++i) {
            const int e = i * L + lane;
            const float l = live && e < a.E ? load_as_f32<DT>(a.logits, t * a.stride + e) : none;
            total += l > none ? (l == top ? 1.0 : exp((double)l - (double)top)) : 0.0;
        }
        total = lanes_sum64<L>(total);
    }
    if (scored) {
        float sum = 0.0f, largest = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // (0 of -inf; a NaN where the largest logit is infinite, and then in doubt)
            if (a.sigmoid) score[i] = __builtin_amdgcn_rcpf(add_rn(1.0f, __expf(-val[i])));
            else score[i] = __expf(val[i] - top);
            sum = add_rn(sum, score[i]);
        }
        if (!a.sigmoid) {
            sum = lanes_sum<L>(sum);
            const float inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < NV; ++i) score[i] = mul_rn(score[i], inv);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v = score[i];
            if (a.bias) {
                v = add_rn(v, a.bias[min(i * L + lane, a.E - 1)]);
                val[i] = val[i] > none && v > none ? v : none;   // (a NaN would pass the maxima and minima by)
                v = fabsf(v) < __builtin_inff() ? fabsf(v) : 0.0f;
            }
            largest = fmaxf(largest, fmaxf(score[i], v));
        }
        largest = lanes_maxf<L>(largest);
        error = route_error(a.sigmoid, NV, top, largest);
        sum_error = route_sum_error(error, largest);
        unsure = top == __builtin_inff();
    } else {
        unsure = false;
    }
    constexpr bool narrow = DT != F32;
    if constexpr (GROUPS) {
        const int size = a.E / a.groups;
        auto place = [](int e) { return e + (e >> 4); };
#pragma unroll
        for (int i = 0; i < NV; ++i) worth[place(i * L + lane)] = val[i] > none && !a.bias && sums ? score[i] : val[i];
        __threadfence_block();
        __builtin_amdgcn_wave_barrier();
        constexpr int GN = kRouteMaxGroups / L;   // groups of a lane, neighbours
        float of[GN];
#pragma unroll
        for (int i = 0; i < GN; ++i) {
            const int g = i * L + lane;
            of[i] = none;
            if (g < a.groups) {
                float m1 = none, m2 = none;
                auto take = [&](float v) {
                    m2 = fmaxf(m2, fminf(m1, v));
                    m1 = fmaxf(m1, v);
                };
                int x = 0;
                for (; x + 8 <= size; x += 8) {
                    float v[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) v[y] = worth[place(g * size + x + y)];
#pragma unroll
                    for (int y = 0; y < 8; ++y) take(v[y]);
                }
                for (; x < size; ++x) take(worth[place(g * size + x)]);
                // (two of the lowest values: a worth all the same, and so far from the others
                // that the choice goes to double precision)
                of[i] = sums && m2 > none ? fmaxf(add_rn(m1, m2), -__FLT_MAX__) : m1;
            }
        }
        __builtin_amdgcn_wave_barrier();
        Ranked<L, GN, 6> groups;
        groups.set(of, !scored && narrow, sums ? sum_error : error, lane);
        unsigned long long kept = 0;
        uint32_t last = 0;
        for (int r = 0; r < a.top_groups; ++r) {
            last = groups.next();
            if (last) kept |= 1ull << groups.index(last);
        }
        if (groups.doubt(last, groups.next())) unsure = true;
        // (e + 0.5) / size in fp32 is off an integer by 0.5 / 1024 at least
        const float inv = 1.0f / (float)size;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int g = (int)(((float)(i * L + lane) + 0.5f) * inv);
            if (!((kept >> (g & 63)) & 1)) val[i] = none;
        }
    }
    Ranked<L, NV, (L * NV <= 256 ? 8 : 10)> experts;
    experts.set(val, !a.bias && narrow, a.bias ? error : 0.0f, lane);
    // Two candidates more than are taken.  What comes after them is in doubt where it
    // may belong before the last that is taken; the candidates themselves are put in
    // order by their values in double precision, a candidate to a lane.
    expert = -1;
    uint32_t last = 0;
    for (int r = 0; r < a.k + 2; ++r) {
        const uint32_t k = experts.next();
        if (lane == r) expert = experts.index(k);
        if (r == a.k - 1) last = k;
        if (r == a.k + 1 && experts.doubt(last, k)) unsure = true;
    }
    double s = 0.0, c = -__builtin_inf();
    if (expert >= 0) {
        const double l = (double)load_as_f32<DT>(a.logits, t * a.stride + expert) + 0.0;
        const double x = exp(a.sigmoid ? -l : l - (double)top);
        s = a.sigmoid ? 1.0 / (1.0 + x) : l == (double)top ? 1.0 : x;
        c = l;
        if (a.bias) c = (a.sigmoid ? s : s / total) + (double)a.bias[expert];
    }
    auto misplaced = [&]() {   // the next lane's candidate belongs before this one's
        const double cn = __shfl_down(c, 1);
        const int en = __shfl_down(expert, 1);
        return lane <= a.k && en >= 0 && (cn > c || (cn == c && en < expert));
    };
    if (!experts.exact && __any(misplaced())) {
        for (int pass = 0; pass < 2; ++pass) {   // pairs (0, 1), (2, 3), ..; (1, 2), (3, 4), ..
            const int with = ((lane + pass) ^ 1) - pass;
            const int from = (threadIdx.x & 63) - lane + max(with, 0);
            const double co = __shfl(c, from), so = __shfl(s, from);
            const int eo = __shfl(expert, from);
            const bool first = with > lane;
            const bool theirs = eo >= 0 && expert >= 0 && (co > c || (co == c && eo < expert));
            if (with >= 0 && with <= a.k + 1 && lane <= a.k + 1 && eo >= 0 && expert >= 0 && theirs == first) {
                c = co;
                s = so;
                expert = eo;
            }
        }
        if (misplaced()) unsure = true;
        // (any lane's doubt is the token's)
        unsure = lanes_maxf<L>(unsure ? 1.0f : 0.0f) > 0.0f;
    }
    if (lane >= a.k) {
        expert = -1;
        s = 0.0;
    }
    if (a.renormalize) total = lanes_sum64<L>(s);
    else if (a.sigmoid) total = 1.0;
    weight = (float)(total > 0.0 ? s / total * (double)a.scale : 0.0);
}

// (sixteen experts a lane take more than the 128 registers of 1024 threads)
template <int NV> constexpr int route_scored_threads() { return NV > 8 ? 512 : 1024; }

template <int DT, int L, int NV, bool GROUPS, bool ONE>
__global__ __launch_bounds__(route_scored_threads<NV>()) void route_scored_kernel(RouteScoredArgs a, int64_t chunk)
{
    constexpr int kThreads = route_scored_threads<NV>();
    __shared__ int cnt[kRouteMaxExperts], off[kRouteMaxExperts + 1];
    constexpr int kInDoubt = -2;   // experts of a token that is to be chosen in double precision
    __shared__ int doubts;
    // a wave's: 64 / L tokens in fp32, or one in double precision
    constexpr int NW = (L * NV + 63) / 64;
    __shared__ double worth[GROUPS ? kThreads / 64 : 1][GROUPS ? 64 * NW > 34 * NV ? 64 * NW : 34 * NV : 1];
    const int tid = threadIdx.x, lane = tid & (L - 1), wl = tid & 63;
    for (int e = tid; e < a.E; e += kThreads) cnt[e] = 0;
    if (tid == 0) doubts = 0;
    __syncthreads();
    const int64_t t0 = blockIdx.x * chunk, t1 = min(t0 + chunk, a.T);
    double* const own = worth[GROUPS ? tid >> 6 : 0];
    // (all lanes of a wave stay in the loop: lanes read one another)
    for (int64_t tw = t0 + (tid >> 6) * (64 / L); tw < t1; tw += kThreads / L) {
        const int64_t t = tw + wl / L;
        int e;
        float w;
        bool unsure;
        route_quick_token<DT, L, NV, GROUPS>(a, t, t < t1, lane, (float*)own + (GROUPS ? wl / L * (L * NV * 17 / 16) : 0), e, w, unsure);
        if (unsure) doubts = 1;
        if (lane < a.k && t < t1) {
            a.weights[t * a.k + lane] = w;
            a.experts[t * a.k + lane] = unsure ? kInDoubt : e;
            if (e >= 0 && !unsure) atomicAdd(&cnt[e], 1);
        }
    }
    __syncthreads();
    if (doubts) {   // a wave to a token
        for (int64_t t = t0 + (tid >> 6); t < t1; t += kThreads / 64) {
            if (__builtin_amdgcn_readfirstlane(a.experts[t * a.k]) != kInDoubt) continue;
            int e, l = wl;
            float w;
            asm volatile("" : "+v"(l));
            route_scored_token<64, NW, GROUPS>(a, t, true, l, own, e, w);
            if (wl < a.k) {
                a.weights[t * a.k + wl] = w;
                a.experts[t * a.k + wl] = e;
                if (e >= 0) atomicAdd(&cnt[e], 1);
            }
        }
    }
    __syncthreads();
    route_chunk_done<ONE>(a, cnt, off);
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

// `kernel` on the chunks of a.T tokens, then, where there is more than one, the sort
template <class Args>
hipError_t route_launch(const Args& a, void (*one)(Args, int64_t), void (*many)(Args, int64_t), int threads, hipStream_t st)
{
    const int64_t chunks = route_chunks(a.T), chunk = (a.T + chunks - 1) / chunks;
    hipLaunchKernelGGL(chunks == 1 ? one : many, dim3((unsigned)chunks), dim3((unsigned)threads), 0, st, a, chunk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || chunks == 1) return e;
    hipLaunchKernelGGL(route_sort_kernel, dim3((unsigned)chunks), dim3(kSortThreads), 0, st, a, chunk, (int)chunks);
    return hipGetLastError();
}

template <int DT, int L, int NV> hipError_t route_nv(const RouteArgs& a, hipStream_t st)
{
    return route_launch<RouteArgs>(a, route_kernel<DT, L, NV, true>, route_kernel<DT, L, NV, false>, 1024, st);
}

template <int DT, int L, int NV> hipError_t route_scored_nv(const RouteScoredArgs& a, hipStream_t st)
{
    if (a.groups > a.top_groups)
        return route_launch<RouteScoredArgs>(a, route_scored_kernel<DT, L, NV, true, true>, route_scored_kernel<DT, L, NV, true, false>,
                                             route_scored_threads<NV>(), st);
    return route_launch<RouteScoredArgs>(a, route_scored_kernel<DT, L, NV, false, true>, route_scored_kernel<DT, L, NV, false, false>,
                                         route_scored_threads<NV>(), st);
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

template <int DT> hipError_t route_scored_dt(const RouteScoredArgs& a, hipStream_t st)
{
    // (the candidates, two more than are taken, have a lane each)
    if (a.E <= 256 && a.k <= 14)
        return a.E <= 32 ? route_scored_nv<DT, 16, 2>(a, st) : a.E <= 64 ? route_scored_nv<DT, 16, 4>(a, st)
               : a.E <= 128 ? route_scored_nv<DT, 16, 8>(a, st) : route_scored_nv<DT, 16, 16>(a, st);
    return a.E <= 256 ? route_scored_nv<DT, 64, 4>(a, st) : route_scored_nv<DT, 64, 16>(a, st);
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

hipError_t launch_route_scored(const RouteScoredArgs& a, hipStream_t st)
{
    switch (a.dtype) {
    case F32: return route_scored_dt<F32>(a, st);
    case F16: return route_scored_dt<F16>(a, st);
    case BF16: return route_scored_dt<BF16>(a, st);
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
