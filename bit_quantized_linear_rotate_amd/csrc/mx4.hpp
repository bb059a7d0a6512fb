// Launch interfaces and device helpers of the MX4 (microscaled 4-bit floating
// point) operators: the quantiser and its inverse, the product, the product
// grouped by expert, routing and combining.
//
// MX4: 32 consecutive k of a row share a power-of-two scale 2^X; an element is
// an e2m1 code (sign bit 3; magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6) standing for
// code * 2^X.  Codes are (rows, K/2) bytes, even k in the low nibble.  Scale
// bytes (X + 127; 255 makes the block NaN) are kept in slabs of 256 k:
// byte b of row r in slab s, at (s * rows + r) * 8 + b, belongs to k =
// 256 s + 32 b ... + 31; bytes past K/32 are zero.  A slab holds the scales of
// one K step of the product for neighbouring rows in neighbouring bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {

constexpr int kMxBlock = 32;     // elements per scale
constexpr int kMxSlab = 256;     // elements per row of a scale slab (8 scales)

inline int64_t mx4_slabs(int64_t K) { return (K + kMxSlab - 1) / kMxSlab; }

struct Mx4QuantArgs {
    const void* x;
    int dtype;
    int64_t M, K, sm, sk;          // strides in elements
    int g;                         // Hadamard group, 0: no rotation
    const int8_t* sign_in;         // (g,) or nullptr
    const int8_t* sign_out;
    uint8_t* codes;                // (M, K/2)
    uint8_t* scales;               // (slabs, M, 8)
};
hipError_t launch_mx4_quantize(const Mx4QuantArgs& a, hipStream_t st);
hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* out,
                                 int out_dtype, hipStream_t st);

struct Mx4GemmArgs {
    const uint8_t* a;              // (M, K/2) codes
    const uint8_t* sa;             // (slabs, M, 8)
    int64_t M, K, N;
    const uint8_t* b;              // (N, K/2), or (E, N, K/2)
    const uint8_t* sb;             // (slabs, N, 8), or (E, slabs, N, 8)
    const void* bias;              // (N,) or (E, N), or nullptr
    int bias_dtype;
    void* out;                     // (M, N), or (R, N)
    int out_dtype;
    // grouped by expert (E > 0): sorted row i of [offsets[e], offsets[e + 1])
    // is row rows[i] of a (row i where rows is null)
    int E = 0;
    int64_t R = 0;
    const int32_t* offsets = nullptr;   // (E + 1,)
    const int32_t* rows = nullptr;      // (R,) or nullptr
    // gated: the N columns are N/2 gates and N/2 ups; the result is the MX4
    // form of silu(gate) * up, in place of out
    uint8_t* out_codes = nullptr;       // (R, N/4)
    uint8_t* out_scales = nullptr;      // (slabs of N/2, R, 8)
};
// the kernel a call takes (host-only)
enum { kMx4Skinny = 0, kMx4Tile64 = 1, kMx4Tile128 = 2, kMx4Tile256 = 3 };
int mx4_gemm_path(const Mx4GemmArgs& a);
hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, hipStream_t st);

// Routing: each token's top_k experts by logit (ties: the lower index; -inf and
// NaN logits are never taken), their softmax weights, and the stable sort of
// the (token, choice) slots by expert.
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
struct RouteArgs {
    const void* logits;            // (T, E), row stride `stride` elements
    int dtype;
    int64_t T, stride;
    int E, k;
    int renormalize;               // weights: softmax over the chosen (1) or over all experts (0)
    float* weights;                // (T, k)
    int32_t* experts;              // (T, k), -1: none
    int32_t* rows;                 // (T k,) token of each sorted row, -1 past the last
    int32_t* pos;                  // (T, k) sorted row of each slot, -1: none
    int32_t* offsets;              // (E + 1,)
    int32_t* hist;                 // workspace (route_chunks(T), E)
};
int64_t route_chunks(int64_t T);   // 1: no workspace needed
hipError_t launch_route(const RouteArgs& a, hipStream_t st);

// out[t] = sum_j weights[t][j] * y[pos[t][j]], fp32, j in order
struct CombineArgs {
    const void* y;                 // (R, N)
    int dtype;                     // of y
    int64_t R, T, N;
    int k;
    const int32_t* pos;            // (T, k)
    const float* weights;          // (T, k)
    void* out;                     // (T, N)
    int out_dtype;                 // dtype, or any where that is fp32
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t st);

}  // namespace w4a4
