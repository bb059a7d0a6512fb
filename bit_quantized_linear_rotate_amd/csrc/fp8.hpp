// Launch interfaces of the operators on block-scaled 8-bit floating point (fp8): the
// quantisers of rows and of weights, their inverses, and the product, dense and
// grouped by expert.
//
// Codes are OCP e4m3 (bias 7, largest 448, 0x7f a NaN).  An activation's fp32 scale
// belongs to 128 consecutive k of a row and is kept k-block-major, (ceil(K/128),
// rows): a step of the product is a block, and neighbouring rows' scales of a step
// are neighbours.  A weight's scale belongs to 128 rows by 128 k, (ceil(N/128),
// ceil(K/128)).  The last blocks may be short; K is a multiple of 16, so that rows
// keep the alignment of 16-byte loads.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {

constexpr int kFp8Block = 128;

__host__ __device__ inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

struct Fp8QuantArgs {
    const void* x;
    int dtype;
    int64_t M, K, sm, sk;          // strides in elements
    int g;                         // Hadamard group, 0: no rotation
    const int8_t* sign_in;         // (g,) or nullptr
    const int8_t* sign_out;
    uint8_t* codes;                // (M, K), or (E, M, K)
    float* scales;                 // (blocks of K, M); weights: (E, blocks of M, blocks of K)
    int64_t E = 1, se = 0;         // weights: matrices and their stride
};
hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, hipStream_t st);
hipError_t launch_fp8_quantize_weights(const Fp8QuantArgs& a, hipStream_t st);
// E == 0: rows with scales (blocks, M); else E matrices of weights (M, K)
hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t E, int64_t M, int64_t K, void* out,
                                 int out_dtype, hipStream_t st);

struct Fp8GemmArgs {
    const uint8_t* a;              // (M, K) codes
    const float* sa;               // (blocks of K, M)
    int64_t M, K, N;
    const uint8_t* b;              // (N, K), or (E, N, K)
    const float* sb;               // (blocks of N, blocks of K), or E of them
    const void* bias;              // (N,) or (E, N), or nullptr
    int bias_dtype;
    void* out;                     // (M, N), or (R, N)
    int out_dtype;
    bool half = false;             // products on the fp16 matrix cores, for fp32 outputs and (always) gated ones
    // grouped by expert (E > 0): sorted row i of [offsets[e], offsets[e + 1])
    // is row rows[i] of a (row i where rows is null)
    int E = 0;
    int64_t R = 0;
    const int32_t* offsets = nullptr;   // (E + 1,)
    const int32_t* rows = nullptr;      // (R,) or nullptr
    // gated: the N columns are N/2 gates and N/2 ups (N/2 a multiple of 128); the
    // result is the fp8 form of silu(gate) * up, in place of out
    uint8_t* out_codes = nullptr;       // (R, N/2)
    float* out_scales = nullptr;        // (N/256, R)
};
constexpr int64_t kFp8MaxRowBytes = (int64_t)1 << 23;   // of outputs, in the tile kernel
// the kernel a call takes (host-only)
enum { kFp8Skinny = 0, kFp8Tile64 = 1, kFp8Tile128 = 2, kFp8Tile256 = 3 };
int fp8_gemm_path(const Fp8GemmArgs& a);
hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t st);

}  // namespace w4a4
