// grad_gemm.h -- products of gradients with int8 codes (gfx950), private to the library:
//
//   C[i][j] (+)= 2^-k sum_r A[i][r] * B[r][j]
//
// B holds int8 codes, which bf16 and fp16 hold exactly, so the products are exact and only the fp32
// accumulation rounds besides A's own rounding.  A holds fp32 values scaled by a power of two, 2^k, in
//   two pieces (P = 2): the value rounded to bf16 and the remainder rounded to fp16.  The remainder is at most 2^-8 of
//     the value and keeps 11 bits: relative error 2^-19.  (Two bf16 pieces reach 2^-17.)
//   one piece (P = 1): the value rounded to fp16, 2^-11.  (bf16: 2^-8.)
// fp16 ends at 2^-24, so k puts the largest possible value just inside its range (grad_exponent): what is smaller
// than 2^-29 of that loses bits, at 2^-40 all of fp16's; the bf16 piece keeps its 8 at any size.  Where a row of A has
// a factor of its own, k is the row's: rows of any size keep their bits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace dfssm {

// What bounds A's values and so scales them: a common factor's partial maxima, and a factor for each row.
constexpr int kMaximaBlocks = 64;  // one a lane
struct GradFactors {
    const float* maxima;  // [kMaximaBlocks]
    const float* rows;    // [I] (then C is fp32), or NULL: the factor 1
};

// v < 2^exponent for any finite v.
__device__ __forceinline__ int above_exponent(float v) { return (int)(__float_as_uint(v) >> 23 & 255u) - 126; }

// k for values below the product of a common factor < 2^common and a row's factor: 2^k times them is at most 2^23 with two
// pieces (the remainder then stays below 2^15) and 2^15 with one.  The row's factor times 2^k is an fp32 number.
template <int P>
__device__ __forceinline__ int grad_exponent(int common, float row) {
    const int k = (P == 2 ? 23 : 15) - common, most = 120;
    return (k < most ? k : most) - above_exponent(row);
}
constexpr float kNoRow = 0.5f;  // a row's factor of 1: below 2^0

// One row of A holds, for each block of 32 r, the block's 32 first pieces and then (P = 2) its 32
// second pieces: 64 P bytes.  Row strides are multiples of 128 bytes, R is padded with zeros to them.
struct GradGemmArgs {
    const uint8_t* a;      // [>= I rows][lda bytes]
    int64_t lda;           // bytes; 256 rows stay below 2^30
    const int8_t* b;       // [R][ldb], 16-byte aligned rows
    int64_t ldb;
    int64_t I, J, R;       // J % 16 == 0
    GradFactors factors;   // A's scale
    void* c;               // fp32 or bf16 [I][ldc]
    int64_t ldc;
    int64_t slab;          // elements between the outputs of two splits of R (fp32)
    int64_t wide_rows;     // the first rows of C by 256 x 256 tiles (a multiple of 256, or all), the rest by 64 x 256
    int splits;
    bool accumulate;       // add to what C holds
    bool bf16_out;
};

hipError_t launch_grad_gemm(const GradGemmArgs& a, int pieces, hipStream_t stream);

// The rows that 256 x 256 tiles take and the splits of R (at most max_splits; each writes a slab that is summed
// later) that a product takes, and about how long it runs, in us.
struct GradShape {
    int64_t wide_rows;
    int splits;
    float cost;
};
GradShape grad_shape(int64_t I, int64_t J, int64_t R, int pieces, int min_splits, int max_splits);

}  // namespace dfssm
