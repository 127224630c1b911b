// grad_gemm.h -- products of bf16 gradients with int8 codes (gfx950), private to the library:
//
//   C[i][j] (+)= sum_r A[i][r] * B[r][j]
//
// A holds fp32 values as one bf16 piece (P = 1: the value rounded, relative error at most 2^-8) or two
// (P = 2: the rounded value and the rounded remainder, 2^-16), B int8 codes, which bf16 holds exactly, so the
// pieces' products are exact and only the fp32 accumulation rounds besides.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dfssm {

// One row of A holds, for each block of 32 r, the block's 32 first pieces and then (P = 2) its 32
// second pieces: 64 P bytes.  Row strides are multiples of 128 bytes, R is padded with zeros to them.
struct GradGemmArgs {
    const uint8_t* a;      // [>= I rows][lda bytes]
    int64_t lda;           // bytes; 256 rows stay below 2^30
    const int8_t* b;       // [R][ldb], 16-byte aligned rows
    int64_t ldb;
    int64_t I, J, R;       // J % 16 == 0
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
