// cross_entropy.hip -- softmax cross entropy over the int8 vocabulary matrix, and its gradients
// (gfx950), without the M x V logits in memory:
//
//   z[m][v] = s_x[m] (s_e[v] sum_k e[v][k] x_q[m][k])      lse[m] = log sum_v exp z[m][v]
//   loss[m] = lse[m] - z[m][target]                          (0 where the target is no row of e)
//   d[m][v] = dloss[m] (exp(z[m][v] - lse[m]) - [v = target])
//   dx[m]   = sum_v d[m][v] s_e[v] e[v]        de[v] = sum_m d[m][v] s_x[m] x_q[m]
//
// Forward: each workgroup forms a tile of logits (tile_i8.h: exact int32 accumulators, a token per
// lane, the vocabulary along its registers), takes each token's maximum and sum of exponentials over
// the tile's rows, and writes that pair; a second kernel joins a token's pairs in tile order and
// forms the target's logit by itself.  Exponents are base 2: z log2 e.
//
// Backward, one piece of the vocabulary at a time: a tile kernel forms the piece's logits again and
// from them d, twice: d s_e with the vocabulary contiguous (for dx) and d s_x with the tokens contiguous
// (for de), in 16-bit pieces (grad_gemm.h); two products with the codes then give the piece's rows of de
// and its share of dx.  The gradient's type sets the pieces: fp32 takes two (relative error at most
// 2^-19 of each d: below the summation's where sums are long, above it where they are short, de of 64 tokens 6.6e-7 against
// 64 bits), bf16 one (2^-11, an eighth of the final rounding).  Recomputing the logits costs one
// int8 product; keeping them would cost 4 M V bytes written and read.
//
// What bounds it: forward, the int8 products under the power limit (tile_i8.h); backward, 4096 tokens x 50280 rows x
// 2048 fp32 in 3.3 ms: the products for dx and de 1.28 and 1.34 ms (grad_gemm.h), the gradient tiles 0.67 ms, of which
// about 0.25 are their 8 bytes a logit (1.6 GB), written in bursts between the products.
#include <math.h>

#include "grad_gemm.h"
#include "tile_i8.h"

namespace dfssm {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.69314718055994530942;

struct LossArgs {
    const int8_t* x_q;
    const float* s_x;
    int64_t M, V;
    int K, ntw, ntt;
    const int8_t* e;
    const float* s_e;
    float2* part;   // [ntw][M]: a tile's maximum (of z log2 e) and sum of 2^(z log2 e - maximum)
};

// ---------------------------------------------------------------- forward
template <class C>
__global__ __launch_bounds__(C::NT, C::kMinWaves) void loss_tile_kernel(LossArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLdsBytes];
    const TilePos pos = tile_pos(blockIdx.x, a.ntw, a.ntt);
    const int64_t n0 = (int64_t)pos.w * C::BW, m0 = (int64_t)pos.t * C::BT;
    const int wrows = (int)(a.V - n0 < C::BW ? a.V - n0 : C::BW);
    const int trows = (int)(a.M - m0 < C::BT ? a.M - m0 : C::BT);
    v16i acc[C::WB][C::TB];
    const bool holds = tile_i8<C, true>(a.e + n0 * a.K, a.K, wrows, a.x_q + m0 * a.K, a.K, trows, a.K, lds, acc);

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int ww = wave % C::WW, tw = wave / C::WW;
    const int l32 = lane & 31, g = lane >> 5;
    const int wn = ww * C::WB * 32;
    float se[C::WB][16];
#pragma unroll
    for (int b = 0; b < C::WB; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int r = wn + b * 32 + 8 * (v >> 2) + 4 * g + (v & 3);
            se[b][v] = a.s_e[n0 + (r < wrows ? r : wrows - 1)];
        }
    lds_barrier();
    float2* const red = reinterpret_cast<float2*>(lds);  // [WW][BT]
    const float neg = -__builtin_inff();
#pragma unroll
    for (int tb = 0; tb < C::TB && holds; ++tb) {
        const int t = (tw * C::TB + tb) * 32 + l32;
        const float sx2 = a.s_x[m0 + (t < trows ? t : trows - 1)] * kLog2e;
        float z[C::WB][16], top = neg;
#pragma unroll
        for (int b = 0; b < C::WB; ++b)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                z[b][v] = sx2 * (se[b][v] * (float)acc[b][tb][v]);
                if (wrows < C::BW && wn + b * 32 + 8 * (v >> 2) + 4 * g + (v & 3) >= wrows) z[b][v] = neg;
                top = fmaxf(top, z[b][v]);
            }
        const float base = top == neg ? 0.0f : top;  // (no row of the wave's range exists, or all are -infinity)
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < C::WB; ++b)
#pragma unroll
            for (int v = 0; v < 16; ++v) sum += __builtin_amdgcn_exp2f(z[b][v] - base);
        // the two halves of the wave hold the same tokens
        const float otop = __shfl_xor(top, 32), osum = __shfl_xor(sum, 32);
        const float both = fmaxf(top, otop), b2 = both == neg ? 0.0f : both;
        sum = g == 0 ? sum * __builtin_amdgcn_exp2f(top - b2) + osum * __builtin_amdgcn_exp2f(otop - b2) : 0.0f;
        if (g == 0) red[ww * C::BT + t] = make_float2(both, sum);
    }
    lds_barrier();
    for (int t = threadIdx.x; t < trows; t += C::NT) {
        float top = neg;
#pragma unroll
        for (int w = 0; w < C::WW; ++w) top = fmaxf(top, red[w * C::BT + t].x);
        const float base = top == neg ? 0.0f : top;  // (every logit of the tile may be -infinity)
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < C::WW; ++w) sum += red[w * C::BT + t].y * __builtin_amdgcn_exp2f(red[w * C::BT + t].x - base);
        a.part[(int64_t)pos.w * a.M + m0 + t] = make_float2(top, sum);
    }
}

// Joins the tiles' pairs in tile order and forms the target's logit: 16 tokens to a workgroup of
// 1024 threads, 64 threads to a token (one wave).
__global__ __launch_bounds__(1024) void loss_join_kernel(LossArgs a, const int32_t* __restrict__ targets,
                                                         float* __restrict__ loss, float* __restrict__ lse) {
    // pairs[wave][token]: a wave reads 16 tokens x 4 tiles, consecutive tokens side by side
    __shared__ float2 pairs[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m0 = (int64_t)blockIdx.x * 16;
    const float neg = -__builtin_inff();
    float top = neg, sum = 0.0f;
    if (m0 + (lane & 15) < a.M)
        for (int w = wave * 4 + (lane >> 4); w < a.ntw; w += 64) {
            const float2 p = a.part[(int64_t)w * a.M + m0 + (lane & 15)];
            const float t = fmaxf(top, p.x), base = t == neg ? 0.0f : t;
            sum = sum * __builtin_amdgcn_exp2f(top - base) + p.y * __builtin_amdgcn_exp2f(p.x - base);
            top = t;
        }
    pairs[wave][lane] = make_float2(top, sum);
    __syncthreads();
    const int64_t m = m0 + wave;
    if (m >= a.M) return;
    // lane i holds pair i of the wave's token: waves i / 4, tile classes i % 4
    const float2 p = pairs[lane >> 2][(lane & 3) * 16 + wave];
    const float all = wave_max(p.x);
    float s = p.y == 0.0f ? 0.0f : p.y * __builtin_amdgcn_exp2f(p.x - all);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    const float l = (float)(((double)all + (double)__log2f(s)) * kLn2);  // (one rounding, of the result)

    const int32_t target = targets[m];
    float out = 0.0f;
    if (target >= 0 && target < a.V) {
        const int8_t* x = a.x_q + m * a.K;
        const int8_t* e = a.e + (int64_t)target * a.K;
        int32_t dot = 0;
        for (int k = lane * 16; k < a.K; k += 64 * 16) {
            const v4i xv = *reinterpret_cast<const v4i*>(x + k), ev = *reinterpret_cast<const v4i*>(e + k);
#pragma unroll
            for (int j = 0; j < 4; ++j) dot = __builtin_amdgcn_sdot4(xv[j], ev[j], dot, false);
        }
        dot = wave_sum(dot);
        out = l - a.s_x[m] * (a.s_e[target] * (float)dot);
    }
    if (lane == 0) {
        lse[m] = l;
        loss[m] = out;
    }
}

// ---------------------------------------------------------------- backward
struct GradArgs {
    const int8_t* x_q;
    const float* s_x;
    int64_t M, V;    // V: rows of the piece (a piece starts at v0)
    int64_t v0, vocab;
    int K, ntw, ntt;
    const int8_t* e;     // the piece's rows and scales
    const float* s_e;
    const int32_t* targets;
    const float* lse;
    const float* dloss;
    const float* maxima; // [2][kMaximaBlocks]: of |s_e|, |dloss s_x| (tokens that count)
    uint16_t* gx;        // [tokens][Vp P]: d s_e, or NULL
    uint16_t* gw;        // [Vp][Mp P]: d s_x, or NULL
    int64_t ldgx, ldgw;  // elements
};

// Partial maxima of what bounds d s_e (with the token's dloss) and d s_x (|p - [v = target]| <= 1): they scale d into
// fp16's range.  An infinite dloss s_x takes no part: its own gradients are infinite or NaN at any scale, and the others
// keep theirs.
__global__ __launch_bounds__(256) void grad_maxima_kernel(const float* __restrict__ s_e, int64_t V,
                                                          const float* __restrict__ s_x,
                                                          const float* __restrict__ dloss,
                                                          const int32_t* __restrict__ targets, int64_t M,
                                                          float* __restrict__ maxima) {
    __shared__ float part[2][4];
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)kMaximaBlocks * 256;
    float e = 0.0f, dx = 0.0f;
    for (int64_t i = first; i < V; i += step) e = fmaxf(e, fabsf(s_e[i]));
    for (int64_t i = first; i < M; i += step) {
        const int64_t target = targets[i];
        if (target >= 0 && target < V) {
            const float lx = fabsf(dloss[i] * s_x[i]);
            if (lx < __builtin_inff()) dx = fmaxf(dx, lx);
        }
    }
    e = wave_max(e);
    dx = wave_max(dx);
    if ((threadIdx.x & 63) == 0) {
        part[0][threadIdx.x >> 6] = e;
        part[1][threadIdx.x >> 6] = dx;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        const float* p = part[threadIdx.x];
        maxima[threadIdx.x * kMaximaBlocks + blockIdx.x] = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
    }
}

// Two values rounded to bf16 or fp16, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, (v2bf){(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ uint32_t pack_fp16(float a, float b) {
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, (v2h){(_Float16)a, (_Float16)b});
}

// Four values in pieces: with two, rounded to bf16 and the remainders to fp16; with one, rounded to fp16.
template <int P>
__device__ __forceinline__ void split4(const float (&x)[4], uint2& first, uint2& second) {
    if constexpr (P == 2) {
        first = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        second = make_uint2(
            pack_fp16(x[0] - __uint_as_float(first.x << 16), x[1] - __uint_as_float(first.x & 0xFFFF0000u)),
            pack_fp16(x[2] - __uint_as_float(first.y << 16), x[3] - __uint_as_float(first.y & 0xFFFF0000u)));
    } else {
        first = make_uint2(pack_fp16(x[0], x[1]), pack_fp16(x[2], x[3]));
    }
}

// A 32 x 32 block of pieces from a wave's LDS block to memory: 16 bytes a lane, whole rows of 64 P bytes.
template <int P>
__device__ __forceinline__ void store_block(const uint8_t* blk, int ld_blk, uint16_t* dst, int64_t ld, int lane) {
    constexpr int L = 4 * P;  // lanes per row
#pragma unroll
    for (int r = 0; r < 32; r += kWave / L) {
        const int row = r + lane / L;
        const v4i v = *reinterpret_cast<const v4i*>(blk + row * ld_blk + (lane % L) * 16);
        *reinterpret_cast<v4i*>(dst + row * ld + (lane % L) * 8) = v;
    }
}

// What lies past the vocabulary or the tokens inside the padded buffers is zero: the products read it against zero
// codes, and an infinite one would make them NaN.  Both forms of d go through LDS, so that memory is written in whole
// rows of a block (64 P bytes): written from the registers, d s_x would go out in 2-byte stores.
template <class C, int P>
__global__ __launch_bounds__(C::NT, C::kMinWaves) void grad_tile_kernel(GradArgs a) {
    constexpr int kLd = 64 * P + 16;            // a block row in LDS
    constexpr int kBlk = 2 * 32 * kLd;          // a wave's two blocks
    static_assert(C::WW * C::TW * kBlk <= C::kLdsBytes, "the epilogue's blocks fit the tile's buffers");
    __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLdsBytes];
    const TilePos pos = tile_pos(blockIdx.x, a.ntw, a.ntt);
    const int64_t n0 = (int64_t)pos.w * C::BW, m0 = (int64_t)pos.t * C::BT;
    const int wrows = (int)(a.V - n0 < C::BW ? a.V - n0 : C::BW);
    const int trows = (int)(a.M - m0 < C::BT ? a.M - m0 : C::BT);
    const int lane = threadIdx.x & (kWave - 1);
    const float max_e = a.maxima[lane], max_dx = a.maxima[kMaximaBlocks + lane];
    v16i acc[C::WB][C::TB];
    const bool holds = tile_i8<C, true>(a.e + n0 * a.K, a.K, wrows, a.x_q + m0 * a.K, a.K, trows, a.K, lds, acc);

    const int above_e = above_exponent(wave_max(max_e)), up_w = grad_exponent<P>(above_exponent(wave_max(max_dx)), kNoRow);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int ww = wave % C::WW, tw = wave / C::WW;
    const int l32 = lane & 31, g = lane >> 5;
    const int wn = ww * C::WB * 32;
    float se[C::WB][16];
#pragma unroll
    for (int b = 0; b < C::WB; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int r = wn + b * 32 + 8 * (v >> 2) + 4 * g + (v & 3);
            se[b][v] = a.s_e[n0 + (r < wrows ? r : wrows - 1)];
        }
    lds_barrier();
    if (!holds) return;                         // (no barrier follows)
    uint8_t* const bx = lds + wave * kBlk;      // [token][vocabulary row]
    uint8_t* const bw = bx + 32 * kLd;          // [vocabulary row][token]
#pragma unroll
    for (int tb = 0; tb < C::TB; ++tb) {
        const int t = (tw * C::TB + tb) * 32 + l32;
        const int64_t m = m0 + (t < trows ? t : trows - 1);
        const int64_t target = a.targets[m];
        const bool counts = t < trows && target >= 0 && target < a.vocab;
        // (p is formed from z - lse: in base 2 the roundings of lse log2 e and s_x log2 e would be p's largest errors;
        // 0 where the token does not count, whatever its scale and its logits are: the mask takes out a NaN, too)
        const float sx = counts ? a.s_x[m] : 0.0f, lse = counts ? a.lse[m] : 0.0f;
        const uint32_t keep = counts ? 0xFFFFFFFFu : 0u;
        const float dloss = counts ? a.dloss[m] : 0.0f;
        const float dl = __builtin_amdgcn_ldexpf(dloss, grad_exponent<P>(above_e, dloss));
        const float dlx = __builtin_amdgcn_ldexpf(dloss * sx, up_w);
        const int tl = counts ? (int)(target - a.v0 - n0 - wn) : -1;     // the target's row in the wave's range
#pragma unroll
        for (int b = 0; b < C::WB; ++b) {
            float p[16];
#pragma unroll
            for (int v = 0; v < 16; ++v)
                p[v] = __uint_as_float(keep & __float_as_uint(__builtin_amdgcn_exp2f(
                    __builtin_fmaf(se[b][v] * (float)acc[b][tb][v], sx, -lse) * kLog2e)));
            if (wrows < C::BW) {  // rows that do not exist: their exp(0 - lse) has no bound
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    if (wn + b * 32 + 8 * (v >> 2) + 4 * g + (v & 3) >= wrows) p[v] = 0.0f;
            }
            if (__ballot(tl >= b * 32 && tl < b * 32 + 32)) {
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    if (tl == b * 32 + 8 * (v >> 2) + 4 * g + (v & 3)) p[v] -= 1.0f;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint2 first, second;
                float x[4];
                if (a.gx) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = p[4 * q + j] * dl * se[b][4 * q + j];
                    split4<P>(x, first, second);
                    *reinterpret_cast<uint2*>(bx + l32 * kLd + (8 * q + 4 * g) * 2) = first;
                    if constexpr (P == 2) *reinterpret_cast<uint2*>(bx + l32 * kLd + 64 + (8 * q + 4 * g) * 2) = second;
                }
                if (a.gw) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = p[4 * q + j] * dlx;
                    split4<P>(x, first, second);
                    uint8_t* const dst = bw + (8 * q + 4 * g) * kLd + l32 * 2;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        *reinterpret_cast<uint16_t*>(dst + j * kLd) = (uint16_t)((j < 2 ? first.x : first.y) >> (16 * (j & 1)));
                        if constexpr (P == 2)
                            *reinterpret_cast<uint16_t*>(dst + j * kLd + 64) =
                                (uint16_t)((j < 2 ? second.x : second.y) >> (16 * (j & 1)));
                    }
                }
            }
            wave_lds_order();
            const int64_t nb = n0 + wn + b * 32, mb = m0 + (tw * C::TB + tb) * 32;  // the block's first row and token
            if (a.gx) store_block<P>(bx, kLd, a.gx + mb * a.ldgx + nb * P, a.ldgx, lane);
            if (a.gw) store_block<P>(bw, kLd, a.gw + nb * a.ldgw + mb * P, a.ldgw, lane);
            wave_lds_order();
        }
    }
}

// dx = the sum of its slabs (one for each piece and split), rounded to its type.  Unrolled: with few tokens there are few
// threads, and a load at a time would be its time (5 tokens, 64 slabs: 19 us, 6.3 with 8 in flight).
template <bool kBf16>
__global__ __launch_bounds__(256) void slab_sum_kernel(const float* __restrict__ slabs, int splits, int64_t n,
                                                       void* __restrict__ out) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
        v4f s = *reinterpret_cast<const v4f*>(slabs + i);
#pragma unroll 8
        for (int k = 1; k < splits; ++k) s += *reinterpret_cast<const v4f*>(slabs + k * n + i);
        if constexpr (kBf16) {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + i) =
                make_uint2(bf16_bits(s.x) | (bf16_bits(s.y) << 16), bf16_bits(s.z) | (bf16_bits(s.w) << 16));
        } else {
            *reinterpret_cast<v4f*>(static_cast<float*>(out) + i) = s;
        }
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tiles of the gradient kernel for a piece's rows: of those with 64 tokens or more, so that the padded
// tokens of d s_x fill whole chunks of the product (64 tokens) and are all written.  The smallest splits K
// and only serves a round of the 256 CUs (25 tokens x 11898 rows x 2480 9.8 us, 13.4 by the next one; 4096 x 1128 x 2048,
// in 4 1/2 rounds 41 us, 35 by 256 x 192).
TileSplit grad_tiles(int64_t M, int64_t rows, int64_t K) {
    const int64_t smallest = ((M + 63) / 64) * ((rows + 63) / 64);
    return split_rows(rows, M, K, kTile256, smallest <= 256 ? kTileKinds64 : kTile64x64);
}

// How a backward call is cut and where its workspace lies; the size query and the call agree on it.
struct Plan {
    int64_t Mp;      // tokens padded for every tile: ceil(M / t) t for t = 64, 128, 192 and 256
    int64_t piece;   // vocabulary rows per piece, a multiple of 256
    int splits;      // of dx's sum over a piece
    int slabs;       // fp32 slabs of dx in the workspace; 0: dx itself is the only one
    bool add;        // the pieces add to the same slabs
    size_t maxima, gx, gw, dx, bytes;
};

constexpr int64_t kMaxSlabBytes = (int64_t)512 << 20, kMaxPieceBytes = (int64_t)640 << 20;
constexpr int64_t kMaxSlabs = 256;  // (64 splits of four pieces)

// About how long a piece takes: its gradient tiles and its products (dx with the slabs it adds), and the launches.
float piece_cost(int64_t M, int64_t rows, int64_t K, int P, bool want_dx, bool want_de) {
    const float tiles = 1.35f * grad_tiles(M, rows, K).cost;  // (the epilogue is the heavier one)
    return tiles + (want_dx ? grad_shape(M, K, rows, P, 1, 64).cost : 0.0f) +
           (want_de ? grad_shape(rows, K, M, P, 1, 1).cost : 0.0f) + 4.0f;
}

Plan make_plan(int64_t M, int64_t V, int64_t K, bool bf16, bool want_dx, bool want_de) {
    const int P = bf16 ? 1 : 2;
    Plan p{};
    p.Mp = (M + 255) / 64 * 64;
    // The longest piece whose d takes at most 640 MB (2048 rows at the least); among pieces up to it, the one that
    // wastes least: pieces of equal length, and pieces whose tiles of de fill whole rounds of the 256 CUs, with
    // a short last one (4096 tokens x 50280 rows: 3 pieces of 16384 rows, two rounds each, and a rest, instead of 7 of 7424).
    const int64_t per_row = p.Mp * P * 2 * ((want_dx ? 1 : 0) + (want_de ? 1 : 0));
    const int64_t all = ceil_div(V, 256);
    int64_t most = kMaxPieceBytes / per_row / 256;
    if (most < 8) most = 8;
    if (most > all) most = all;
    float best = 3.0e38f;
    auto consider = [&](int64_t k) {
        if (k < 1 || k > most || k < most / 4) return;
        const int64_t rows = k * 256, full = V / rows, rest = V - full * rows;
        const float cost = (float)full * piece_cost(M, rows, K, P, want_dx, want_de) +
                           (rest ? piece_cost(M, rest, K, P, want_dx, want_de) : 0.0f);
        if (cost < best) {
            best = cost;
            p.piece = rows;
        }
    };
    const int64_t fewest = ceil_div(all, most), tj = ceil_div(K, 256);
    for (int64_t n = fewest; n < fewest + 6; ++n) consider(ceil_div(all, n));
    for (int64_t r = 1; r <= 4; ++r) consider(256 * r / tj);
    size_t at = 0;
    auto take = [&](size_t b) {
        const size_t was = at;
        at += (b + 255) / 256 * 256;
        return was;
    };
    p.maxima = take(2 * kMaximaBlocks * sizeof(float));
    if (want_dx) {
        // Each piece has slabs of its own, summed at the end: adding to a slab at the end of every piece's
        // product costs more (all workgroups read and write at once, and nothing else runs).  Not past 512 MB or 256 slabs.
        const int64_t pieces = ceil_div(V, p.piece), slab = M * K * 4;
        const int64_t most_slabs = kMaxSlabBytes / slab < kMaxSlabs ? kMaxSlabBytes / slab : kMaxSlabs;
        const int64_t room = most_slabs / pieces;
        p.add = pieces > 1 && room < 1;
        p.splits = grad_shape(M, K, p.piece < V ? p.piece : V, P, 1, (int)(p.add || room < 1 ? 1 : room > 64 ? 64 : room)).splits;
        p.slabs = (int)(p.add ? p.splits : pieces * p.splits);
        if (p.slabs == 1 && !bf16) p.slabs = 0;
        p.gx = take((size_t)(p.Mp * p.piece * P * 2));
        p.dx = take((size_t)(p.slabs * slab));
    }
    if (want_de) p.gw = take((size_t)(p.piece * p.Mp * P * 2));
    // The workspace is what the limits above allow, not what this plan takes (at most that): plans of shorter batches may
    // take more, and a size that never falls as M, V or K grows serves them all.
    int64_t d = kMaxPieceBytes > 8 * 256 * per_row ? kMaxPieceBytes : 8 * 256 * per_row, slabs = 0;
    if (d > all * 256 * per_row) d = all * 256 * per_row;
    if (want_dx) {
        const int64_t slab = M * K * 4, few = slab * kMaxSlabs < kMaxSlabBytes ? slab * kMaxSlabs : kMaxSlabBytes;
        slabs = slab > few ? slab : few;
    }
    p.bytes = (size_t)(2 * kMaximaBlocks * sizeof(float) + d + (slabs + 255) / 256 * 256);
    return p;
}

template <int P>
hipError_t launch_grad_kind(GradArgs a, int kind, hipStream_t stream) {
    return with_tile(kind, [&](auto tile) {
        using C = decltype(tile);
        if constexpr (C::BT >= 64) {
            a.ntt = (int)ceil_div(a.M, C::BT);
            a.ntw = (int)ceil_div(a.V, C::BW);
            grad_tile_kernel<C, P><<<dim3((unsigned)(a.ntw * a.ntt)), C::NT, 0, stream>>>(a);
            return hipGetLastError();
        } else {
            return hipErrorInvalidValue;
        }
    });
}

template <int P>
hipError_t launch_grad_tiles(const GradArgs& a, hipStream_t stream) {
    const TileSplit split = grad_tiles(a.M, a.V, a.K);
    GradArgs part = a;
    part.V = split.main;
    if (hipError_t err = launch_grad_kind<P>(part, split.kind, stream)) return err;
    if (split.main == a.V) return hipSuccess;
    part.V = a.V - split.main;
    part.v0 = a.v0 + split.main;
    part.e = a.e + split.main * a.K;
    part.s_e = a.s_e + split.main;
    if (a.gx) part.gx = a.gx + split.main * P;
    if (a.gw) part.gw = a.gw + split.main * a.ldgw;
    return launch_grad_kind<P>(part, split.tail, stream);
}

hipError_t launch_loss_kind(LossArgs a, int kind, hipStream_t stream) {
    return with_tile(kind, [&](auto tile) {
        using C = decltype(tile);
        a.ntw = (int)ceil_div(a.V, C::BW);
        a.ntt = (int)ceil_div(a.M, C::BT);
        loss_tile_kernel<C><<<dim3((unsigned)((int64_t)a.ntw * a.ntt)), C::NT, 0, stream>>>(a);
        return hipGetLastError();
    });
}

// Row tiles of the forward pass: of the main rows, and of all.
int64_t main_row_tiles(const TileSplit& s) { return ceil_div(s.main, tile_shape(s.kind).rows); }
int64_t row_tiles(const TileSplit& s, int64_t V) {
    return main_row_tiles(s) + (s.main < V ? ceil_div(V - s.main, tile_shape(s.tail).rows) : 0);
}

// The tiles' pairs that the forward pass has room for: all that tiles of 128 rows or more write, and 2^20, so that few
// tokens may take smaller ones.  It grows with M and V: a longer batch's workspace serves a shorter one.
int64_t most_pairs(int64_t M, int64_t V) { return M * ceil_div(V, 128) + ((int64_t)1 << 20); }

// The forward pass's tiles.  (Past that room, of few shapes and at most 8 % by the cost: 320 tokens x 430248 rows x 32 with
// 64 rows a tile.)
TileSplit loss_tiles(int64_t M, int64_t V, int64_t K) {
    const TileSplit s = split_rows(V, M, K);
    return row_tiles(s, V) * M <= most_pairs(M, V) ? s : split_rows(V, M, K, kTile256, kTileKinds128);
}

}  // namespace

size_t cross_entropy_workspace_bytes(int64_t M, int64_t V, int64_t K) {
    (void)K;
    return (size_t)most_pairs(M, V) * sizeof(float2);
}

hipError_t launch_cross_entropy(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K, const int8_t* e,
                                const float* s_e, const int32_t* targets, float* loss, float* lse, void* workspace,
                                hipStream_t stream) {
    LossArgs a{x_q, s_x, M, V, (int)K, 0, 0, e, s_e, static_cast<float2*>(workspace)};
    const TileSplit split = loss_tiles(M, V, K);
    a.V = split.main;
    if (hipError_t err = launch_loss_kind(a, split.kind, stream)) return err;
    if (split.main < V) {
        LossArgs rest = a;
        rest.V = V - split.main;
        rest.e = e + split.main * K;
        rest.s_e = s_e + split.main;
        rest.part = a.part + main_row_tiles(split) * M;
        if (hipError_t err = launch_loss_kind(rest, split.tail, stream)) return err;
    }
    a.V = V;
    a.ntw = (int)row_tiles(split, V);
    loss_join_kernel<<<dim3((unsigned)ceil_div(M, 16)), 1024, 0, stream>>>(a, targets, loss, lse);
    return hipGetLastError();
}

size_t cross_entropy_backward_workspace_bytes(int64_t M, int64_t V, int64_t K, bool bf16, bool want_dx, bool want_de) {
    return make_plan(M, V, K, bf16, want_dx, want_de).bytes;
}

hipError_t launch_cross_entropy_backward(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K,
                                         const int8_t* e, const float* s_e, const int32_t* targets, const float* lse,
                                         const float* dloss, void* dx, void* de, bool bf16, bool accumulate,
                                         void* workspace, hipStream_t stream) {
    const Plan p = make_plan(M, V, K, bf16, dx != nullptr, de != nullptr);
    const int P = bf16 ? 1 : 2;
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    float* const maxima = reinterpret_cast<float*>(ws + p.maxima);
    grad_maxima_kernel<<<kMaximaBlocks, 256, 0, stream>>>(s_e, V, s_x, dloss, targets, M, maxima);
    if (hipError_t err = hipGetLastError()) return err;
    for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
        const int64_t rows = V - v0 < p.piece ? V - v0 : p.piece;
        GradArgs g{x_q, s_x, M, rows, v0, V, (int)K, 0, 0, e + v0 * K, s_e + v0, targets, lse, dloss, maxima,
                   dx ? reinterpret_cast<uint16_t*>(ws + p.gx) : nullptr,
                   de ? reinterpret_cast<uint16_t*>(ws + p.gw) : nullptr, p.piece * P, p.Mp * P};
        if (hipError_t err = P == 1 ? launch_grad_tiles<1>(g, stream) : launch_grad_tiles<2>(g, stream)) return err;
        if (dx) {
            float* const slab = reinterpret_cast<float*>(ws + p.dx) + (p.add ? 0 : v0 / p.piece * p.splits * M * K);
            const GradGemmArgs a{ws + p.gx, p.piece * P * 2, g.e, K, M, K, rows, {maxima, dloss}, p.slabs ? slab : dx, K, M * K,
                                 grad_shape(M, K, rows, P, p.splits, p.splits).wide_rows, p.splits, p.add && v0 > 0, false};
            if (hipError_t err = launch_grad_gemm(a, P, stream)) return err;
        }
        if (de) {
            const GradGemmArgs a{ws + p.gw, p.Mp * P * 2, x_q, K, rows, K, M, {maxima + kMaximaBlocks, nullptr},
                                 static_cast<uint8_t*>(de) + v0 * K * (bf16 ? 2 : 4), K, 0,
                                 grad_shape(rows, K, M, P, 1, 1).wide_rows, 1, accumulate, bf16};
            if (hipError_t err = launch_grad_gemm(a, P, stream)) return err;
        }
    }
    if (dx && p.slabs) {
        const int64_t n = M * K;
        int64_t blocks = ceil_div(n, 1024);
        if (blocks > 2048) blocks = 2048;
        const float* slabs = reinterpret_cast<const float*>(ws + p.dx);
        if (bf16) slab_sum_kernel<true><<<dim3((unsigned)blocks), 256, 0, stream>>>(slabs, p.slabs, n, dx);
        else slab_sum_kernel<false><<<dim3((unsigned)blocks), 256, 0, stream>>>(slabs, p.slabs, n, dx);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace dfssm
