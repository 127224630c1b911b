// int8_gemm.hip -- the int8 product with one scale per token and one per channel (gfx950):
//
//   acc[m][n] = sum_k W[n][k] x_q[m][k]             (exact int32)
//   y[m][n]   = s_x[m] * (s_w[n] * acc[m][n])       (fp32, two roundings; rounded once more to bf16)
//
// for any number of tokens: the LM head over a whole prompt, or an int8 layer.  The tile
// product is tile_i8.h's.  The epilogue turns each 32-token block of a wave through LDS, so
// that lanes write runs of a token's row instead of 16-byte pieces of 32 rows.
//
// What bounds it: many tokens, the products under the power limit and, in bursts that nothing overlaps, the stores
// (2048 x 50280 x 2048: 241 us for bf16; the loss over the same logits 218); few tokens, reading w once
// (50280 x 2048, 1 to 64 tokens: 17 to 19 us, 5.5 to 6 TB/s); few rows, the latency of K's chunks in a workgroup, and
// CUs without one (1 x 2048 x 4096: 6.1 us, 64 workgroups).  For up to 16 tokens it is faster than the head's GEMV
// (int8_head.hip; 50280 x 2048 20.9 against 24.5 us in a graph over uncached copies, 8512 x 2048 7.4 against 16.2).
// Measured and not kept (before the rest of a last round went to small tiles): stores past the caches (275 against 276 us for 412 MB, 545 against 517 for 824), device-scope
// stores (333), two smaller tiles to a CU so that stores overlap products (310 streamed, 337 not).
#include <type_traits>

#include "tile_i8.h"

namespace dfssm {

namespace {

struct GemmArgs {
    const int8_t* x_q;
    int64_t ldx;
    const float* s_x;
    const int8_t* w;
    int64_t ldw;
    const float* s_w;
    void* y;
    int64_t ldy;
    int64_t M, N;
    int K, ntw, ntt;
};

typedef uint32_t v2u __attribute__((ext_vector_type(2)));

template <class C, bool kFast, bool kBf16>
__global__ __launch_bounds__(C::NT, C::kMinWaves) void int8_gemm_kernel(GemmArgs a) {
    constexpr int kLd = C::WB * 32 + 4;  // floats per token row of a wave's LDS block
    constexpr int kEpi = C::WW * C::TW * 32 * kLd * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLdsBytes > kEpi ? C::kLdsBytes : kEpi];
    const TilePos pos = tile_pos(blockIdx.x, a.ntw, a.ntt);
    const int64_t n0 = (int64_t)pos.w * C::BW, m0 = (int64_t)pos.t * C::BT;
    const int wrows = (int)(a.N - n0 < C::BW ? a.N - n0 : C::BW);
    const int trows = (int)(a.M - m0 < C::BT ? a.M - m0 : C::BT);
    v16i acc[C::WB][C::TB];
    const bool holds = tile_i8<C, kFast>(a.w + n0 * a.ldw, a.ldw, wrows, a.x_q + m0 * a.ldx, a.ldx, trows, a.K, lds, acc);

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int ww = wave % C::WW, tw = wave / C::WW;
    const int l32 = lane & 31, g = lane >> 5;
    const int wn = ww * C::WB * 32;            // the wave's first weight row in the tile
    const int live_n = wrows - wn;             // outputs of a token that exist in the wave's range
    lds_barrier();
    if (!holds) return;  // (no barrier follows)
    float* const blk = reinterpret_cast<float*>(lds) + wave * 32 * kLd;
    // the lane's row scales: rows past N are clamped (their outputs are not stored)
    float sw[C::WB][16];
#pragma unroll
    for (int b = 0; b < C::WB; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int r = wn + b * 32 + 8 * (v >> 2) + 4 * g + (v & 3);
            sw[b][v] = a.s_w[n0 + (r < wrows ? r : wrows - 1)];
        }
#pragma unroll
    for (int tb = 0; tb < C::TB; ++tb) {
        const int t0 = (tw * C::TB + tb) * 32;
        const float sx = a.s_x[m0 + (t0 + l32 < trows ? t0 + l32 : trows - 1)];
#pragma unroll
        for (int b = 0; b < C::WB; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v4f o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = sx * (sw[b][4 * q + e] * (float)acc[b][tb][4 * q + e]);
                *reinterpret_cast<v4f*>(blk + l32 * kLd + b * 32 + 8 * q + 4 * g) = o;
            }
        // (the block is the wave's own)
        wave_lds_order();
        constexpr int L = C::WB * 8;  // lanes per token row, four outputs each
        const int c = (lane % L) * 4;
#pragma unroll
        for (int r = 0; r < 32; r += kWave / L) {
            const int tr = r + lane / L;
            const v4f o = *reinterpret_cast<const v4f*>(blk + tr * kLd + c);
            if (t0 + tr < trows && c < live_n) {
                const int64_t at = (m0 + t0 + tr) * a.ldy + n0 + wn + c;
                if (c + 4 <= live_n) {
                    // four outputs at any address (rows of 20001 fp32 x 2000 tokens x 784: 71 us, as rows of 20000;
                    // element by element 104, in runs of a row by elements 77)
                    if constexpr (kBf16) {
                        const v2u p = {bf16_bits(o.x) | (bf16_bits(o.y) << 16), bf16_bits(o.z) | (bf16_bits(o.w) << 16)};
                        __builtin_memcpy(static_cast<uint16_t*>(a.y) + at, &p, 8);
                    } else {
                        __builtin_memcpy(static_cast<float*>(a.y) + at, &o, 16);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < live_n) {
                            if constexpr (kBf16) static_cast<uint16_t*>(a.y)[at + e] = (uint16_t)bf16_bits(o[e]);
                            else static_cast<float*>(a.y)[at + e] = o[e];
                        }
                }
            }
        }
        wave_lds_order();
    }
}

template <bool kFast, bool kBf16>
hipError_t launch_kind(GemmArgs a, int kind, hipStream_t stream) {
    return with_tile(kind, [&](auto tile) {
        using T = decltype(tile);
        using C = std::conditional_t<kFast || T::BW * T::BT < 65536, T, TileI8<2, 2, 2, 2>>;
        a.ntw = (int)((a.N + C::BW - 1) / C::BW);
        a.ntt = (int)((a.M + C::BT - 1) / C::BT);
        const dim3 grid((unsigned)((int64_t)a.ntw * a.ntt));
        int8_gemm_kernel<C, kFast, kBf16><<<grid, C::NT, 0, stream>>>(a);
        return hipGetLastError();
    });
}

template <bool kFast, bool kBf16>
hipError_t launch_tiles(const GemmArgs& a, hipStream_t stream) {
    // (unaligned rows take more registers to stage: not with the largest tile)
    const TileSplit split = split_rows(a.N, a.M, a.K, kFast ? kTile256 : kTile256x192);
    GemmArgs part = a;
    part.N = split.main;
    if (hipError_t err = launch_kind<kFast, kBf16>(part, split.kind, stream)) return err;
    if (split.main == a.N) return hipSuccess;
    part.N = a.N - split.main;
    part.w = a.w + split.main * a.ldw;
    part.s_w = a.s_w + split.main;
    part.y = static_cast<uint8_t*>(a.y) + split.main * (kBf16 ? 2 : 4);
    return launch_kind<kFast, kBf16>(part, split.tail, stream);
}

}  // namespace

hipError_t launch_int8_gemm(const int8_t* x_q, int64_t ldx, const float* s_x, int64_t M, int64_t N, int64_t K,
                            const int8_t* w, int64_t ldw, const float* s_w, void* y, int64_t ldy, bool bf16,
                            hipStream_t stream) {
    auto al16 = [](const void* p) { return ((uintptr_t)p & 15u) == 0; };
    const bool fast = al16(x_q) && al16(w) && ldx % 16 == 0 && ldw % 16 == 0 && K % 16 == 0;
    // A launch holds at most 2^32 threads: larger products go slice by slice.
    constexpr int64_t kRows = (int64_t)1 << 20, kTokens = (int64_t)1 << 17;
    for (int64_t n0 = 0; n0 < N; n0 += kRows)
        for (int64_t m0 = 0; m0 < M; m0 += kTokens) {
            const GemmArgs a{x_q + m0 * ldx, ldx, s_x + m0, w + n0 * ldw, ldw, s_w + n0,
                             static_cast<uint8_t*>(y) + (m0 * ldy + n0) * (bf16 ? 2 : 4), ldy,
                             M - m0 < kTokens ? M - m0 : kTokens, N - n0 < kRows ? N - n0 : kRows, (int)K, 0, 0};
            const hipError_t err = fast ? (bf16 ? launch_tiles<true, true>(a, stream) : launch_tiles<true, false>(a, stream))
                                        : (bf16 ? launch_tiles<false, true>(a, stream) : launch_tiles<false, false>(a, stream));
            if (err) return err;
        }
    return hipSuccess;
}

}  // namespace dfssm
