// grad_gemm.hip -- C (+)= A B for gradients A in bf16 and fp16 pieces and int8 codes B (gfx950; see grad_gemm.h).
//
// v_mfma_f32_32x32x16_{bf16,f16} with A's rows from LDS as they lie in memory (128-byte chunks, pieces
// swizzled as in tile_i8.h) and B's codes in LDS as bytes, row by row.  B's fragment needs 8
// consecutive r of one column: ds_read_b64_tr_b8 transposes 8 rows x 16 columns of bytes on the
// way to the registers, where the codes become bf16 and fp16 (exact).  Keeping B as bytes in memory and
// LDS halves its traffic and needs no transposed copy.  C's columns run along the lanes, so stores are runs of a row.
//
// What bounds it: the matrix cores under the power limit.  7424 x 2048 x 4096 with two pieces ran 187 us (1.33 PFLOP/s of
// products; the large bf16 product of the library reaches 1.41 on this GPU), at 2.0 GHz and 58 % of the matrix cores' cycles.
// On the way: 214 us with the loads sunk to a chunk's end and LDS conflicts, 203 with both mended, 197 with the
// staging spread between the products, 187 with the third LDS buffer.
#include <type_traits>

#include "device_common.h"
#include "grad_gemm.h"

namespace dfssm {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kLoadDead = 0x40000000;  // a load offset past every resource used here (below 2^30): reads zero

template <int MB_, int NB_, int MW_, int NW_>
struct GradTile {
    static constexpr int MB = MB_, NB = NB_, MW = MW_, NW = NW_;
    static constexpr int BM = 32 * MB * MW, BN = 32 * NB * NW, NT = kWave * MW * NW;
};

// Four codes (bytes of w) as bf16 and as fp16, two words each.  An integer of 8 bits leaves the low half of
// its fp32 form zero, so the high half is its bf16 form.
__device__ __forceinline__ void codes4_both(int w, uint32_t& b0, uint32_t& b1, uint32_t& h0, uint32_t& h1) {
    const float f0 = (float)(int8_t)w, f1 = (float)(int8_t)(w >> 8), f2 = (float)(int8_t)(w >> 16),
                f3 = (float)(w >> 24);
    b0 = perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
    b1 = perm(__float_as_uint(f3), __float_as_uint(f2), 0x07060302u);
    h0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f0, f1));
    h1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f2, f3));
}

// As fp16 alone: a byte u = code + 128 under the high byte 0x64 is the fp16 number 1024 + u; subtracting
// 1152 leaves the code.
__device__ __forceinline__ void codes4_fp16(int w, uint32_t& h0, uint32_t& h1) {
    const uint32_t u = (uint32_t)w ^ 0x80808080u;
    const v2h off = {(_Float16)1152.0f, (_Float16)1152.0f};
    h0 = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, perm(0x64646464u, u, 0x04010400u)) - off);
    h1 = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, perm(0x64646464u, u, 0x04030402u)) - off);
}

// kRows: A's rows have factors of their own.
template <class C, int P, bool kBf16, bool kAdd, bool kRows>
__global__ __launch_bounds__(C::NT, C::NT / 256) void grad_gemm_kernel(GradGemmArgs a, int nti, int ntj,
                                                                      int chunks_per_split) {
    constexpr int kR = 64 / P;              // r per chunk: 128 bytes of an A row
    constexpr int kLdB = C::BN + 16;        // 8 rows x 16 bytes read together hit distinct banks
    constexpr int kA = C::BM * 128, kBuf = kA + kR * kLdB;
    constexpr int PA = C::BM * 8 / C::NT;   // 16-byte pieces per thread per chunk
    constexpr int PB = kR * C::BN / 16 / C::NT;
    constexpr int TB = C::BN / 16;          // threads per B row
    static_assert(PA * C::NT == C::BM * 8 && PB * C::NT * 16 == kR * C::BN && PB >= 1, "pieces split evenly");
    static_assert(3 * kBuf <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(16))) uint8_t lds[3 * kBuf];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave % C::MW, wn = wave / C::MW;
    const int l32 = lane & 31, g = lane >> 5, l16 = lane & 15;

    // tiles of one XCD run along j within a row of tiles: they share A's rows
    const int nt = nti * ntj;
    const int per = nt >> 3, rem = nt & 7, xcd = blockIdx.x & 7;
    const int tile = xcd * per + (xcd < rem ? xcd : rem) + (int)(blockIdx.x >> 3);
    const int ti = tile / ntj, tj = tile - ti * ntj;
    const int64_t i0 = (int64_t)ti * C::BM, j0 = (int64_t)tj * C::BN;
    const int rows = (int)(a.I - i0 < C::BM ? a.I - i0 : C::BM);
    const int cols = (int)(a.J - j0 < C::BN ? a.J - j0 : C::BN);
    const int nchunks = (int)((a.R + kR - 1) / kR);
    const int c0 = blockIdx.y * chunks_per_split;
    const int c1 = c0 + chunks_per_split < nchunks ? c0 + chunks_per_split : nchunks;
    const float maximum = a.factors.maxima[lane];

    const __amdgpu_buffer_rsrc_t ar = make_rsrc(a.a + i0 * a.lda, (uint32_t)((rows - 1) * a.lda + (int64_t)nchunks * 128));
    const int arow = tid >> 3, apiece = tid & 7;
    const int aoff = (int)(arow * a.lda) + apiece * 16, astep = (int)((C::NT / 8) * a.lda);
    const int brow = tid / TB, bcol = (tid % TB) * 16;
    const int boff = bcol < cols ? (int)(brow * a.ldb) + bcol : kLoadDead;
    const int bstep = bcol < cols ? (int)((C::NT / TB) * a.ldb) : 0;
    v4i va[PA], vb[PB];
    // Chunk c's source, past the split's end nothing: piece by piece, A's pieces first.
    auto a_offset = [&](int c) { return c < c1 ? aoff + c * 128 : kLoadDead; };
    auto b_rows = [&](int c) {
        const int64_t left = c < c1 ? a.R - (int64_t)c * kR : 0;
        const int br = (int)(left < kR ? left : kR);
        return make_rsrc(a.b + (c < c1 ? (int64_t)c * kR * a.ldb : 0) + j0, br > 0 ? (uint32_t)((br - 1) * a.ldb + cols) : 0u);
    };
    auto load_a = [&](int j, int off) { va[j] = __builtin_amdgcn_raw_buffer_load_b128(ar, off + j * astep, 0, 0); };
    auto load_b = [&](int j, __amdgpu_buffer_rsrc_t rb) {
        vb[j] = __builtin_amdgcn_raw_buffer_load_b128(rb, boff + j * bstep, 0, 0);
    };
    auto store_a = [&](int j, uint8_t* buf) {
        *reinterpret_cast<v4i*>(buf + (arow + j * (C::NT / 8)) * 128 + ((apiece ^ ((arow >> 1) & 7)) << 4)) = va[j];
    };
    auto store_b = [&](int j, uint8_t* buf) {
        *reinterpret_cast<v4i*>(buf + kA + (brow + j * (C::NT / TB)) * kLdB + bcol) = vb[j];
    };
    // the pieces that step s of a chunk stages
    auto for_pieces = [&](int s, auto fa, auto fb) {
#pragma unroll
        for (int j = 0; j < PA; ++j)
            if (j * 4 / PA == s) fa(j);
#pragma unroll
        for (int j = 0; j < PB; ++j)
            if (j * 4 / PB == s) fb(j);
    };

    v16f acc[C::MB][C::NB];
#pragma unroll
    for (int x = 0; x < C::MB; ++x)
#pragma unroll
        for (int y = 0; y < C::NB; ++y)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[x][y][v] = 0.0f;

    const int sw7 = (l32 >> 1) & 7;
    const uint8_t* const afrag = lds + (wm * C::MB * 32 + l32) * 128;
    // lane's source chunk of the transposing read: row 8 g + l16 / 2, columns 16 (group & 1) + 8 (l16 & 1)
    uint8_t* const bfrag =
        lds + kA + (8 * g + (l16 >> 1)) * kLdB + wn * C::NB * 32 + ((lane >> 4) & 1) * 16 + (l16 & 1) * 8;

    // step s of a chunk: 16 r of one piece of A with the fragments of B it needs
    struct Frags {
        v4u a[C::MB];
    };
    struct Codes {
        v4u bf[P == 2 ? C::NB : 1], h[C::NB];
    };
    auto read_a = [&](int cur, int p, int s, Frags& f) {
        const int piece = (P == 1 ? 0 : 4 * p) + 2 * s + g;
#pragma unroll
        for (int x = 0; x < C::MB; ++x)
            f.a[x] = *reinterpret_cast<const v4u*>(afrag + cur + x * 32 * 128 + ((piece ^ sw7) << 4));
    };
    auto read_b = [&](int cur, int s, v2i (&w)[C::NB]) {
#pragma unroll
        for (int y = 0; y < C::NB; ++y)
            w[y] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) v2i*)(bfrag + cur + s * 16 * kLdB + y * 32));
    };
    auto convert = [&](const v2i (&w)[C::NB], Codes& f) {
#pragma unroll
        for (int y = 0; y < C::NB; ++y) {
            uint32_t h0, h1, h2, h3;
            if constexpr (P == 2) {
                uint32_t b0, b1, b2, b3;
                codes4_both(w[y].x, b0, b1, h0, h1);
                codes4_both(w[y].y, b2, b3, h2, h3);
                f.bf[y] = (v4u){b0, b1, b2, b3};
            } else {
                codes4_fp16(w[y].x, h0, h1);
                codes4_fp16(w[y].y, h2, h3);
            }
            f.h[y] = (v4u){h0, h1, h2, h3};
        }
    };
    // first: the piece is the bf16 one
    auto multiply = [&](const Frags& f, const Codes& b, bool first) {
#pragma unroll
        for (int x = 0; x < C::MB; ++x)
#pragma unroll
            for (int y = 0; y < C::NB; ++y) {
                if (P == 2 && first)
                    acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(v8bf, f.a[x]), __builtin_bit_cast(v8bf, b.bf[P == 2 ? y : 0]), acc[x][y], 0, 0, 0);
                else
                    acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, f.a[x]),
                                                                       __builtin_bit_cast(v8h, b.h[y]), acc[x][y], 0, 0, 0);
            }
    };

#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int c = c0 + i;
        const int ao = a_offset(c);
        const __amdgpu_buffer_rsrc_t rb = b_rows(c);
#pragma unroll
        for (int s = 0; s < 4; ++s) {  // in the order of the loop's steps, so that its waits count right
            for_pieces(s, [&](int j) { load_a(j, ao); }, [&](int j) { load_b(j, rb); });
            __builtin_amdgcn_sched_barrier(0);
        }
        if (i < 2)
#pragma unroll
            for (int s = 0; s < 4; ++s) for_pieces(s, [&](int j) { store_a(j, lds + i * kBuf); }, [&](int j) { store_b(j, lds + i * kBuf); });
    }
    // Four steps of MB x NB products a chunk: (s, piece) in the order 00 01 10 11, or four s with one piece.
    // Between a step's products the next step's fragments are read and a quarter of the staging runs, one
    // instruction at a time (a wave issues in order: a burst would hold back the products behind it).
    // Three LDS buffers: one is computed from, the next is complete (its first fragments are read before the
    // barrier, so the products go on right behind it), the third is written from the registers.
    Frags f0, f1;
    v2i w0[C::NB], w1[C::NB];
    Codes fb, fn;
    lds_barrier();
    int cur = 0, nxt = kBuf, far = 2 * kBuf;
    auto at = [&](int buf, int i, Frags& f) {
        if constexpr (P == 1) read_a(buf, 0, i, f);
        else read_a(buf, i & 1, i >> 1, f);
    };
    at(0, 0, f0);
    read_b(0, 0, w0);
    if constexpr (P == 1) read_b(0, 1, w1);
    convert(w0, fb);
    for (int c = c0; c < c1; ++c) {
        const int ao = a_offset(c + 3);
        const __amdgpu_buffer_rsrc_t rb = b_rows(c + 3);
        auto stage = [&](int s) {
            for_pieces(
                s,
                [&](int j) {
                    store_a(j, lds + far);
                    load_a(j, ao);
                },
                [&](int j) {
                    store_b(j, lds + far);
                    load_b(j, rb);
                });
        };
        auto spread = [&]() {
#pragma unroll
            for (int i = 0; i < C::MB * C::NB; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
                __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // an LDS write
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // a load
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // conversions
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (P == 1) {
            at(cur, 1, f1);
            stage(0);
            multiply(f0, fb, false);
            convert(w1, fn);
            read_b(cur, 2, w0);
            spread();
            at(cur, 2, f0);
            stage(1);
            multiply(f1, fn, false);
            convert(w0, fb);
            read_b(cur, 3, w1);
            spread();
            at(cur, 3, f1);
            stage(2);
            multiply(f0, fb, false);
            convert(w1, fn);
            read_b(nxt, 0, w0);
            spread();
            at(nxt, 0, f0);
            stage(3);
            multiply(f1, fn, false);
            convert(w0, fb);
            read_b(nxt, 1, w1);
            spread();
        } else {
            at(cur, 1, f1);
            read_b(cur, 1, w1);
            stage(0);
            multiply(f0, fb, true);
            spread();
            at(cur, 2, f0);
            stage(1);
            multiply(f1, fb, false);
            convert(w1, fn);
            spread();
            at(cur, 3, f1);
            stage(2);
            multiply(f0, fn, true);
            read_b(nxt, 0, w0);
            spread();
            at(nxt, 0, f0);
            stage(3);
            multiply(f1, fn, false);
            convert(w0, fb);
            spread();
        }
        const int was = cur;
        cur = nxt;
        nxt = far;
        far = was;
        lds_barrier();
    }

    const int common = above_exponent(wave_max(maximum));
    const int down = -grad_exponent<P>(common, kNoRow);
    int* const row_down = reinterpret_cast<int*>(lds);
    if constexpr (kRows) {  // (the loop's last barrier freed the buffers)
        for (int r = tid; r < C::BM; r += C::NT)
            row_down[r] = r < rows ? -grad_exponent<P>(common, a.factors.rows[i0 + r]) : 0;
        lds_barrier();
    }
#pragma unroll
    for (int y = 0; y < C::NB; ++y) {
        const int col = wn * C::NB * 32 + y * 32 + l32;
        if (col >= cols) continue;
#pragma unroll
        for (int x = 0; x < C::MB; ++x)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int row = wm * C::MB * 32 + x * 32 + 8 * (v >> 2) + 4 * g + (v & 3);
                if (row >= rows) continue;
                const int64_t at = blockIdx.y * a.slab + (i0 + row) * a.ldc + j0 + col;
                const float value = __builtin_amdgcn_ldexpf(acc[x][y][v], kRows ? row_down[row] : down);
                if constexpr (kBf16) {
                    __bf16* p = static_cast<__bf16*>(a.c) + at;
                    *p = (__bf16)(kAdd ? (float)*p + value : value);
                } else {
                    float* p = static_cast<float*>(a.c) + at;
                    *p = kAdd ? *p + value : value;
                }
            }
    }
}

using Wide = GradTile<4, 2, 2, 4>;   // 256 x 256, 8 waves
using Short = GradTile<2, 2, 1, 4>;  // 64 x 256, 4 waves: few rows of A

template <class C, int P>
hipError_t launch_c(const GradGemmArgs& a, hipStream_t stream) {
    const int nti = (int)((a.I + C::BM - 1) / C::BM), ntj = (int)((a.J + C::BN - 1) / C::BN);
    constexpr int kR = 64 / P;
    const int64_t nchunks = (a.R + kR - 1) / kR;
    const int per = (int)((nchunks + a.splits - 1) / a.splits);
    const dim3 grid((unsigned)(nti * ntj), (unsigned)a.splits);
    auto run = [&](auto bf16, auto add, auto has_rows) {
        grad_gemm_kernel<C, P, bf16.value, add.value, has_rows.value><<<grid, C::NT, 0, stream>>>(a, nti, ntj, per);
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    if (a.factors.rows) {  // dx, in fp32 slabs
        if (a.bf16_out) return hipErrorInvalidValue;
        if (a.accumulate) run(no, yes, yes);
        else run(no, no, yes);
    } else if (a.bf16_out) {
        if (a.accumulate) run(yes, yes, no);
        else run(yes, no, no);
    } else {
        if (a.accumulate) run(no, yes, no);
        else run(no, no, no);
    }
    return hipGetLastError();
}

float grad_cost(bool wide, int64_t I, int64_t J, int64_t R, int P, int splits) {
    const int64_t bm = wide ? Wide::BM : Short::BM;
    const int64_t n = ((I + bm - 1) / bm) * ((J + Wide::BN - 1) / Wide::BN) * splits;
    float per_r;
    if (wide) per_r = (P == 2 ? 0.0434f : 0.0264f) * (float)((n + 255) / 256);
    else per_r = P == 2 ? 0.0160f + 0.0000448f * (float)(n > 256 ? n - 256 : 0) : 0.0104f + 0.0000397f * (float)(n > 256 ? n - 256 : 0);
    return 8.0f + per_r * (float)R / (float)splits;
}

}  // namespace

// Costs measured with J = 2048: wide tiles run one to a CU, 178 us (two pieces; one: 110) a round of 256 at
// R = 4096; short ones 65 us (43) up to 256 of them and 207 (165) for 1024.  So short ones take what wide
// ones would fill badly: I = 1128 101 against 179 us with the gradient tiles, I = 300 (R 50280) 195 against 221,
// I = 512 (R 50280) 276 against 234.
GradShape grad_shape(int64_t I, int64_t J, int64_t R, int pieces, int min_splits, int max_splits) {
    // (the last: as many short tiles as the CUs hold at once, 3 a CU with two pieces, 2 with one)
    const int64_t short_tiles = (I + Short::BM - 1) / Short::BM * ((J + Wide::BN - 1) / Wide::BN);
    const int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, (int)((pieces == 2 ? 768 : 512) / short_tiles)};
    GradShape best{0, min_splits, 3.0e38f};
    const int64_t ti = (I + Wide::BM - 1) / Wide::BM, tj = (J + Wide::BN - 1) / Wide::BN;
    for (int s : kSplits) {
        if (s < min_splits || s > max_splits || (s > min_splits && R / s < 256)) continue;
        const float slabs = max_splits > min_splits ? (float)(I * J) * (float)s * 4.0f / 4.0e6f : 0.0f;  // read once more
        auto consider = [&](int64_t rows, float cost) {
            if (cost + slabs < best.cost) best = GradShape{rows, s, cost + slabs};
        };
        consider(0, grad_cost(false, I, J, R, pieces, s));
        consider(I, grad_cost(true, I, J, R, pieces, s));
        // wide tiles for whole rounds, short ones for the rest (50280 rows: 6 rounds and 144 short tiles, not 7 rounds)
        const int64_t main = ti * tj * s / 256 * 256 / (tj * s) * Wide::BM;
        if (main > 0 && main < I)
            consider(main, grad_cost(true, main, J, R, pieces, s) + grad_cost(false, I - main, J, R, pieces, s));
    }
    return best;
}

hipError_t launch_grad_gemm(const GradGemmArgs& a, int pieces, hipStream_t stream) {
    GradGemmArgs part = a;
    if (a.wide_rows > 0) {
        part.I = a.wide_rows;
        if (hipError_t err = pieces == 1 ? launch_c<Wide, 1>(part, stream) : launch_c<Wide, 2>(part, stream)) return err;
    }
    if (a.wide_rows == a.I) return hipSuccess;
    part.I = a.I - a.wide_rows;
    part.a = a.a + a.wide_rows * a.lda;
    if (a.factors.rows) part.factors.rows = a.factors.rows + a.wide_rows;
    part.c = static_cast<uint8_t*>(a.c) + a.wide_rows * a.ldc * (a.bf16_out ? 2 : 4);
    return pieces == 1 ? launch_c<Short, 1>(part, stream) : launch_c<Short, 2>(part, stream);
}

}  // namespace dfssm
