// tile_i8.h -- one output tile of an int8 x int8 product (gfx950), shared by the int8
// product and the cross entropy over the vocabulary.  Private to the library.
//
//   acc[w][t] = sum_k W[w][k] X[t][k]      (exact int32)
//
// for BW rows of W (weights, vocabulary) and BT rows of X (tokens).  W is the A operand of
// v_mfma_i32_32x32x32_i8 and X the B operand, so a lane ends with one token (column
// lane & 31) and 16 weight rows of each 32 x 32 block: 8 (v / 4) + 4 (lane / 32) + v % 4 for
// register v.  A softmax over the weights' axis then reduces inside a lane's registers, and four
// consecutive registers are four consecutive outputs of a token.
//
// Both operands go through LDS in chunks of 128 k: 8 threads stage a row's 128 bytes (a whole
// cache line).  LDS has 64 banks, so two rows of a chunk span them once; the 16-byte pieces of row r are
// stored at piece ^ (r / 2 & 7), so that the 16 lanes that read together (16 rows, one piece) meet
// different banks (with r & 7 a third of the LDS cycles were conflicts).  Two LDS buffers, one barrier per chunk;
// loads run two chunks ahead (registers hold the chunk after the one in LDS).  Chunks of 64 k,
// with three buffers or with two smaller tiles per CU, measured 8 % slower: half-line loads.
//
// What bounds it: 2048 tokens x 50280 rows x 2048 ran 239 us as logits' statistics in 7 rounds of 256 x 256 tiles (1.8
// POPS; 218 us since the last round's rest goes to small tiles); without staging 207, so most of it is the products
// under the power limit (the GPU clocks down to 2.0 GHz at 45 % matrix-core occupancy) and each tile's epilogue (about
// 5 of 33 us), which nothing overlaps.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace dfssm {

constexpr int kTileChunk = 128;               // k bytes per chunk
constexpr int kTileDead = 0x40000000;         // a load offset past every tile's resource (row strides end at 2^22): reads zero

// WW x TW waves, each with WB x TB blocks of 32 x 32; KS such groups of waves take every KS-th chunk of K each and
// add up their sums through LDS (small tiles: they are used where there are few, and K's length is the time).
template <int WB_, int TB_, int WW_, int TW_, int KS_ = 1>
struct TileI8 {
    static constexpr int WB = WB_, TB = TB_, WW = WW_, TW = TW_, KS = KS_;
    static constexpr int BW = 32 * WB * WW, BT = 32 * TB * TW;
    static constexpr int NG = kWave * WW * TW, NT = NG * KS;  // threads of a K group, of the workgroup
    static constexpr int PW = BW * 8 / NG, PT = BT * 8 / NG;  // 16-byte pieces per thread per chunk
    static constexpr int kBufBytes = (BW + BT) * kTileChunk;
    static constexpr int kLdsBytes = 2 * kBufBytes * KS;
    static constexpr int kMinWaves = NT >= 256 ? NT / 256 : 1;  // per SIMD, for one workgroup on a CU
    static_assert(PW * NG == BW * 8 && PT * NG == BT * 8, "pieces split evenly over the threads");
    static_assert(NT <= 512 && BW <= 256 && BT <= 256, "tile sizes");
    static_assert((KS - 1) * WB * TB * 16 * NG * 4 <= kLdsBytes, "the K groups' sums fit the buffers");
};

// A 16-byte value shifted down by s bytes (zeros from 16 on).
__device__ __forceinline__ uint4 shift_bytes(uint4 v, int s) {
    uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
    if (s >= 8) {
        lo = s < 16 ? hi : 0;
        hi = 0;
        s -= 8;
    }
    const int bits = 8 * (s & 7);
    lo = lo >> bits | (hi << 1) << (63 - bits);
    hi >>= bits;
    return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
}

// Pieces of one operand's chunk for one thread.  kFast: base and row stride are multiples of 16
// and so is K; a piece is then wholly inside or outside its row, and the buffer resource's range
// check zeroes rows past the last.  Otherwise 16-byte loads at any address that never leave the row: a piece
// that would is loaded from the row's last 16 bytes and shifted on its way to LDS (rows of less than
// 16 bytes are gathered by bytes); rows past the last repeat it, and their outputs are not used.
template <bool kFast, int P, int kRowStep>
struct Stager {
    static_assert(kRowStep % 2 == 0, "the rows of a thread's pieces differ by whole pairs");
    __amdgpu_buffer_rsrc_t rsrc;
    const int8_t* base;
    int64_t ld;
    int row0, piece, off0;
    int row_off[P];
    uint4 v[P];

    __device__ __forceinline__ void init(const int8_t* p, int64_t ld_, int rows, int K, int tid) {
        base = p;
        ld = ld_;
        row0 = tid >> 3;
        piece = tid & 7;
        if constexpr (kFast) {
            rsrc = make_rsrc(p, rows > 0 ? (uint32_t)((rows - 1) * ld_ + K) : 0u);
            off0 = (int)(row0 * ld_);
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) row_off[j] = (int)(min(row0 + j * kRowStep, rows - 1) * ld_);
        }
    }
    // Piece j of a chunk: off = offset(chunk) first.  kInner: rows of 16 bytes or more, and for store a piece that
    // its row holds.
    __device__ __forceinline__ int offset(int chunk, int K) const {
        const int k = chunk * kTileChunk + piece * 16;
        if constexpr (kFast) return off0 + (k < K ? k : kTileDead);
        return k;
    }
    template <bool kInner = false>
    __device__ __forceinline__ void load(int j, int off, int K) {
        if constexpr (kFast) {
            const v4i r = __builtin_amdgcn_raw_buffer_load_b128(rsrc, off + j * (int)(kRowStep * ld), 0, 0);
            v[j] = make_uint4((uint32_t)r.x, (uint32_t)r.y, (uint32_t)r.z, (uint32_t)r.w);
        } else if (kInner || K >= 16) {
            __builtin_memcpy(&v[j], base + (uint32_t)(row_off[j] + min(off, K - 16)), 16);
        } else {
            v[j] = load16_guarded<false>(reinterpret_cast<const uint8_t*>(base) + row_off[j], off, K);
        }
    }
    // off: the offset that piece j was loaded with.
    template <bool kInner = false>
    __device__ __forceinline__ void store(int j, uint8_t* lds, int off, int K) const {
        uint4 r = v[j];
        if constexpr (!kFast && !kInner) {
            // only a row's last chunk (and what follows it) holds pieces that leave the row
            if (off - piece * 16 + kTileChunk > K && K >= 16) r = shift_bytes(r, max(off - (K - 16), 0));
        }
        *reinterpret_cast<uint4*>(lds + (row0 + j * kRowStep) * kTileChunk +
                                  ((piece ^ (((row0 >> 1) + j * kRowStep / 2 % 8) & 7)) << 4)) = r;
    }
    // All pieces of a chunk.
    __device__ __forceinline__ void load_all(int chunk, int K) {
        const int off = offset(chunk, K);
#pragma unroll
        for (int j = 0; j < P; ++j) load(j, off, K);
    }
    __device__ __forceinline__ void store_all(int chunk, uint8_t* lds, int K) const {
        const int off = offset(chunk, K);
#pragma unroll
        for (int j = 0; j < P; ++j) store(j, lds, off, K);
    }
};

// The tile's accumulators.  w, x: the tile's first rows; wrows, trows: rows of them that exist
// (the others read zero).  Every thread of the group calls it; LDS is free again after the
// caller's next barrier.  Returns whether this wave holds the sums (the first K group's do).
template <class C, bool kFast>
__device__ __forceinline__ bool tile_i8(const int8_t* __restrict__ w, int64_t ldw, int wrows,
                                        const int8_t* __restrict__ x, int64_t ldx, int trows, int K,
                                        uint8_t* __restrict__ lds, v16i (&acc)[C::WB][C::TB]) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave_wg = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int kg = wave_wg / (C::WW * C::TW), wave = wave_wg % (C::WW * C::TW);
    const int tid = wave * kWave + lane;  // thread within the K group
    const int ww = wave % C::WW, tw = wave / C::WW;
    const int l32 = lane & 31, g = lane >> 5;
    uint8_t* const all_lds = lds;
    lds += kg * 2 * C::kBufBytes;

    Stager<kFast, C::PW, C::NG / 8> sw;
    Stager<kFast, C::PT, C::NG / 8> st;
    sw.init(w, ldw, wrows, K, tid);
    st.init(x, ldx, trows, K, tid);
#pragma unroll
    for (int a = 0; a < C::WB; ++a)
#pragma unroll
        for (int b = 0; b < C::TB; ++b) acc[a][b] = (v16i){0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};

    // chunk i of this K group is chunk i KS + kg of K; every group takes the same number (past K: zeros)
    const int nch = ((K + kTileChunk - 1) / kTileChunk + C::KS - 1) / C::KS;
    constexpr int kXOff = C::BW * kTileChunk;
    const uint8_t* const wfrag = lds + (ww * C::WB * 32 + l32) * kTileChunk;
    const uint8_t* const xfrag = lds + kXOff + (tw * C::TB * 32 + l32) * kTileChunk;
    const int sw7 = (l32 >> 1) & 7;

    sw.load_all(kg, K);
    st.load_all(kg, K);
    sw.store_all(kg, lds, K);
    st.store_all(kg, lds + kXOff, K);
    // in the order of the loop's steps: the waits for them then count only what lies between
    const int ow1 = sw.offset(C::KS + kg, K), ot1 = st.offset(C::KS + kg, K);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int j = 0; j < C::PW; ++j)
            if (j * 4 / C::PW == s) sw.load(j, ow1, K);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < C::PT; ++j)
            if (j * 4 / C::PT == s) st.load(j, ot1, K);
        __builtin_amdgcn_sched_barrier(0);
    }
    struct Frags {
        v4i w[C::WB], x[C::TB];
    };
    auto read = [&](int cur, int s, Frags& f) {
        const int off = cur + (((2 * s + g) ^ sw7) << 4);
#pragma unroll
        for (int a = 0; a < C::WB; ++a) f.w[a] = *reinterpret_cast<const v4i*>(wfrag + off + a * 32 * kTileChunk);
#pragma unroll
        for (int b = 0; b < C::TB; ++b) f.x[b] = *reinterpret_cast<const v4i*>(xfrag + off + b * 32 * kTileChunk);
    };
    auto multiply = [&](const Frags& f) {
#pragma unroll
        for (int a = 0; a < C::WB; ++a)
#pragma unroll
            for (int b = 0; b < C::TB; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[a], f.x[b], acc[a][b], 0, 0, 0);
    };
    // One of a chunk's four steps: the products of `f`, and between them the reads of the next step's
    // fragments and a quarter of the staging (registers to the other buffer, then the loads that refill
    // them).  A wave issues in order, so a burst of LDS or memory instructions would hold back the
    // products behind it; the pattern spreads them one by one over the products.
    auto step = [&](auto inner, int s, int cur, int nxt, int ow, int ot, int held, const Frags& f, Frags* next) {
        constexpr bool kInner = decltype(inner)::value;
        if (next) read(cur, s + 1, *next);
#pragma unroll
        for (int j = 0; j < C::PW; ++j)
            if (j * 4 / C::PW == s) {
                sw.template store<kInner>(j, lds + nxt, held, K);
                sw.template load<kInner>(j, ow, K);
            }
#pragma unroll
        for (int j = 0; j < C::PT; ++j)
            if (j * 4 / C::PT == s) {
                st.template store<kInner>(j, lds + nxt + kXOff, held, K);
                st.template load<kInner>(j, ot, K);
            }
        multiply(f);
        if constexpr (kInner) {
#pragma unroll
            for (int i = 0; i < C::WB * C::TB; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
                __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // an LDS write
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // a load
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    Frags f0, f1;
    auto chunk = [&](auto inner, int c) {
        lds_barrier();
        const int cur = (c & 1) * C::kBufBytes, nxt = C::kBufBytes - cur;
        // (past the last chunk zeros are staged that nothing reads)
        const int ow = sw.offset((c + 2) * C::KS + kg, K), ot = st.offset((c + 2) * C::KS + kg, K);
        // (the offset of the chunk that the registers hold; used where rows are not aligned, and there it is the same for both)
        const int held = st.offset((c + 1) * C::KS + kg, K);
        read(cur, 0, f0);
        __builtin_amdgcn_sched_barrier(0);
        step(inner, 0, cur, nxt, ow, ot, held, f0, &f1);
        step(inner, 1, cur, nxt, ow, ot, held, f1, &f0);
        step(inner, 2, cur, nxt, ow, ot, held, f0, &f1);
        step(inner, 3, cur, nxt, ow, ot, held, f1, nullptr);
    };
    int c = 0;
    if constexpr (kFast) {
        for (; c < nch; ++c) chunk(std::true_type{}, c);
    } else {
        // without the shifts' branches while the chunk that the registers hold is inside the rows
        // (300 rows x 4000 tokens x 8001: 43 us, 54 with them in every chunk)
        for (const int inside = K / kTileChunk / C::KS - 1; c < inside; ++c) chunk(std::true_type{}, c);
        for (; c < nch; ++c) chunk(std::false_type{}, c);
    }
    if constexpr (C::KS > 1) {
        int32_t* const sums = reinterpret_cast<int32_t*>(all_lds) + tid;
        lds_barrier();
#pragma unroll
        for (int a = 0; a < C::WB; ++a)
#pragma unroll
            for (int b = 0; b < C::TB; ++b)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    if (kg) sums[(((kg - 1) * C::WB * C::TB + a * C::TB + b) * 16 + v) * C::NG] = acc[a][b][v];
        lds_barrier();
#pragma unroll
        for (int q = 0; q < C::KS - 1; ++q)
#pragma unroll
            for (int a = 0; a < C::WB; ++a)
#pragma unroll
                for (int b = 0; b < C::TB; ++b)
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (!kg) acc[a][b][v] += sums[((q * C::WB * C::TB + a * C::TB + b) * 16 + v) * C::NG];
    }
    return kg == 0;
}

// ---- which tile a shape takes (host)

enum TileKind { kTile256, kTile256x192, kTile128, kTile128x64, kTile64x64, kTile128x32, kTile64x32, kTile32x32, kTileKinds };
constexpr int kTileKinds64 = kTile64x64 + 1;  // the first ones: 64 tokens or more
constexpr int kTileKinds128 = kTile128x64 + 1;  // 128 rows or more

struct TileShape {
    int rows, tokens;
    float fixed;        // us that do not grow with K
    float first, more;  // us for up to 256 tiles, and for each further 256, at K = 2048
};
// Measured on 512 to 50280 rows x 1 to 2048 tokens, K 512 to 8192, large ones in long runs under the power limit.
// Large tiles reread least and win when they fill the GPU (50280 rows x 1500 tokens, K 2048, in this order:
// 183, 199, 207, 235 us; x 300 tokens, of which the second wastes least: 59, 53, 60, 62); small ones win when they do
// not (2048 rows x 1 token, K 4096: 39 us for the first, then 17, 12, 9.5, 11, 7.2, 6.1 from the third on), or when
// the large ones' last round would be nearly empty (8512 rows x 300 tokens: 26, 22, 13, 13 us).
inline const TileShape& tile_shape(int kind) {
    static const TileShape t[kTileKinds] = {
        {256, 256, 7.0f, 24.0f, 34.0f}, {256, 192, 6.5f, 21.0f, 30.0f}, {128, 128, 4.1f, 10.7f, 11.5f},
        {128, 64, 3.3f, 7.9f, 7.8f},    {64, 64, 3.4f, 6.3f, 3.4f},     {128, 32, 2.9f, 6.8f, 4.0f},
        {64, 32, 3.6f, 5.4f, 2.35f},    {32, 32, 3.95f, 5.0f, 4.0f}};
    return t[kind];
}

inline float tile_cost(int kind, int64_t rows, int64_t tokens, int64_t K) {
    const TileShape& t = tile_shape(kind);
    const int64_t n = ((rows + t.rows - 1) / t.rows) * ((tokens + t.tokens - 1) / t.tokens);
    return t.fixed + (t.first - t.fixed + (float)((n - 1) / 256) * t.more) * ((float)K / 2048.0f);
}

// The cheapest of the tiles [from, to).
inline int pick_tile(int64_t rows, int64_t tokens, int64_t K, int from = 0, int to = kTileKinds) {
    int best = from;
    for (int k = from + 1; k < to; ++k)
        if (tile_cost(k, rows, tokens, K) < tile_cost(best, rows, tokens, K)) best = k;
    return best;
}

// Rows [0, main) by one tile, the rest by another (main == rows: no rest).
struct TileSplit {
    int64_t main;
    int kind, tail;
    float cost;
};

// The cheapest of the tiles [from, to) for all rows, or the largest tile for as many rows as fill whole rounds of
// the 256 CUs and another for the rest, in a launch of its own (50280 rows: 1024 tokens 3 rounds and
// 144 small tiles instead of 4 rounds, 130 -> 113 us; 2048 tokens 231 -> 213 us).
inline TileSplit split_rows(int64_t rows, int64_t tokens, int64_t K, int from = 0, int to = kTileKinds) {
    const int one = pick_tile(rows, tokens, K, from, to);
    TileSplit best{rows, one, one, tile_cost(one, rows, tokens, K)};
    const TileShape& big = tile_shape(kTile256);
    const int64_t ntt = (tokens + big.tokens - 1) / big.tokens, ntw = (rows + big.rows - 1) / big.rows;
    const int64_t main = ntw * ntt / 256 * 256 / ntt * big.rows;
    if (from <= kTile256 && main > 0 && main < rows) {
        const int tail = pick_tile(rows - main, tokens, K, from, to);
        const float cost = tile_cost(kTile256, main, tokens, K) + tile_cost(tail, rows - main, tokens, K);
        if (cost < best.cost) best = TileSplit{main, kTile256, tail, cost};
    }
    return best;
}

// f(Tile{}) for the tile of a kind.
template <class F>
auto with_tile(int kind, F f) {
    switch (kind) {
        case kTile256: return f(TileI8<2, 4, 4, 2>{});
        case kTile256x192: return f(TileI8<2, 3, 4, 2>{});
        case kTile128: return f(TileI8<2, 2, 2, 2>{});
        case kTile128x64: return f(TileI8<1, 2, 4, 1>{});
        case kTile128x32: return f(TileI8<1, 1, 4, 1>{});
        case kTile64x64: return f(TileI8<1, 1, 2, 2, 2>{});
        case kTile64x32: return f(TileI8<1, 1, 2, 1, 4>{});
        default: return f(TileI8<1, 1, 1, 1, 8>{});
    }
}

// Tile index of a workgroup.  Workgroups go to the 8 XCDs in turn; each XCD gets a contiguous
// run of tiles, so tiles that share operands share an L2.  Tiles run token tile by token
// tile within groups of 8 token tiles: a group's tokens stay in L2 while the weights stream.
struct TilePos {
    int w, t;
};
__device__ __forceinline__ TilePos tile_pos(int bid, int ntw, int ntt) {
    const int nt = ntw * ntt;
    const int per = nt >> 3, rem = nt & 7;
    const int xcd = bid & 7;
    const int tile = xcd * per + (xcd < rem ? xcd : rem) + (bid >> 3);
    const int group = tile / (ntw * 8);
    const int in = tile - group * ntw * 8;
    const int gt = ntt - group * 8 < 8 ? ntt - group * 8 : 8;
    TilePos p;
    p.w = in / gt;
    p.t = group * 8 + in % gt;
    return p;
}

}  // namespace dfssm
