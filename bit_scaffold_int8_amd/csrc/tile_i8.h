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
// cache line), and the 16-byte pieces of row r are stored at piece ^ (r & 7), so that the 8
// lanes that read together (8 rows, one piece) hit all banks.  Two LDS buffers, one barrier per
// chunk; loads run two chunks ahead (registers hold the chunk after the one in LDS).
#pragma once

#include "device_common.h"

namespace dfssm {

constexpr int kTileChunk = 128;               // k bytes per chunk
constexpr int kTileDead = 0x40000000;         // a load offset past every tile's resource: reads zero
constexpr int64_t kTileMaxLd = (int64_t)1 << 22;  // row stride limit: 256 rows stay below kTileDead

// WW x TW waves; each owns WB x TB blocks of 32 x 32.
template <int WB_, int TB_, int WW_, int TW_>
struct TileI8 {
    static constexpr int WB = WB_, TB = TB_, WW = WW_, TW = TW_;
    static constexpr int BW = 32 * WB * WW, BT = 32 * TB * TW;
    static constexpr int NT = kWave * WW * TW;
    static constexpr int PW = BW * 8 / NT, PT = BT * 8 / NT;  // 16-byte pieces per thread per chunk
    static constexpr int kBufBytes = (BW + BT) * kTileChunk;
    static constexpr int kLdsBytes = 2 * kBufBytes;
    static_assert(PW * NT == BW * 8 && PT * NT == BT * 8, "pieces split evenly over the threads");
    static_assert(NT % 64 == 0 && BW <= 256 && BT <= 256, "tile sizes");
};

// Pieces of one operand's chunk for one thread.  kFast: base and row stride are multiples of 16
// and so is K; a piece is then wholly inside or outside its row, and the buffer resource's range
// check zeroes rows past the last.  Otherwise 16-byte loads at any address, gathered by bytes
// where a piece crosses the row's end.
template <bool kFast, int P, int kRowStep>
struct Stager {
    __amdgpu_buffer_rsrc_t rsrc;
    const int8_t* base;
    int64_t ld;
    int row0, rows, piece, off0;
    uint4 v[P];

    __device__ __forceinline__ void init(const int8_t* p, int64_t ld_, int rows_, int K, int tid) {
        base = p;
        ld = ld_;
        rows = rows_;
        row0 = tid >> 3;
        piece = tid & 7;
        if constexpr (kFast) {
            rsrc = make_rsrc(p, rows_ > 0 ? (uint32_t)((rows_ - 1) * ld_ + K) : 0u);
            off0 = (int)(row0 * ld_);
        }
    }
    // Piece j of a chunk: off = offset(chunk) first.
    __device__ __forceinline__ int offset(int chunk, int K) const {
        const int k = chunk * kTileChunk + piece * 16;
        if constexpr (kFast) return off0 + (k < K ? k : kTileDead);
        return k;
    }
    __device__ __forceinline__ void load(int j, int off, int K) {
        if constexpr (kFast) {
            const v4i r = __builtin_amdgcn_raw_buffer_load_b128(rsrc, off + j * (int)(kRowStep * ld), 0, 0);
            v[j] = make_uint4((uint32_t)r.x, (uint32_t)r.y, (uint32_t)r.z, (uint32_t)r.w);
        } else {
            const int row = row0 + j * kRowStep;
            uint4 r = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows && off < K) {
                const uint8_t* src = reinterpret_cast<const uint8_t*>(base) + row * ld + off;
                if (off + 16 <= K) __builtin_memcpy(&r, src, 16);
                else r = load16_guarded<false>(src, 0, K - off);
            }
            v[j] = r;
        }
    }
    __device__ __forceinline__ void store(int j, uint8_t* lds) const {
        *reinterpret_cast<uint4*>(lds + (row0 + j * kRowStep) * kTileChunk + ((piece ^ ((row0 >> 1) & 7)) << 4)) = v[j];
    }
    // All pieces of a chunk.
    __device__ __forceinline__ void load_all(int chunk, int K) {
        const int off = offset(chunk, K);
#pragma unroll
        for (int j = 0; j < P; ++j) load(j, off, K);
    }
    __device__ __forceinline__ void store_all(uint8_t* lds) const {
#pragma unroll
        for (int j = 0; j < P; ++j) store(j, lds);
    }
};

// The tile's accumulators.  w, x: the tile's first rows; wrows, trows: rows of them that exist
// (the others read zero).  Every thread of the group calls it; LDS is free again after the
// caller's next barrier.
template <class C, bool kFast>
__device__ __forceinline__ void tile_i8(const int8_t* __restrict__ w, int64_t ldw, int wrows,
                                        const int8_t* __restrict__ x, int64_t ldx, int trows, int K,
                                        uint8_t* __restrict__ lds, v16i (&acc)[C::WB][C::TB]) {
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int ww = wave % C::WW, tw = wave / C::WW;
    const int l32 = lane & 31, g = lane >> 5;

    Stager<kFast, C::PW, C::NT / 8> sw;
    Stager<kFast, C::PT, C::NT / 8> st;
    sw.init(w, ldw, wrows, K, tid);
    st.init(x, ldx, trows, K, tid);
#pragma unroll
    for (int a = 0; a < C::WB; ++a)
#pragma unroll
        for (int b = 0; b < C::TB; ++b) acc[a][b] = (v16i){0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};

    const int nch = (K + kTileChunk - 1) / kTileChunk;
    constexpr int kXOff = C::BW * kTileChunk;
    const uint8_t* const wfrag = lds + (ww * C::WB * 32 + l32) * kTileChunk;
    const uint8_t* const xfrag = lds + kXOff + (tw * C::TB * 32 + l32) * kTileChunk;
    const int sw7 = (l32 >> 1) & 7;

    sw.load_all(0, K);
    st.load_all(0, K);
    sw.store_all(lds);
    st.store_all(lds + kXOff);
    // in the order of the loop's steps: the waits for them then count only what lies between
    const int ow1 = sw.offset(1, K), ot1 = st.offset(1, K);
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
    auto step = [&](int s, int cur, int nxt, int ow, int ot, const Frags& f, Frags* next) {
        if (next) read(cur, s + 1, *next);
#pragma unroll
        for (int j = 0; j < C::PW; ++j)
            if (j * 4 / C::PW == s) {
                sw.store(j, lds + nxt);
                sw.load(j, ow, K);
            }
#pragma unroll
        for (int j = 0; j < C::PT; ++j)
            if (j * 4 / C::PT == s) {
                st.store(j, lds + nxt + kXOff);
                st.load(j, ot, K);
            }
        multiply(f);
        if constexpr (kFast) {
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
    for (int c = 0; c < nch; ++c) {
        lds_barrier();
        const int cur = (c & 1) * C::kBufBytes, nxt = C::kBufBytes - cur;
        // (past the last chunk zeros are staged that nothing reads)
        const int ow = sw.offset(c + 2, K), ot = st.offset(c + 2, K);
        read(cur, 0, f0);
        __builtin_amdgcn_sched_barrier(0);
        step(0, cur, nxt, ow, ot, f0, &f1);
        step(1, cur, nxt, ow, ot, f1, &f0);
        step(2, cur, nxt, ow, ot, f0, &f1);
        step(3, cur, nxt, ow, ot, f1, nullptr);
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
