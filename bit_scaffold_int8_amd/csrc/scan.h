// scan.h -- what the Mamba-2 scan and its gradients share (gfx950), private to the library: how sequences are cut
// into chunks and segments, the layouts of the workspace, and matrix products of fp32 values on the bf16 matrix cores.
//
// Products: the 16x16x32 bf16 instruction takes, from lane (r = lane % 16, q = lane / 16), eight values of row
// (or column) r.  Which of the 32 summed places they are is free as long as both operands agree; here
//   place(q, j) = 4 q + j % 4 + 16 (j / 4)
// Its result holds column r, rows 4 q + v: so two results stacked by rows are an operand of the next product as
// they stand, and an operand's values lie in two groups of four neighbours.
//
// An fp32 value enters as bf16 pieces x = p0 + p1 + p2 (each the rounding of what is left; after three the rest is below
// 2^-24 of x), and a product of two such takes the six products of pieces down to 2^-16: what it leaves out is of
// the size of fp32's own rounding.  A bf16 value is its own only piece.  Against the fp32 matrix
// instructions (1/16 of the rate) that is 2.7 times the rate for fp32 data and 5.3 times or more for bf16 data.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sequences.h"

namespace dfssm {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kChunk = 64;     // tokens of a chunk
constexpr int kP = 64;         // channels of a head
constexpr int kHeadArrays = 7; // per chunk and head, 64 values each:
enum { kCsHi, kCsLo, kStep, kWeight, kDecay, kEnter, kLeave };
//   cs = log2 of the decay from the chunk's start through token t, as hi + lo (summed in fp64: differences of
//   close ones keep fp32's precision however far the sum has come);  step = dt;  weight = dt 2^(cs_end - cs);  decay = 2^cs;
//   enter = the decay from the start of the token's tile of 16 through it;  leave = dt times the decay behind it to its tile's end.
// The decay between tokens of different tiles is the product of a leave, the tiles in between (their last enter) and an
// enter: all of them at most 1, so that none can overflow, and one product where a difference and an exponential would be.

struct ScanArgs {
    Sequences seq;
    int H, G;
    const void *x, *B, *C;
    const float* dt;
    int64_t ldx, lddt, ldb, ldc;
    const float *A_log, *D, *dt_bias;
    // workspace
    int4* chunks;     // [chunk]: first row, rows, sequence (-1: no such chunk), -
    int4* segments;   // [segment]: first chunk, chunks, sequence (-1: none), number within the sequence
    int* first_segment;  // [S + 1]
    int nchunks, nsegments, per_segment;  // bounds of the numbers, chunks of a segment
    uint8_t* groups;  // [chunk][G] blocks of group_bytes
    float* heads;     // [chunk][H][kHeadArrays][kChunk]
};

// A table's entry in scalar registers (it is the same for the whole wave, which the compiler cannot see of a load: buffers made from
// it would be loops over the lanes).
__device__ __forceinline__ int4 uniform(int4 v) {
    return make_int4(__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y),
                     __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w));
}

__device__ __forceinline__ int4 chunk_of(const ScanArgs& a, int c) {
    if (a.chunks) return uniform(a.chunks[c]);
    const int per = (a.seq.L + kChunk - 1) / kChunk, s = c / per, i = c - s * per;
    const int left = a.seq.L - i * kChunk;
    return uniform(make_int4(s * a.seq.L + i * kChunk, left < kChunk ? left : kChunk, s, 0));
}

// 2^(hi + lo), or 0 (without a branch: the exponential of a difference that is far below its range).
__device__ __forceinline__ float decay_between(float hi, float lo, bool on) {
    return __builtin_amdgcn_exp2f(on ? hi + lo : -1e30f);
}

// A group's block for one chunk: products C_t . B_s (fp32, results of 16 x 16), then three sets of pieces, each
// [piece][16-row tile][32-place step][lane][8]:
//   rows   rows of C (forward) or of B (backward) along the state
//   across  B, across the tokens (rows of it: state places)
//   cross   C, across the tokens (backward)
template <int kN, int kPieces>
struct GroupBlock {
    static constexpr int kG = kChunk * kChunk * 4, kPlane = kChunk * kN * 2, kSet = kPieces * kPlane;
    static constexpr int kRows = kG, kAcross = kRows + kSet, kCross = kAcross + kSet;
    static constexpr int forward = kCross, backward = kCross + kSet;
};

template <int kPieces>
struct Pieces {
    v8bf p[kPieces];
};

// (Two values at a time by their bits: written element by element, each piece is converted once to be kept and once more
// to be taken off.)
template <int kPieces>
__device__ __forceinline__ Pieces<kPieces> split(const float (&x)[8]) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    typedef float v2f __attribute__((ext_vector_type(2)));
    Pieces<kPieces> out;
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        v4u bits;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bits[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{r[2 * j], r[2 * j + 1]}), v2bf));
            if (i + 1 < kPieces) {
                r[2 * j] -= __uint_as_float(bits[j] << 16);
                r[2 * j + 1] -= __uint_as_float(bits[j] & 0xFFFF0000u);
            }
        }
        out.p[i] = __builtin_bit_cast(v8bf, bits);
    }
    return out;
}

// acc += a b: the products of pieces whose numbers add up to at most 2, the small ones first.
template <int kA, int kB>
__device__ __forceinline__ v4f mma(const Pieces<kA>& a, const Pieces<kB>& b, v4f acc) {
#pragma unroll
    for (int sum = 2; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < kA; ++i)
            if (sum - i >= 0 && sum - i < kB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[sum - i], acc, 0, 0, 0);
    return acc;
}

constexpr int products_of(int a, int b) {
    int n = 0;
    for (int i = 0; i < a; ++i)
        for (int j = 0; j < b; ++j) n += i + j <= 2 ? 1 : 0;
    return n;
}

// The order of a stretch of steps that each read fragments from LDS and multiply them: the reads of the next kAhead
// steps go out before a step's products.  Left alone, the compiler reads a step's fragments right before its products (a sweep for
// the states of 16384 tokens bf16 175 us, with this order 164; one for y gains nothing).
// kLoads loads from memory go out with the first steps, one each: all at once they hold up what comes behind them (139).
template <int kReads, int kProducts, int kCount, int kAhead, int kLoads>
__device__ __forceinline__ void read_ahead() {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);   // LDS reads
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, kProducts, 0);                             // matrix instructions
        if (i < kLoads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);                     // loads
        if (i + kAhead < kCount) __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// The sum of two products of which the second was formed with one operand negated.  The matrix instructions round their sums
// down, not to nearest: an error of the same sign everywhere, which sums over many tokens keep (dA_log of 2048 tokens
// against 64 bits: 6e-7, where single tokens' gradients have 2e-7).  Of two sums of opposite sign it cancels.
__device__ __forceinline__ v4f opposite(const v4f (&half)[2]) { return half[0] - half[1]; }

// Pieces stored [piece][...][lane][8]; `plane` bytes from piece to piece.
template <int kPieces>
__device__ __forceinline__ Pieces<kPieces> load_pieces(const uint8_t* at, int plane) {
    Pieces<kPieces> out;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) out.p[i] = *reinterpret_cast<const v8bf*>(at + i * plane);
    return out;
}
template <int kPieces>
__device__ __forceinline__ void store_pieces(uint8_t* at, int plane, const Pieces<kPieces>& v) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) *reinterpret_cast<v8bf*>(at + i * plane) = v.p[i];
}

__device__ __forceinline__ int place(int q, int j) { return 4 * q + (j & 3) + 16 * (j >> 2); }

// softplus with the identity above 20, as the decode step has it
__device__ __forceinline__ float scan_softplus(float v) { return v > 20.0f ? v : log1pf(expf(v)); }

// How sequences are cut: bounds of the tables, and a sweep's workgroups.
struct ScanPlan {
    int nchunks, nsegments, per_segment;
    int waves;        // of a sweep's workgroup: two for each head
    bool segmented;   // some sequence may have more than one segment
};

hipError_t launch_scan_prepare(const ScanArgs& a, bool bf16, int N, bool backward, hipStream_t stream);

// One sweep over the chunks of every segment with the state in registers:
//   state <- 2^cs_end state + sum_t weight_t v_t k_t^T
// kLocal keeps what a segment adds to a state of zero, and its decay; kStarts stores the state at the start of each
// chunk; kOutput computes y.  Backwards (reverse) v is dy, k is C, and the weight is the decay from the chunk's start.
enum SweepMode { kLocal, kStarts, kOutput };
struct SweepArgs {
    ScanArgs a;
    const void* v;       // x, or dy
    int64_t ldv;
    int key;             // offset of the key's set in a group's block
    int group_bytes;
    bool reverse;
    const float* start;  // [S][H][64][N]: the caller's states, or NULL: zeros
    float* end;          // the same, or NULL
    float* segment_states;  // [segment][H][64][N] in the registers' order, when the sequences are segmented; or NULL
    float* segment_decay;   // [segment][H]
    float* starts;       // [chunk][H][64][N]   (kStarts)
    void* y;             // (kOutput)
    int64_t ldy;
};
hipError_t launch_sweep(const SweepArgs& s, const ScanPlan& plan, bool bf16, int N, SweepMode mode, hipStream_t stream);

// f for the type of the data and d_state (64 or 128), as constants.
template <class F>
hipError_t with_kind(bool bf16, int N, F f) {
    if (N == 128) return bf16 ? f(std::true_type(), std::integral_constant<int, 128>()) : f(std::false_type(), std::integral_constant<int, 128>());
    return bf16 ? f(std::true_type(), std::integral_constant<int, 64>()) : f(std::false_type(), std::integral_constant<int, 64>());
}

// The host's side of the forward pass that the backward pass shares (mamba2_scan.hip).
ScanPlan scan_plan(const Sequences& seq, int H, int G);
int scan_group_bytes(bool bf16, int N, bool backward);
size_t scan_workspace(ScanArgs& a, SweepArgs& s, uint8_t* ws, int64_t T, int64_t S, int64_t H, int64_t G, int N, int group_bytes);

}  // namespace dfssm
