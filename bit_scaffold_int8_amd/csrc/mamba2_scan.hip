// mamba2_scan.hip -- the Mamba-2 scan over packed sequences (gfx950): a linear attention whose state decays by
// a factor for each head and token.
//
//   h_t = e^{a_t} h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t,   a_t = -dt_t exp(A_log)
//
// Two forms.  Short sequences (single tokens above all) go token by token through the recurrence, like the decode step: the
// states, 32 KB a head, are read and written once and everything else is small.  Longer ones go in chunks of 64 tokens, in
// which the recurrence is a product of matrices (cs: the decays' running sum within the chunk):
//
//   y_t = sum_{s <= t} e^{cs_t - cs_s} (C_t . B_s) dt_s x_s  +  e^{cs_t} h_start C_t  +  D x_t
//   h_end = e^{cs_end} h_start + sum_s e^{cs_end - cs_s} dt_s x_s B_s^T
//
//  * prepare: for each chunk, what its heads share: the products C . B of a group, B and C as bf16 pieces in the order in
//    which the matrix instructions take them (scan.h), and the decays of each head.
//  * sweep: a wave owns 32 channels of a head and walks over the chunks of a segment with their state, 32 x N fp32
//    values, in registers as the matrix instructions' accumulators.  These are at the same time operands of h C: the state
//    goes through no memory between chunks.  The heads of a workgroup (four or two) share the pieces of B and C in LDS.
//  * One sequence has too few heads to fill the GPU, so it is cut into segments of several chunks: a first sweep
//    finds what each segment adds to the state, a small kernel joins them in order, the second sweep starts from the joined ones.
//
// Measured, 64 heads of 64 channels, d_state 128, in us, means of 12 launches (prepare, first sweep, join, second sweep):
//   2048 tokens fp32   9.2, 22, 11.5, 42;   16384 tokens bf16   19, 68, 12, 155 (at best 138)
//   five packed sequences of 0 to 2500 tokens, 4101 in all, bf16   8.7 (and 5.1 for the tables), 25, 13, 53
// The sweeps are bound by the issue of their instructions.  For y of bf16 data a wave issues 184 matrix instructions a chunk (16
// cycles of a SIMD each) and 1040 vector ones (to split the state and the chunk's weights into pieces, above all): 34 and 48 % of
// the SIMDs' busy cycles (counters), and with two waves to a SIMD the two kinds hardly overlap.  fp32 data take 3 pieces, 456 and 1500
// instructions (38 and 31 %), and there the segments' states, 64 KB a head and segment written and read, cost as much as the
// chunks.  The sweeps that store the states of every chunk are bound by that: 8 x 2048 tokens bf16 160 us, 4.2 TB/s (145 at best).
// (At 16384 tokens the whole is 285 MB and 225 us: a quarter of the memory's rate.)
#include <math.h>

#include "scan.h"

namespace dfssm {

namespace {

constexpr double kLog2eD = 1.4426950408889634074;

// w: 1 the sequence's first segment, 2 its last
__device__ __forceinline__ int4 segment_of(const ScanArgs& a, int g) {
    if (a.segments) return uniform(a.segments[g]);
    const int chunks = (a.seq.L + kChunk - 1) / kChunk, per = (chunks + a.per_segment - 1) / a.per_segment;
    const int s = g / per, i = g - s * per, left = chunks - i * a.per_segment;
    return uniform(make_int4(s * chunks + i * a.per_segment, left < a.per_segment ? left : a.per_segment, s,
                             (i == 0 ? 1 : 0) | (i == per - 1 ? 2 : 0)));
}

// ---------------------------------------------------------------- the tables of packed sequences

// Chunks and segments of every sequence, one after another (a sequence without tokens has one empty chunk: its state passes
// through).  One workgroup: a running sum over the sequences, then each table entry finds its sequence by bisection.
__global__ __launch_bounds__(1024) void scan_tables_kernel(ScanArgs a, int* __restrict__ first_chunk) {
    __shared__ int2 sums[1024];
    __shared__ int2 base;
    const int tid = threadIdx.x, S = a.seq.S;
    if (tid == 0) base = make_int2(0, 0);
    __syncthreads();
    for (int s0 = 0; s0 < S; s0 += 1024) {
        const int s = s0 + tid;
        int2 n = make_int2(0, 0);
        if (s < S) {
            const Span p = span_of(a.seq, s);
            n.x = p.end > p.begin ? (p.end - p.begin + kChunk - 1) / kChunk : 1;
            n.y = (n.x + a.per_segment - 1) / a.per_segment;
        }
        sums[tid] = n;
        __syncthreads();
        for (int d = 1; d < 1024; d <<= 1) {
            const int2 o = tid >= d ? sums[tid - d] : make_int2(0, 0);
            __syncthreads();
            sums[tid].x += o.x;
            sums[tid].y += o.y;
            __syncthreads();
        }
        if (s < S) {
            // (bad offsets may claim more chunks than there is room for: those past it do not exist)
            const int c = base.x + sums[tid].x - n.x, g = base.y + sums[tid].y - n.y;
            first_chunk[s] = c < a.nchunks ? c : a.nchunks;
            a.first_segment[s] = g < a.nsegments ? g : a.nsegments;
        }
        __syncthreads();
        if (tid == 0) {
            base.x = base.x + sums[1023].x < a.nchunks ? base.x + sums[1023].x : a.nchunks;
            base.y = base.y + sums[1023].y < a.nsegments ? base.y + sums[1023].y : a.nsegments;
        }
        __syncthreads();
    }
    if (tid == 0) {
        first_chunk[S] = base.x;
        a.first_segment[S] = base.y;
    }
    __syncthreads();
    auto owner = [&](const int* first, int i) {  // the last sequence that starts at entry i or before it
        int lo = 0, hi = S - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    for (int i = tid; i < a.nchunks; i += 1024) {
        int4 v = make_int4(0, 0, -1, 0);
        if (i < first_chunk[S]) {
            const int s = owner(first_chunk, i);
            const Span p = span_of(a.seq, s);
            const int at = p.begin + (i - first_chunk[s]) * kChunk, left = p.end - at;
            v = make_int4(at, left < 0 ? 0 : left < kChunk ? left : kChunk, s, 0);
        }
        a.chunks[i] = v;
    }
    for (int i = tid; i < a.nsegments; i += 1024) {
        int4 v = make_int4(0, 0, -1, 0);
        if (i < a.first_segment[S]) {
            const int s = owner(a.first_segment, i), n = i - a.first_segment[s];
            const int c = first_chunk[s] + n * a.per_segment, left = first_chunk[s + 1] - c;
            // (no chunks are left only where bad offsets claimed more than there is room for)
            v = make_int4(c, left < a.per_segment ? left : a.per_segment, left > 0 ? s : -1,
                          (n == 0 ? 1 : 0) | (i + 1 == a.first_segment[s + 1] ? 2 : 0));
        }
        a.segments[i] = v;
    }
}

// ---------------------------------------------------------------- prepare

// The decays of one head over a chunk, a token a lane.
__device__ void head_arrays(const ScanArgs& a, const int4& ch, int c, int h) {
    const int lane = threadIdx.x & 63;
    float dt = 0.0f;
    if (lane < ch.y) dt = scan_softplus(a.dt[(int64_t)(ch.x + lane) * a.lddt + h] + a.dt_bias[h]);
    // A factor below 2^-4096 is zero, and so is every product of decays that has it: cut there, the sums stay finite.
    double cs = -(double)dt * (double)expf(a.A_log[h]) * kLog2eD;
    cs = cs < -4096.0 ? -4096.0 : cs;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(cs, d);
        if (lane >= d) cs += o;
    }
    const double end = __shfl(cs, 63);
    float* const out = a.heads + ((int64_t)c * a.H + h) * kHeadArrays * kChunk + lane;
    const float hi = (float)cs;
    out[kCsHi * kChunk] = hi;
    out[kCsLo * kChunk] = (float)(cs - (double)hi);
    out[kStep * kChunk] = dt;
    out[kWeight * kChunk] = dt * __builtin_amdgcn_exp2f((float)(end - cs));
    out[kDecay * kChunk] = __builtin_amdgcn_exp2f(hi);
    const double before = __shfl(cs, lane < 16 ? 0 : (lane & 48) - 1), behind = __shfl(cs, lane | 15);
    out[kEnter * kChunk] = __builtin_amdgcn_exp2f((float)(cs - (lane < 16 ? 0.0 : before)));
    out[kLeave * kChunk] = dt * __builtin_amdgcn_exp2f((float)(behind - cs));
}

// Workgroups (chunk, y): y below G a group's products and its pieces along the state, below 2 G those across the tokens, behind
// them the decays of 16 heads each.
constexpr int kPrepareWaves = 8, kPrepareHeads = 2 * kPrepareWaves;
template <bool kBf16, int kN, bool kBackward>
__global__ __launch_bounds__(kPrepareWaves * 64) void prepare_kernel(ScanArgs a) {
    constexpr int kPieces = kBf16 ? 1 : 3, kLd = kN + 4, kTiles = kN / 16, kSteps = kN / 32, kThreads = kPrepareWaves * 64;
    using Block = GroupBlock<kN, kPieces>;
    __shared__ __attribute__((aligned(16))) float rows[2][kChunk * kLd];
    const int c = blockIdx.x;
    const int4 ch = chunk_of(a, c);
    if (ch.z < 0 || ch.y <= 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if ((int)blockIdx.y >= 2 * a.G) {
        for (int h = ((int)blockIdx.y - 2 * a.G) * kPrepareHeads + wave, n = 0; n < 2; ++n, h += kPrepareWaves)
            if (h < a.H) head_arrays(a, ch, c, h);
        return;
    }
    const bool is_across = (int)blockIdx.y >= a.G;
    const int g = is_across ? blockIdx.y - a.G : blockIdx.y;
    using E = Elem<kBf16>;
    const int matrices = is_across && !kBackward ? 1 : 2;     // (forward, B alone is wanted across the tokens)
#pragma unroll 4
    for (int i = tid; i < matrices * kChunk * (kN / 4); i += kThreads) {
        const int which = i / (kChunk * (kN / 4)), r = i / (kN / 4) % kChunk, k = i % (kN / 4) * 4;
        const int64_t at = (int64_t)(ch.x + (r < ch.y ? r : 0)) * (which ? a.ldc : a.ldb) + g * kN + k;
        v4f v = E::load4(static_cast<const typename E::type*>(which ? a.C : a.B) + at);
        if (r >= ch.y) v = v4f{0.0f, 0.0f, 0.0f, 0.0f};   // (whatever lies behind the sequence takes no part)
        *reinterpret_cast<v4f*>(&rows[which][r * kLd + k]) = v;
    }
    __syncthreads();
    uint8_t* const out = a.groups + ((int64_t)c * a.G + g) * (kBackward ? Block::backward : Block::forward);
    const int r = lane & 15, q = lane >> 4;
    // eight values of a token's row / across the tokens
    auto along = [&](int which, int tile, int step, float sign = 1.0f) {
        const float* p = &rows[which][(tile * 16 + r) * kLd + step * 32 + 4 * q];
        const v4f lo = sign * *reinterpret_cast<const v4f*>(p), hi = sign * *reinterpret_cast<const v4f*>(p + 16);
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        return split<kPieces>(v);
    };
    auto across = [&](int which, int tile, int step) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = rows[which][(step * 32 + place(q, j)) * kLd + tile * 16 + r];
        return split<kPieces>(v);
    };
    if (is_across) {
        for (int i = wave; i < kTiles * 2; i += kPrepareWaves) {
            store_pieces(out + Block::kAcross + (i * 64 + lane) * 16, Block::kPlane, across(0, i / 2, i % 2));
            if constexpr (kBackward)
                store_pieces(out + Block::kCross + (i * 64 + lane) * 16, Block::kPlane, across(1, i / 2, i % 2));
        }
        return;
    }
    // products: forward rows s, columns t (s <= t); backward rows t, columns s
    constexpr int kRowSide = kBackward ? 1 : 0;
    int n = 0;
    for (int rt = 0; rt < 4; ++rt)
        for (int ct = 0; ct < 4; ++ct) {
            if (kBackward ? ct > rt : ct < rt) continue;
            if (n++ % kPrepareWaves != wave) continue;
            v4f acc[2] = {};
            for (int k = 0; k < kSteps; k += 2) {
                acc[0] = mma(along(kRowSide, rt, k), along(1 - kRowSide, ct, k), acc[0]);
                acc[1] = mma(along(kRowSide, rt, k + 1, -1.0f), along(1 - kRowSide, ct, k + 1), acc[1]);
            }
            *reinterpret_cast<v4f*>(out + ((rt * 4 + ct) * 64 + lane) * 16) = opposite(acc);
        }
    for (int i = wave; i < 4 * kSteps; i += kPrepareWaves)
        store_pieces(out + Block::kRows + (i * 64 + lane) * 16, Block::kPlane, along(1 - kRowSide, i / kSteps, i % kSteps));
}

// ---------------------------------------------------------------- the sweep

// A part of what the heads share on its way from memory through registers to LDS: loaded while something else is worked on,
// written when that is done.  (Loads straight to LDS would cost no registers, but the compiler lets no later read of LDS
// pass one.)  Past the buffer it is zero.
template <int kBytes, int kThreads>
struct Staged {
    static constexpr int kEach = (kBytes + kThreads * 16 - 1) / (kThreads * 16);
    v4i v[kEach];
    __device__ __forceinline__ void load(const void* from, uint32_t bytes) {
        const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(from, bytes);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            v[i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rsrc, (i * kThreads + (int)threadIdx.x) * 16, 0, 0));
    }
    __device__ __forceinline__ void store(uint8_t* lds) const {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (kBytes % (kThreads * 16) == 0 || (i * kThreads + (int)threadIdx.x) * 16 < kBytes)
                *reinterpret_cast<v4i*>(lds + (i * kThreads + threadIdx.x) * 16) = v[i];
    }
};

__device__ __forceinline__ void unpack(float (&f)[8], v4f lo, v4f hi) {
    f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w, f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
}
__device__ __forceinline__ v4f at4(const float* p) { return *reinterpret_cast<const v4f*>(p); }

// A workgroup: four heads of a group (or two: the host's rule), a wave 32 channels of one.  A lane's two tiles of 16 channels hold the even and the
// odd ones, so that it reads and writes quads.  What the heads share of a chunk comes to LDS in two parts, each loaded
// while the other is worked on: products and C (for y), then B across the tokens (for the state); without y, B's
// part of the next chunk.
// (The bound: two waves to a SIMD; what lets only one workgroup of four waves on a CU has one.)
template <bool kBf16, int kN, int kMode, int kWaves>
__global__ __launch_bounds__(kWaves * 64, kWaves == 4 && (kMode == kOutput || !kBf16) ? 1 : 2) void sweep_kernel(SweepArgs s) {
    constexpr int kSweepThreads = kWaves * 64, kSweepHeads = kWaves / 2;
    // pieces of the data; of the state and of the chunk's own products where y is bf16: two leave an error of 2^-17, far
    // below its rounding; of what goes into the state, which is fp32 whatever the data: three
    constexpr int kData = kBf16 ? 1 : 3, kOut = kBf16 ? 2 : 3, kInto = 3;
    constexpr int kTiles = kN / 16, kSteps = kN / 32, kSize = RowBuffer<kBf16>::kSize;
    using Block = GroupBlock<kN, kData>;
    constexpr bool kY = kMode == kOutput;
    constexpr int kFirst = Block::kG + Block::kSet, kArrays = kSweepHeads * kHeadArrays * kChunk * 4;
    static_assert(Block::kRows == Block::kG, "the products and C's rows lie side by side");
    // y's two parts twice where there is room (bf16), so that a chunk needs one barrier and the waves drift apart: one's matrix
    // instructions run beside another's vector ones
    constexpr bool kTwice = kY && kBf16;
    __shared__ __attribute__((aligned(16))) uint8_t first_lds_[kY ? (kTwice ? 2 : 1) * kFirst : Block::kSet];
    __shared__ __attribute__((aligned(16))) uint8_t key_lds_[(kTwice ? 2 : 1) * Block::kSet];
    __shared__ __attribute__((aligned(16))) uint8_t head_lds[2][kArrays];
    const ScanArgs& a = s.a;
    const int per_group = a.H / a.G, quads = (per_group + kSweepHeads - 1) / kSweepHeads;
    const int seg = blockIdx.x / (a.G * quads), rest = blockIdx.x % (a.G * quads);
    const int g = rest / quads, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int head0 = rest % quads * kSweepHeads, in_group = head0 + (wave >> 1), half = wave & 1;
    const bool live = in_group < per_group;      // (the last heads of a group may not fill a workgroup)
    const int head = g * per_group + (live ? in_group : head0);
    const uint32_t array_bytes = (uint32_t)((per_group - head0 < kSweepHeads ? per_group - head0 : kSweepHeads) * kHeadArrays * kChunk * 4);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int4 sg = segment_of(a, seg);
    if (sg.z < 0) return;
    const int p0 = half * 32 + 2 * r;            // the lane's first channel

    auto chunk_at = [&](int i) { return s.reverse ? sg.x + sg.y - 1 - i : sg.x + i; };
    auto block_of = [&](int c) { return a.groups + ((int64_t)c * a.G + g) * s.group_bytes; };
    Staged<kArrays, kSweepThreads> next_arrays;
    Staged<kFirst, kSweepThreads> next_first;
    Staged<Block::kSet, kSweepThreads> next_key;
    auto load_arrays = [&](int i) {
        next_arrays.load(a.heads + ((int64_t)chunk_at(i) * a.H + g * per_group + head0) * kHeadArrays * kChunk, array_bytes);
    };

    // The state as sigma h.  The matrix instructions round down; with sigma changing from chunk to chunk their errors do, too.
    v4f h[kTiles][2];
    const int64_t mine = ((int64_t)sg.z * a.H + head) * kP * kN;
    float sigma = sg.x & 1 ? -1.0f : 1.0f;
    v4f* const slot = s.segment_states ? reinterpret_cast<v4f*>(s.segment_states) +
                                             (((int64_t)seg * a.H + head) * 2 + half) * kTiles * 2 * 64 + lane : nullptr;
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            h[n][p] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (kMode != kLocal) {
                if (slot) h[n][p] = sigma * slot[(n * 2 + p) * 64];
                else if (s.start) h[n][p] = sigma * at4(s.start + mine + (p0 + p) * kN + n * 16 + 4 * q);
            }
        }
    float through = 1.0f;  // the segment's decay
    const float skip = kY ? a.D[head] : 0.0f;
    const int count = chunk_of(a, sg.x).y > 0 ? sg.y : 0;   // (a sequence without tokens has one empty chunk)

    float v[2][2][8];
    typename RowBuffer<kBf16>::Pair raw[2][8];
    auto load_v = [&](int i) {   // the chunk's rows of v, places of the sums along its tokens; zero behind the sequence
        const int4 ch = chunk_of(a, chunk_at(i));
        const RowBuffer<kBf16> rows(s.v, ch.x, s.ldv, ch.y, head * kP + half * 32, 32);
        const int own = opaque(4 * q * (int)s.ldv + 2 * r) * kSize;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) raw[k][j] = rows.load2(own + (k * 32 + place(0, j)) * (int)s.ldv * kSize);
    };
    auto take_v = [&]() {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[k][0][j] = RowBuffer<kBf16>::first(raw[k][j]);
                v[k][1][j] = RowBuffer<kBf16>::second(raw[k][j]);
            }
    };
    if (count > 0) {
        load_arrays(0);
        if constexpr (kY) next_first.load(block_of(sg.x), kFirst);
        if constexpr (!kY || kTwice) next_key.load(block_of(chunk_at(0)) + s.key, Block::kSet);
        if constexpr (!kY) load_v(0);
    }
    for (int i = 0; i < count; ++i) {
        const int c = chunk_at(i), following = i + 1 < count ? i + 1 : i;   // (the last chunk's loads are idle ones: no branch)
        const float* const arrays = reinterpret_cast<const float*>(head_lds[i & 1]) + (live ? wave >> 1 : 0) * kHeadArrays * kChunk;
        uint8_t* const first_lds = first_lds_ + (kTwice ? (i & 1) * kFirst : 0);
        uint8_t* const key_lds = !kY && (i & 1) ? first_lds_ : key_lds_ + (kTwice ? (i & 1) * Block::kSet : 0);
        next_arrays.store(head_lds[i & 1]);
        if constexpr (kY) next_first.store(first_lds);
        if constexpr (!kY || kTwice) next_key.store(key_lds);
        lds_barrier();
        if constexpr (kY) {
            load_v(i);
            v4f y[4][2];
#pragma unroll
            for (int t = 0; t < 4; ++t) y[t][0] = y[t][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            const uint8_t* const rows = first_lds + Block::kRows + lane * 16;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                Pieces<kOut> state[2];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float f[8];
                    unpack(f, h[2 * k][p], h[2 * k + 1][p]);
                    state[p] = split<kOut>(f);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const Pieces<kData> cr = load_pieces<kData>(rows + (t * kSteps + k) * 1024, Block::kPlane);
                    y[t][0] = mma(cr, state[0], y[t][0]);
                    y[t][1] = mma(cr, state[1], y[t][1]);
                }
            }
            read_ahead<kData, 2 * products_of(kData, kOut), 4 * kSteps, 2, 16>();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const v4f e = sigma * at4(arrays + kDecay * kChunk + t * 16 + 4 * q);
                y[t][0] *= e;
                y[t][1] *= e;
            }
            take_v();
            float enter[4], between[4];     // between[t]: the decay of tile t as a whole
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                enter[t] = arrays[kEnter * kChunk + t * 16 + r];
                between[t] = arrays[kEnter * kChunk + t * 16 + 15];
            }
            const uint8_t* const products = first_lds + lane * 16;
#pragma unroll
            for (int k = 0; k < 2; ++k) {   // 32 tokens s, two tiles
                Pieces<kData> x[2];
                x[0] = split<kData>(v[k][0]);
                x[1] = split<kData>(v[k][1]);
                const v4f leave[2] = {at4(arrays + kLeave * kChunk + k * 32 + 4 * q), at4(arrays + kLeave * kChunk + k * 32 + 16 + 4 * q)};
#pragma unroll
                for (int t = 2 * k; t < 4; ++t) {
                    float w[8];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int st = 2 * k + u;   // the tile of s
                        v4f part = {0.0f, 0.0f, 0.0f, 0.0f};
                        if (st < t) {
                            float f = enter[t];
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                if (m > st && m < t) f *= between[m];
                            part = *reinterpret_cast<const v4f*>(products + (st * 4 + t) * 1024) * (leave[u] * f);
                        } else if (st == t) {
                            const float hi = arrays[t * 16 + r], lo = arrays[kCsLo * kChunk + t * 16 + r];
                            const v4f his = at4(arrays + t * 16 + 4 * q), los = at4(arrays + kCsLo * kChunk + t * 16 + 4 * q);
                            const v4f step = at4(arrays + kStep * kChunk + t * 16 + 4 * q);
                            const v4f product = *reinterpret_cast<const v4f*>(products + (t * 4 + t) * 1024);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                part[j] = product[j] * (step[j] * decay_between(hi - his[j], lo - los[j], r >= 4 * q + j));
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[u * 4 + j] = part[j];
                    }
                    const Pieces<kOut> wp = split<kOut>(w);
                    y[t][0] = mma(wp, x[0], y[t][0]);
                    y[t][1] = mma(wp, x[1], y[t][1]);
                }
            }
            if constexpr (!kTwice) {   // (three pieces are too many registers to hold before)
                __builtin_amdgcn_sched_barrier(0);
                next_key.load(block_of(c) + s.key, Block::kSet);
            }
            if (live) {
                const int4 ch = chunk_of(a, c);
                const RowBuffer<kBf16> out(s.y, ch.x, s.ldy, ch.y, head * kP + half * 32, 32);
                const int to = opaque(4 * q * (int)s.ldy + 2 * r) * kSize;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        out.store2(fmaf(skip, v[t >> 1][0][(t & 1) * 4 + j], y[t][0][j]),
                                   fmaf(skip, v[t >> 1][1][(t & 1) * 4 + j], y[t][1][j]), to + (t * 16 + j) * (int)s.ldy * kSize);
            }
            if constexpr (!kTwice) {
                next_key.store(key_lds);
                lds_barrier();
            }
            load_arrays(following);
            next_first.load(block_of(chunk_at(following)), kFirst);
            if constexpr (kTwice) next_key.load(block_of(chunk_at(following)) + s.key, Block::kSet);
        } else {
            take_v();
            // (before the stores: a wait for loads waits for the stores before them)
            load_arrays(following);
            next_key.load(block_of(chunk_at(following)) + s.key, Block::kSet);
            load_v(following);
            if constexpr (kMode == kStarts) {
                const __amdgpu_buffer_rsrc_t out =
                    make_rsrc(s.starts + ((int64_t)c * a.H + head) * kP * kN, live ? kP * kN * 4 : 0);
                const int to = opaque(p0 * kN + 4 * q) * 4;
#pragma unroll
                for (int n = 0; n < kTiles; ++n)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, sigma * h[n][p]), out, to + (p * kN + n * 16) * 4, 0, 0);
            }
        }
        const float last = arrays[kDecay * kChunk + kChunk - 1];
        through *= last;
        Pieces<kInto> in[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float* const from = arrays + (s.reverse ? kDecay : kWeight) * kChunk + k * 32 + 4 * q;
            float w[8];
            unpack(w, -sigma * at4(from), -sigma * at4(from + 16));
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = v[k][p][j] * w[j];
                in[k][p] = split<kInto>(f);
            }
        }
        const uint8_t* const keys = key_lds + lane * 16;
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            const Pieces<kData> key0 = load_pieces<kData>(keys + n * 2048, Block::kPlane);
            const Pieces<kData> key1 = load_pieces<kData>(keys + n * 2048 + 1024, Block::kPlane);
            v4f add[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) add[p] = mma(key0, in[0][p], v4f{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                add[p] = mma(key1, in[1][p], add[p]);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[n][p][j] = fmaf(h[n][p][j], -last, add[p][j]);
            }
        }
        read_ahead<kData, 2 * products_of(kData, kInto), 2 * kTiles, 2, (kY ? Staged<kFirst, kSweepThreads>::kEach : 16) + 1 + (!kY || kTwice ? Staged<Block::kSet, kSweepThreads>::kEach : 0)>();
        sigma = -sigma;
    }
    if (!live) return;
    if constexpr (kMode == kLocal) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int p = 0; p < 2; ++p) slot[(n * 2 + p) * 64] = sigma * h[n][p];
        if (half == 0 && lane == 0) s.segment_decay[(int64_t)seg * a.H + head] = through;
    } else if (s.end && (sg.w & (s.reverse ? 1 : 2))) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int p = 0; p < 2; ++p) *reinterpret_cast<v4f*>(s.end + mine + (p0 + p) * kN + n * 16 + 4 * q) = sigma * h[n][p];
    }
}

// The state at the start of every segment of a sequence, in place of what the segments add.
template <int kN>
__global__ __launch_bounds__(256) void join_segments_kernel(SweepArgs s) {
    constexpr int kTiles = kN / 16, kEach = kP * kN / 4;   // v4f of a head
    const int sequence = blockIdx.x / s.a.H, head = blockIdx.x % s.a.H;
    const int i = blockIdx.y * 256 + threadIdx.x;
    const int lane = i & 63, p = i / 64 % 2, n = i / 128 % kTiles, half = i / (128 * kTiles);
    const int per = (s.a.seq.L + kChunk - 1) / kChunk;
    const int each = s.a.segments ? 0 : (per + s.a.per_segment - 1) / s.a.per_segment;
    const int first = s.a.segments ? s.a.first_segment[sequence] : sequence * each;
    const int count = (s.a.segments ? s.a.first_segment[sequence + 1] : first + each) - first;
    v4f h = {0.0f, 0.0f, 0.0f, 0.0f};
    if (s.start)
        h = *reinterpret_cast<const v4f*>(s.start + (((int64_t)sequence * s.a.H + head) * kP + half * 32 + 2 * (lane & 15) + p) * kN +
                                          n * 16 + 4 * (lane >> 4));
    v4f* const states = reinterpret_cast<v4f*>(s.segment_states);
#pragma unroll 4
    for (int k = 0; k < count; ++k) {
        const int64_t at = (int64_t)(s.reverse ? first + count - 1 - k : first + k) * s.a.H + head;
        const v4f add = states[at * kEach + i];
        const float decay = s.segment_decay[at];
        states[at * kEach + i] = h;
        h = h * decay + add;
    }
}

// ---------------------------------------------------------------- the recurrence, token by token

// As in the decode step, 16 channels of a head to a workgroup and 16 threads to a channel: each state value is read
// and written once by one thread.  A wave forms the steps and decays of 64 tokens at once, a token a lane; four tokens' rows are
// in flight together.  With one sequence the launch and the chain of loads are its time (4.2 us); with many, the states: 64
// sequences of a token 50 us, 5.3 TB/s of the 270 MB.  Longer ones are bound by latency, a turn of four tokens 1.2 us at 64 heads.
template <bool kBf16, int kN>
__global__ __launch_bounds__(256) void recurrent_kernel(SweepArgs s) {
    constexpr int kV = kN / 16, kV4 = kV / 4;
    using E = Elem<kBf16>;
    using T = typename E::type;
    const ScanArgs& a = s.a;
    const int head = blockIdx.x / 4, p = blockIdx.x % 4 * 16 + threadIdx.x / 16, q = threadIdx.x % 16;
    const int sequence = blockIdx.y, g = head / (a.H / a.G), lane = threadIdx.x & 63;
    const Span span = span_of(a.seq, sequence);
    const int64_t at = (((int64_t)sequence * a.H + head) * kP + p) * kN + kV * q;
    v4f h[kV4];
#pragma unroll
    for (int i = 0; i < kV4; ++i) h[i] = s.start ? *reinterpret_cast<const v4f*>(s.start + at + 4 * i) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
    struct Row {
        float x;
        v4f b[kV4], c[kV4];
    };
    auto fetch = [&](Row& row, int t) {
        row.x = E::load(static_cast<const T*>(s.v) + t * s.ldv + head * kP + p);
#pragma unroll
        for (int i = 0; i < kV4; ++i) {
            row.b[i] = E::load4(static_cast<const T*>(a.B) + t * a.ldb + g * kN + kV * q + 4 * i);
            row.c[i] = E::load4(static_cast<const T*>(a.C) + t * a.ldc + g * kN + kV * q + 4 * i);
        }
    };
    const float rate = expf(a.A_log[head]), bias = a.dt_bias[head], skip = a.D[head];
    auto step = [&](const Row& row, int t, float dt, float decay) {
        const float dtx = dt * row.x;
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < kV4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[i][j] = fmaf(h[i][j], decay, dtx * row.b[i][j]);
                y = fmaf(h[i][j], row.c[i][j], y);
            }
        y += dpp_f<kDppXor1>(y);
        y += dpp_f<kDppXor2>(y);
        y += dpp_f<kDppHalfMirror>(y);
        y += dpp_f<kDppMirror>(y);
        if (q == 0) E::store(static_cast<T*>(s.y) + t * s.ldy + head * kP + p, fmaf(skip, row.x, y));
    };
    for (int t0 = span.begin; t0 < span.end; t0 += 64) {
        const int mine = t0 + lane < span.end ? t0 + lane : span.end - 1, stop = t0 + 64 < span.end ? t0 + 64 : span.end;
        const float dts = scan_softplus(a.dt[mine * a.lddt + head] + bias), decays = expf(-dts * rate);
        auto of = [&](float v, int t) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), t - t0)); };
        int t = t0;
        for (; t + 4 <= stop; t += 4) {
            Row rows[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) fetch(rows[j], t + j);
#pragma unroll
            for (int j = 0; j < 4; ++j) step(rows[j], t + j, of(dts, t + j), of(decays, t + j));
        }
        for (; t < stop; ++t) {
            Row row;
            fetch(row, t);
            step(row, t, of(dts, t), of(decays, t));
        }
    }
    if (s.end)
#pragma unroll
        for (int i = 0; i < kV4; ++i) *reinterpret_cast<v4f*>(s.end + at + 4 * i) = h[i];
}

}  // namespace

hipError_t launch_scan_prepare(const ScanArgs& a, bool bf16, int N, bool backward, hipStream_t stream) {
    if (a.chunks) {
        scan_tables_kernel<<<1, 1024, 0, stream>>>(a, a.first_segment + a.seq.S + 1);
        if (hipError_t err = hipGetLastError()) return err;
    }
    return with_kind(bf16, N, [&](auto b, auto n) {
        const dim3 grid((unsigned)a.nchunks, (unsigned)(2 * a.G + (a.H + kPrepareHeads - 1) / kPrepareHeads));
        if (backward) prepare_kernel<b.value, n.value, true><<<grid, kPrepareWaves * 64, 0, stream>>>(a);
        else prepare_kernel<b.value, n.value, false><<<grid, kPrepareWaves * 64, 0, stream>>>(a);
        return hipGetLastError();
    });
}

hipError_t launch_sweep(const SweepArgs& s, const ScanPlan& plan, bool bf16, int N, SweepMode mode, hipStream_t stream) {
    auto sweep = [&](auto b, auto n, auto w) {
        constexpr int kHeads = w.value / 2, kThreads = w.value * 64;
        const dim3 grid((unsigned)(plan.nsegments * s.a.G * ((s.a.H / s.a.G + kHeads - 1) / kHeads)));
        if constexpr (w.value == 8) if (plan.segmented) {    // (workgroups of two heads are taken where nothing is cut)
            sweep_kernel<b.value, n.value, kLocal, w.value><<<grid, kThreads, 0, stream>>>(s);
            if (hipError_t err = hipGetLastError()) return err;
            join_segments_kernel<n.value><<<dim3((unsigned)(s.a.seq.S * s.a.H), kP * n.value / 1024), 256, 0, stream>>>(s);
            if (hipError_t err = hipGetLastError()) return err;
        }
        if (mode == kStarts) sweep_kernel<b.value, n.value, kStarts, w.value><<<grid, kThreads, 0, stream>>>(s);
        else sweep_kernel<b.value, n.value, kOutput, w.value><<<grid, kThreads, 0, stream>>>(s);
        return hipGetLastError();
    };
    return with_kind(bf16, N, [&](auto b, auto n) {
        return plan.waves == 4 ? sweep(b, n, std::integral_constant<int, 4>()) : sweep(b, n, std::integral_constant<int, 8>());
    });
}

// ---------------------------------------------------------------- the host's side

// Whether the sequences go token by token: by their average length and, in units of 64, the number of heads of all of them.  (Lengths
// that offsets give lie in device memory.  Where one is far above the average it costs what its form costs it, 64 heads, bf16:
// among 63 single tokens a prompt of 500, token by token, 240 us, where the two alone take 44 and 46; among 255 one of 1800
// 947, alone 196 and 62.)
// Measured in us, d_state 128 (token by token 2, 8, 16, 32, 64 tokens | chunks up to 64 tokens):
//   1 x 64 heads, fp32  4.2, 5.6, 7.7, 11.7, 20.0 | 27;   bf16  4.2, 5.5, 7.4, 11.3, 19.1 | 21
//   8 x 64 heads, fp32  10, 17, 26, 45, 79 | 31;   bf16  10, 14, 21, 35, 60 | 25
//   64 x 64 heads, fp32  57, 116, 178, 303, 582 | 115 to 136;   bf16  49, 80, 128, 214, 382 | 88 to 98
bool scan_recurrent(const Sequences& seq, int H) {
    const float units = (float)seq.S * (float)H / 64.0f, tokens = (float)seq.T / (float)seq.S;
    return tokens * (0.15f + 0.13f * units) <= 18.0f + units;
}

// Enough workgroups for one on each CU: what one segment a sequence does not give, more segments do, at the price of a
// second sweep without outputs.  It goes by the number of sequences, as if all were of one length: a long one among many that would fill
// the CUs is not cut, and its chunks go one after another (64 heads, bf16: 16384 tokens in one sequence 289 us in a row of calls,
// 16000 and five of 64 1.18 ms, with 15 or 31 of 64 1.7 ms; with gradients 1.30, 3.8 and 5.7 ms).  Where workgroups of two heads fill three quarters of the CUs without it, they are taken instead
// (8 x 2048 tokens, bf16: states 160 us a sweep, 221 by segments and four heads; one sequence of 16384 tokens, cut into segments
// anyway: 285 us, 221 with four heads; 2048 fp32 78 and 75).
constexpr int kSweepGroups = 256;
constexpr int64_t kMaxSegmentHeads = 8 * kSweepGroups;   // the most heads that have segments' states: 67 MB at d_state 128

ScanPlan scan_plan(const Sequences& seq, int H, int G) {
    ScanPlan p{};
    const int64_t each = (seq.L + kChunk - 1) / kChunk;    // chunks of a sequence, without offsets
    p.nchunks = (int)(seq.cu ? seq.T / kChunk + seq.S : seq.S * each);
    auto units = [&](int heads) { return (int64_t)G * ((H / G + heads - 1) / heads); };
    const bool pairs = seq.S * units(4) < kSweepGroups && seq.S * units(2) * 4 >= kSweepGroups * 3;
    p.waves = pairs ? 4 : 8;
    int64_t per = p.nchunks;
    if (!pairs && seq.S * units(4) < kSweepGroups) per = (p.nchunks * units(4) + kSweepGroups - 1) / kSweepGroups;
    auto segments = [&](int64_t n) { return seq.cu ? p.nchunks / n + seq.S : seq.S * ((each + n - 1) / n); };
    while (per < p.nchunks && segments(per) * H > kMaxSegmentHeads) per *= 2;
    if (per > p.nchunks) per = p.nchunks;
    p.segmented = seq.cu ? per < p.nchunks : per < each;
    if (!p.segmented) per = p.nchunks;
    p.per_segment = (int)per;
    p.nsegments = (int)(p.segmented ? segments(per) : seq.S);
    return p;
}

int scan_group_bytes(bool bf16, int N, bool backward) {
    int bytes = 0;
    (void)with_kind(bf16, N, [&](auto b, auto n) {
        using Block = GroupBlock<n.value, b.value ? 1 : 3>;
        bytes = backward ? Block::backward : Block::forward;
        return hipSuccess;
    });
    return bytes;
}

// The workspace's parts that the forward and the backward pass share, for every number of tokens and sequences up to the
// given ones: bounds of each part, none of which falls as a size grows.
size_t scan_workspace(ScanArgs& a, SweepArgs& s, uint8_t* ws, int64_t T, int64_t S, int64_t H, int64_t G, int N, int group_bytes) {
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t* const p = ws + at;
        at += (size_t)(bytes + 255) / 256 * 256;
        return p;
    };
    const int64_t chunks = T / kChunk + S;
    a.chunks = reinterpret_cast<int4*>(take(chunks * 16));
    a.segments = reinterpret_cast<int4*>(take((chunks + S) * 16));
    a.first_segment = reinterpret_cast<int*>(take((S + 1) * 8));
    a.groups = take(chunks * G * group_bytes);
    a.heads = reinterpret_cast<float*>(take(chunks * H * kHeadArrays * kChunk * 4));
    // (at most a segment a chunk and one more a sequence)
    const int64_t heads = (chunks + S) * H < kMaxSegmentHeads ? (chunks + S) * H : kMaxSegmentHeads;
    s.segment_states = reinterpret_cast<float*>(take(heads * kP * N * 4));
    s.segment_decay = reinterpret_cast<float*>(take(heads * 4));
    return at;
}

size_t mamba2_scan_workspace_bytes(int64_t T, int64_t S, int64_t H, int64_t N, int64_t G) {
    ScanArgs a{};
    SweepArgs s{};
    return scan_workspace(a, s, nullptr, T, S, H, G, (int)N, scan_group_bytes(false, (int)N, false));
}

hipError_t launch_mamba2_scan(ScanArgs a, bool bf16, int N, const float* state_in, float* state_out, void* y, int64_t ldy,
                              void* workspace, hipStream_t stream) {
    SweepArgs s{};
    s.v = a.x;
    s.ldv = a.ldx;
    s.start = state_in;
    s.end = state_out;
    s.y = y;
    s.ldy = ldy;
    if (scan_recurrent(a.seq, a.H)) {
        s.a = a;
        return with_kind(bf16, N, [&](auto b, auto n) {
            recurrent_kernel<b.value, n.value><<<dim3((unsigned)(a.H * 4), (unsigned)a.seq.S), 256, 0, stream>>>(s);
            return hipGetLastError();
        });
    }
    const ScanPlan plan = scan_plan(a.seq, a.H, a.G);
    s.group_bytes = scan_group_bytes(bf16, N, false);
    scan_workspace(a, s, static_cast<uint8_t*>(workspace), a.seq.T, a.seq.S, a.H, a.G, N, s.group_bytes);
    if (!a.seq.cu) a.chunks = a.segments = nullptr;
    if (!plan.segmented) s.segment_states = nullptr;
    a.nchunks = plan.nchunks;
    a.nsegments = plan.nsegments;
    a.per_segment = plan.per_segment;
    s.a = a;
    (void)with_kind(bf16, N, [&](auto b, auto n) {
        s.key = GroupBlock<n.value, b.value ? 1 : 3>::kAcross;
        return hipSuccess;
    });
    if (hipError_t err = launch_scan_prepare(a, bf16, N, false, stream)) return err;
    return launch_sweep(s, plan, bf16, N, kOutput, stream);
}

}  // namespace dfssm
