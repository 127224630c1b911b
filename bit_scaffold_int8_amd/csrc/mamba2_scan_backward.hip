// mamba2_scan_backward.hip -- gradients of the Mamba-2 scan (gfx950).  With dh the gradient of the state,
//
//   dh_t = e^{a_{t+1}} dh_{t+1} + dy_t C_t^T,   dx_t = dt_t dh_t B_t + D dy_t,
//   dB_t = sum over heads dt_t dh_t^T x_t,   dC_t = sum over heads h_t^T dy_t,
//   ddt_t = x_t . (dh_t B_t) - exp(A_log) da_t,   da_t = e^{a_t} <dh_t, h_{t-1}>
//
// By chunks, as forward (scan.h, mamba2_scan.hip): one sweep forwards stores the state h at the start of every
// chunk, one backwards the gradient g at every chunk's end (the same kernel with x -> dy, B -> C), and then all chunks are
// independent.  In one, with L[t][s] = e^{cs_t - cs_s} for s <= t, M[t][s] = dy_t . x_s and K[t][s] = C_t . B_s:
//
//   dx_s = dt_s (sum_t K L dy_t + e^{cs_end - cs_s} g B_s) + D dy_s
//   dC_t = sum over heads (sum_s M L dt_s B_s + e^{cs_t} h^T dy_t)
//   dB_s = sum over heads (sum_t M L dt_s C_t + dt_s e^{cs_end - cs_s} g^T x_s)
//   E[t][s] = M K L:  x_s . (dh_s B_s) = sum_t E[t][s] + e^{cs_end - cs_s} <g, x_s B_s^T>, and da_t adds up what crosses from
//   before t to t or behind it: pairs s < t <= t' of E dt_s, h to t' >= t, s < t to g, and h to g.
//
// A workgroup takes a chunk and some heads of a group one after another; dC and dB, sums over heads, stay in its registers,
// and of the products M L dt B only the sum over the heads of M L dt is formed, and multiplied once.  The shares of several
// workgroups are joined in order.
//
// Measured, 64 heads of 64 channels, d_state 128, in us, means of 12 launches (prepare, sweep forwards, sweep backwards, gradients, joins):
//   2048 tokens fp32   11, 72, 72 (each with its segments), 111 (at best 109), 10.5;   8 x 2048 tokens bf16   22, 161, 161, 641 (598), 5
// The gradient kernel has one workgroup a CU (its registers are full: two waves to a SIMD), and a head of a chunk takes it
// 20 thousand cycles, of which the issue of its vector and matrix instructions (bf16 1120 and 81 a wave) is 11.5: the rest is waiting at
// its two barriers, for the states (64 KB a head and chunk; from the cache it would take 5 % less) and for LDS.
#include <math.h>

#include "scan.h"

namespace dfssm {

namespace {

constexpr int kThreads = 512;
constexpr int kGradGroups = 256;   // workgroups wanted of the gradient kernel: one for each CU
constexpr int kMaxSlabs = 2 * kGradGroups;
constexpr int kSums = 4;           // floats per chunk and head: sums of da a, dy . x, ddt (and one that pads)

struct ScanGradArgs {
    ScanArgs a;
    const void* dy;
    int64_t lddy;
    const float *starts, *ends;    // [chunk][H][64][N]: h at the chunk's start, its gradient at the chunk's end
    void *dx, *dB, *dC;
    int64_t lddx, lddb, lddc;
    float* ddt;
    int64_t ldddt;
    float* sums;                   // [chunk][H][kSums]
    float* slabs;                  // [slice][chunk][G][2][64][N]: shares of dB and dC
    int slices, per_slice, group_bytes;
};

template <bool kBf16, int kN>
struct GradLds {
    static constexpr int kData = kBf16 ? 1 : 3, kOut = kBf16 ? 2 : 3, kPlane = kChunk * kP * 2;
    static constexpr int kDy = 0, kX = kDy + kData * kPlane, kW = kX + kData * kPlane, kRows = kW + kOut * kPlane;
    static constexpr int kK = kRows + kData * kChunk * kN * 2, kPart = kK + kChunk * kChunk * 4;   // (the latter: floats)
    static constexpr int kRowSum = 0, kColSum = 8 * kChunk, kDiag = 12 * kChunk, kDot = 13 * kChunk, kU = 14 * kChunk,
                         kV = kU + kN / 16 * kChunk, kPass = kV + 4 * kChunk;   // (the first two hold doubles)
    static constexpr int kArrays = kPass + 32;                                  // the head's decays
    static constexpr int kParts = kArrays + kHeadArrays * kChunk, bytes = kPart + 2 * kParts * 4;   // (this turn's head and the one before)
    static constexpr int kLdSum = kChunk + 4;                           // the heads' sum of M L dt, over dy, x and W
    static_assert(kChunk * kLdSum * 4 <= kRows, "it fits");
};

// Another lane's value where every lane has a source: without a value to keep for others, no register need be cleared first.
template <int kCtrl>
__device__ __forceinline__ int lane_of(int v) { return __builtin_amdgcn_update_dpp(0, v, kCtrl, 0xF, 0xF, true); }
template <int kCtrl>
__device__ __forceinline__ float lane_of(float v) { return __int_as_float(lane_of<kCtrl>(__float_as_int(v))); }

__device__ __forceinline__ float row_sum(float v) {   // over the 16 lanes of a row
    v += lane_of<kDppXor1>(v);
    v += lane_of<kDppXor2>(v);
    v += lane_of<kDppHalfMirror>(v);
    v += lane_of<kDppMirror>(v);
    return v;
}

// The same in fp64.  E's sums are: what da takes of them is the small difference of what all of a chunk's pairs add up to, and
// its error is the same for many tokens, so that it stays in the sums over the tokens (dA_log of 2048 tokens against 64 bits:
// 1.0e-6 with sums in fp32).
template <int kCtrl>
__device__ __forceinline__ double lane_of(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)lane_of<kCtrl>((int)(uint32_t)(u >> 32)) << 32 |
                                          (uint32_t)lane_of<kCtrl>((int)(uint32_t)u));
}
__device__ __forceinline__ double row_sum(double v) {
    v += lane_of<kDppXor1>(v);
    v += lane_of<kDppXor2>(v);
    v += lane_of<kDppHalfMirror>(v);
    v += lane_of<kDppMirror>(v);
    return v;
}

template <bool kBf16, int kN>
__global__ __launch_bounds__(kThreads, 2) void scan_grad_kernel(ScanGradArgs s) {
    using Lds = GradLds<kBf16, kN>;
    using Block = GroupBlock<kN, Lds::kData>;
    using E = Elem<kBf16>;
    using T = typename E::type;
    constexpr int kSize = RowBuffer<kBf16>::kSize;
    constexpr int kData = Lds::kData, kOut = Lds::kOut, kFull = 3, kPlane = Lds::kPlane;
    // a wave's part of dB and dC: one tile of 16 state places, kTT tiles of tokens
    constexpr int kTiles = kN / 16, kParts = 8 / kTiles, kTT = 4 / kParts, kSteps = kN / 32;
    __shared__ __attribute__((aligned(16))) uint8_t lds[Lds::bytes];
    const ScanArgs& a = s.a;
    const int slice = blockIdx.y % s.slices, g = blockIdx.y / s.slices, c = blockIdx.x;
    const int per_group = a.H / a.G, first = slice * s.per_slice;
    const int last = first + s.per_slice < per_group ? first + s.per_slice : per_group;
    const int4 ch = chunk_of(a, c);
    if (ch.z < 0 || ch.y <= 0) return;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint8_t* const block = a.groups + ((int64_t)c * a.G + g) * s.group_bytes;

    // what stays for all heads: B's rows and K in LDS, and C at the places of this wave's part of dC
    for (int i = tid; i < Block::kSet / 16; i += kThreads)
        *reinterpret_cast<v4i*>(lds + Lds::kRows + i * 16) = *reinterpret_cast<const v4i*>(block + Block::kRows + i * 16);
    for (int i = tid; i < kChunk * kChunk / 4; i += kThreads)
        *reinterpret_cast<v4i*>(lds + Lds::kK + i * 16) = *reinterpret_cast<const v4i*>(block + i * 16);
    for (int i = tid; i < kOut * kPlane / 16; i += kThreads)    // (tiles above the diagonal stay zero)
        *reinterpret_cast<v4i*>(lds + Lds::kW + i * 16) = v4i{0, 0, 0, 0};
    // M's tiles: columns st, rows st + half and st + half + 2 (up to 3).  Waves w and w + 4 are on one SIMD: the ten tiles are dealt so
    // that none has more than three, and wave 4, which has none, finishes the head before (dealt in order, four to one SIMD and one to
    // another, and each wave in turn to finish: 8 x 2048 tokens bf16 617 us, 599 now, at best).
    const int late = wave & 3, st = wave < 4 ? wave >> 1 : 3 - ((late ^ late >> 1) & 1), half = wave < 4 ? wave & 1 : 1 - (late & 1);
    constexpr int kIdle = 4;
    v4f sum_w[2] = {};
    const int nt = wave % kTiles, t0 = wave / kTiles * kTT;
    const RowBuffer<kBf16> c_rows(a.C, ch.x, a.ldc, ch.y, g * kN + nt * 16, 16);
    v4f c_at[kTT], acc_b[kTT], acc_c[kTT];
#pragma unroll
    for (int t = 0; t < kTT; ++t) {
        acc_b[t] = acc_c[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < 4; ++v) c_at[t][v] = c_rows.load((((t0 + t) * 16 + 4 * q + v) * (int)a.ldc + r) * kSize);
    }
    const int pt = wave & 3, sh = wave >> 2;          // dx's tiles: channels pt, tokens 2 sh and 2 sh + 1

    // The kernel's arguments (one struct, at the segment's start), read again where a turn needs them: kept over the turns they would fill the scalar registers
    // and be moved to and from vector ones, 200 instructions a turn (2048 tokens fp32 122 us).
    auto arguments = [] {
        auto p = (const __attribute__((address_space(4))) ScanGradArgs*)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(p));
        return p;
    };

    // What a turn needs of a head's rows and states is loaded in the turn before, as soon as the registers that hold it are free.
    v4f y0, y1, x0, x1;
    float decays = 0.0f;
    static_assert(kHeadArrays * kChunk <= kThreads, "one value a thread");
    auto load_rows = [&](int k, int r, int q) {   // dy and x along the channels: each wave one tile of rows and half of the channels
        const auto now = arguments();
        const int lddy = (int)now->lddy, ldx = (int)now->a.ldx;
        const int p = (g * per_group + k) * kP + (wave & 1) * 32, row = (wave >> 1) * 16 + r;
        const RowBuffer<kBf16> dy_rows(now->dy, ch.x, lddy, ch.y, p, 32), x_rows(now->a.x, ch.x, ldx, ch.y, p, 32);
        const int from_dy = (row * lddy + 4 * q) * kSize, from_x = (row * ldx + 4 * q) * kSize;
        y0 = dy_rows.load4(from_dy), y1 = dy_rows.load4(from_dy + 16 * kSize);
        x0 = x_rows.load4(from_x), x1 = x_rows.load4(from_x + 16 * kSize);
        if (tid < kHeadArrays * kChunk) decays = now->a.heads[((int64_t)c * now->a.H + g * per_group + k) * kHeadArrays * kChunk + tid];
    };
    float h_at[2][8], dh_at[2][8];
    auto load_states = [&](int k, int from) { // the states at this wave's places, across the channels
        const auto now = arguments();
        const int64_t at = ((int64_t)c * now->a.H + g * per_group + k) * kP * kN;
        const RowBuffer<false> h(now->starts, 0, 0, 1, at, kP * kN), dh(now->ends, 0, 0, 1, at, kP * kN);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h_at[i][j] = h.load(from + (i * 32 + place(0, j)) * kN * 4);
                dh_at[i][j] = dh.load(from + (i * 32 + place(0, j)) * kN * 4);
            }
    };
    // ddt of a head and its share of the parameters' sums, a token a lane: by one wave in the turn after the head's own, from
    // what the turn has left in LDS
    auto finish = [&](int k, int lane) {
        const auto now = arguments();
        const int head = g * per_group + k;
        const float* const part = reinterpret_cast<const float*>(lds + Lds::kPart) + (k & 1) * Lds::kParts;
        const float* const arrays = part + Lds::kArrays;
        const double* const row_sums = reinterpret_cast<const double*>(part + Lds::kRowSum);
        const double* const column_sums = reinterpret_cast<const double*>(part + Lds::kColSum);
        const float hi = arrays[lane], lo = arrays[kCsLo * kChunk + lane], dt = arrays[kStep * kChunk + lane];
        const float end_hi = arrays[kChunk - 1], end_lo = arrays[kCsLo * kChunk + kChunk - 1];
        double rows = 0.0;
        float u = 0.0f, v = 0.0f;
        double pass = 0.0;
        for (int i = 0; i <= lane >> 4; ++i) rows += row_sums[i * kChunk + lane];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) u += part[Lds::kU + i * kChunk + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) v += part[Lds::kV + i * kChunk + lane];
#pragma unroll
        for (int i = 0; i < 32; ++i) pass += (double)part[Lds::kPass + i];
        const double columns = column_sums[lane] + column_sums[kChunk + lane];
        u *= arrays[kDecay * kChunk + lane];
        v *= __builtin_amdgcn_exp2f((end_hi - hi) + (end_lo - lo));
        pass *= arrays[kDecay * kChunk + kChunk - 1];
        const float z = (float)columns + part[Lds::kDiag + lane] + v;    // x . (dh B)
        // from t on: rows of E and u, less the columns from t on (pairs that lie behind t whole); before t: v
        double from = rows + (double)u - (double)dt * columns, before = (double)dt * (double)v;
        const double own = before;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double o = __shfl_down(from, d), p = __shfl_up(before, d);
            if (lane + d < 64) from += o;
            if (lane >= d) before += p;
        }
        const float da = (float)(from + (before - own) + pass);
        const float rate = expf(now->a.A_log[head]);
        float raw = 0.0f, ddt = 0.0f;
        if (lane < ch.y) {
            raw = now->a.dt[(int64_t)(ch.x + lane) * now->a.lddt + head] + now->a.dt_bias[head];
            ddt = (z - rate * da) * (raw > 20.0f ? 1.0f : 1.0f / (1.0f + expf(-raw)));
            now->ddt[(int64_t)(ch.x + lane) * now->ldddt + head] = ddt;
        }
        float sum_a = -rate * dt * da, sum_d = part[Lds::kDot + lane], sum_t = ddt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            sum_a += __shfl_xor(sum_a, d);
            sum_d += __shfl_xor(sum_d, d);
            sum_t += __shfl_xor(sum_t, d);
        }
        if (lane == 0)
            *reinterpret_cast<v4f*>(now->sums + ((int64_t)c * now->a.H + head) * kSums) = v4f{sum_a, sum_d, sum_t, 0.0f};
    };
    load_rows(first, r, q);
    for (int k = first; k < last; ++k) {
        // (what depends on the lane is formed anew in each turn: kept over the turns it would fill the registers)
        const int lane = opaque(tid & 63), r = lane & 15, q = lane >> 4;
        const int head = g * per_group + k;
        float* const part = reinterpret_cast<float*>(lds + Lds::kPart) + (k & 1) * Lds::kParts;
        float* const arrays = part + Lds::kArrays;
        if (tid < kHeadArrays * kChunk) arrays[tid] = decays;
        double* const row_sums = reinterpret_cast<double*>(part + Lds::kRowSum);
        double* const column_sums = reinterpret_cast<double*>(part + Lds::kColSum);
        {   // (x's second half negated: opposite())
            const float sign = wave & 1 ? -1.0f : 1.0f;
            const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
            const float x[8] = {sign * x0.x, sign * x0.y, sign * x0.z, sign * x0.w, sign * x1.x, sign * x1.y, sign * x1.z, sign * x1.w};
            store_pieces(lds + Lds::kDy + (wave * 64 + lane) * 16, kPlane, split<kData>(y));
            store_pieces(lds + Lds::kX + (wave * 64 + lane) * 16, kPlane, split<kData>(x));
        }
        load_states(k, (4 * q * kN + nt * 16 + r) * 4);
        float pass = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                pass = fmaf(h_at[i][j], dh_at[i][j], pass);
                if (i) h_at[i][j] = -h_at[i][j];
            }
        const Pieces<kFull> hp[2] = {split<kFull>(h_at[0]), split<kFull>(h_at[1])};
        const Pieces<kFull> dhp[2] = {split<kFull>(dh_at[0]), split<kFull>(dh_at[1])};
        __syncthreads();
        if (k > first && wave == kIdle) finish(k - 1, lane);
        __builtin_amdgcn_sched_barrier(0);
        {   // dC and dB through the states
            v4f us[kTT];     // C . (h^T dy), the wave's places
#pragma unroll
            for (int t = 0; t < kTT; ++t) {
                v4f us_[2], ws_[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
                    us_[j] = mma(load_pieces<kData>(lds + Lds::kDy + (((t0 + t) * 2 + j) * 64 + lane) * 16, kPlane), hp[j], zero);
                    ws_[j] = mma(load_pieces<kData>(lds + Lds::kX + (((t0 + t) * 2 + j) * 64 + lane) * 16, kPlane), dhp[j], zero);
                }
                const v4f u = opposite(us_), w = opposite(ws_);
                acc_c[t] += u * *reinterpret_cast<const v4f*>(arrays + kDecay * kChunk + (t0 + t) * 16 + 4 * q);
                acc_b[t] += w * *reinterpret_cast<const v4f*>(arrays + kWeight * kChunk + (t0 + t) * 16 + 4 * q);
#pragma unroll
                for (int v = 0; v < 4; ++v) us[t][v] = row_sum(u[v] * c_at[t][v]);
            }
            pass = row_sum(pass);
            if (r == 0) {
#pragma unroll
                for (int t = 0; t < kTT; ++t) *reinterpret_cast<v4f*>(part + Lds::kU + nt * kChunk + (t0 + t) * 16 + 4 * q) = us[t];
                part[Lds::kPass + wave * 4 + q] = t0 == 0 ? pass : 0.0f;
            }
        }
        // for dx: the state's gradient along the state
        v4f dh_rows[2 * kSteps];
        {
            const auto now = arguments();
            const RowBuffer<false> dh(now->ends, 0, 0, 1, ((int64_t)c * now->a.H + head) * kP * kN, kP * kN);
#pragma unroll
            for (int n = 0; n < 2 * kSteps; ++n) dh_rows[n] = dh.load4(((pt * 16 + r) * kN + 4 * q + n * 16) * 4);
        }
        __builtin_amdgcn_sched_barrier(0);
        {   // M, K L, E: columns s along the lanes
            const float s_dt = arrays[kStep * kChunk + st * 16 + r];
            double column = 0.0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tt = st + half + 2 * i;
                if (tt >= 4) continue;
                v4f both[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    both[j] = mma(load_pieces<kData>(lds + Lds::kDy + ((tt * 2 + j) * 64 + lane) * 16, kPlane),
                                  load_pieces<kData>(lds + Lds::kX + ((st * 2 + j) * 64 + lane) * 16, kPlane), v4f{0.0f, 0.0f, 0.0f, 0.0f});
                const v4f m = opposite(both);
                v4f f;     // L
                if (tt == st) {
                    const v4f hi = *reinterpret_cast<const v4f*>(arrays + tt * 16 + 4 * q);
                    const v4f lo = *reinterpret_cast<const v4f*>(arrays + kCsLo * kChunk + tt * 16 + 4 * q);
                    const float s_hi = arrays[st * 16 + r], s_lo = arrays[kCsLo * kChunk + st * 16 + r];
#pragma unroll
                    for (int v = 0; v < 4; ++v) f[v] = decay_between(hi[v] - s_hi, lo[v] - s_lo, 4 * q + v >= r);
                } else {
                    // behind s in its tile (leave has dt as a factor, which may be zero: from the sums), the tiles between, before t in its own
                    const float end_hi = arrays[st * 16 + 15], end_lo = arrays[kCsLo * kChunk + st * 16 + 15];
                    float behind = decay_between(end_hi - arrays[st * 16 + r], end_lo - arrays[kCsLo * kChunk + st * 16 + r], true);
                    for (int n = st + 1; n < tt; ++n) behind *= arrays[kEnter * kChunk + n * 16 + 15];
                    f = behind * *reinterpret_cast<const v4f*>(arrays + kEnter * kChunk + tt * 16 + 4 * q);
                }
                const v4f product = *reinterpret_cast<const v4f*>(lds + Lds::kK + ((tt * 4 + st) * 64 + lane) * 16);
                float kl[8], on_e = 0.0f, on_m = 0.0f;    // (on the diagonal)
                double rows[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const bool strict = tt > st || 4 * q + v > r;
                    kl[v] = product[v] * f[v];
                    kl[v + 4] = 0.0f;
                    const float e = m[v] * kl[v];
                    sum_w[i][v] = fmaf(m[v] * f[v], s_dt, sum_w[i][v]);
                    column += strict ? (double)e : 0.0;
                    rows[v] = row_sum(strict ? (double)e * (double)s_dt : 0.0);
                    on_e = r == 4 * q + v ? e : on_e;
                    on_m = r == 4 * q + v ? m[v] : on_m;
                }
                if (tt == st && q == r >> 2) {
                    part[Lds::kDiag + st * 16 + r] = on_e;
                    part[Lds::kDot + st * 16 + r] = on_m;
                }
                const Pieces<kOut> w = split<kOut>(kl);
#pragma unroll
                for (int n = 0; n < kOut; ++n)
                    *reinterpret_cast<v4bf*>(lds + Lds::kW + n * kPlane + ((st * 2 + (tt >> 1)) * 64 + lane) * 16 + (tt & 1) * 8) =
                        __builtin_shufflevector(w.p[n], w.p[n], 0, 1, 2, 3);
                if (r == 0)
#pragma unroll
                    for (int v = 0; v < 4; ++v) row_sums[st * kChunk + tt * 16 + 4 * q + v] = rows[v];
            }
            column += __shfl_xor(column, 16);
            column += __shfl_xor(column, 32);
            if (q == 0) column_sums[half * kChunk + st * 16 + r] = column;
        }
        __syncthreads();
        float dy[2][8], x_at[2][4];     // dy across the tokens, and x where dx lies
        {
            const auto now = arguments();
            const int lddy = (int)now->lddy, ldx = (int)now->a.ldx, p = head * kP + pt * 16;
            const RowBuffer<kBf16> dy_rows(now->dy, ch.x, lddy, ch.y, p, 16), x_rows(now->a.x, ch.x, ldx, ch.y, p, 16);
            const int from_dy = (4 * q * lddy + r) * kSize, from_x = ((sh * 32 + 4 * q) * ldx + r) * kSize;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) dy[i][j] = dy_rows.load(from_dy + (i * 32 + place(0, j)) * lddy * kSize);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) x_at[i][v] = x_rows.load(from_x + (i * 16 + v) * ldx * kSize);
        }
        load_rows(k + 1 < last ? k + 1 : k, r, q);
        __builtin_amdgcn_sched_barrier(0);
        {   // dx
            v4f halves[2][2] = {}, intra[2] = {};
#pragma unroll
            for (int n = 0; n < kSteps; ++n) {
                const v4f lo = dh_rows[2 * n], hi = dh_rows[2 * n + 1];
                const float sign = n & 1 ? -1.0f : 1.0f;
                const float f[8] = {sign * lo.x, sign * lo.y, sign * lo.z, sign * lo.w, sign * hi.x, sign * hi.y, sign * hi.z, sign * hi.w};
                const Pieces<kFull> state = split<kFull>(f);   // (ddt takes of it, too)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    halves[i][n & 1] = mma(load_pieces<kData>(lds + Lds::kRows + (((2 * sh + i) * kSteps + n) * 64 + lane) * 16, Block::kPlane),
                                           state, halves[i][n & 1]);
            }
            __builtin_amdgcn_sched_barrier(0);
            const Pieces<kData> rows[2] = {split<kData>(dy[0]), split<kData>(dy[1])};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (j >= sh)     // (tokens t from the tile's own on)
                        intra[i] = mma(load_pieces<kOut>(lds + Lds::kW + (((2 * sh + i) * 2 + j) * 64 + lane) * 16, kPlane), rows[j], intra[i]);
            const auto now = arguments();
            const float skip = now->a.D[head];
            const int lddx = (int)now->lddx;
            const RowBuffer<kBf16> dx_rows(now->dx, ch.x, lddx, ch.y, head * kP + pt * 16, 16);
            const int to = (4 * q * lddx + r) * kSize;
            v4f along[2];          // x . (g B)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tile = 2 * sh + i;
                const v4f dt = *reinterpret_cast<const v4f*>(arrays + kStep * kChunk + tile * 16 + 4 * q);
                const v4f weight = *reinterpret_cast<const v4f*>(arrays + kWeight * kChunk + tile * 16 + 4 * q);
                const v4f inter = opposite(halves[i]);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    along[i][v] = row_sum(x_at[i][v] * inter[v]);
                    const float own = sh == 0 ? dy[0][i * 4 + v] : dy[1][i * 4 + v];
                    dx_rows.store(fmaf(skip, own, fmaf(dt[v], intra[i][v], weight[v] * inter[v])),
                                  to + (tile * 16 + v) * lddx * kSize);
                }
            }
            if (r == 0)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<v4f*>(part + Lds::kV + pt * kChunk + (2 * sh + i) * 16 + 4 * q) = along[i];
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    if (wave == kIdle) finish(last - 1, lane);

    // dC += W B and dB += W^T C with W the heads' sum of M L dt
    __syncthreads();
    float* const w = reinterpret_cast<float*>(lds);
    for (int i = tid; i < kChunk * Lds::kLdSum; i += kThreads) w[i] = 0.0f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int tt = st + half + 2 * i;
        if (tt >= 4) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v) w[(tt * 16 + 4 * q + v) * Lds::kLdSum + st * 16 + r] = sum_w[i][v];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const Pieces<kData> across = load_pieces<kData>(block + Block::kAcross + ((nt * 2 + j) * 64 + lane) * 16, Block::kPlane);
        const Pieces<kData> cross = load_pieces<kData>(block + Block::kCross + ((nt * 2 + j) * 64 + lane) * 16, Block::kPlane);
#pragma unroll
        for (int t = 0; t < kTT; ++t) {
            const float* const from = w + ((t0 + t) * 16 + r) * Lds::kLdSum + j * 32 + 4 * q;
            const v4f lo = *reinterpret_cast<const v4f*>(from), hi = *reinterpret_cast<const v4f*>(from + 16);
            const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            acc_c[t] = mma(split<kOut>(f), across, acc_c[t]);
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = w[(j * 32 + place(q, i)) * Lds::kLdSum + (t0 + t) * 16 + r];
            acc_b[t] = mma(split<kOut>(e), cross, acc_b[t]);
        }
    }
    float* const slab = s.slabs ? s.slabs + ((((int64_t)slice * a.nchunks + c) * a.G + g) * 2) * kChunk * kN : nullptr;
#pragma unroll
    for (int t = 0; t < kTT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int row = (t0 + t) * 16 + 4 * q + v;
            if (row >= ch.y) continue;
            if (slab) {
                slab[row * kN + nt * 16 + r] = acc_b[t][v];
                slab[(kChunk + row) * kN + nt * 16 + r] = acc_c[t][v];
            } else {
                E::store(static_cast<T*>(s.dB) + (int64_t)(ch.x + row) * s.lddb + g * kN + nt * 16 + r, acc_b[t][v]);
                E::store(static_cast<T*>(s.dC) + (int64_t)(ch.x + row) * s.lddc + g * kN + nt * 16 + r, acc_c[t][v]);
            }
        }
}

// dB and dC: the slices' shares in their order; workgroups (chunk, group, a part of the rows).
template <bool kBf16, int kN>
__global__ __launch_bounds__(256) void join_slabs_kernel(ScanGradArgs s) {
    using E = Elem<kBf16>;
    using T = typename E::type;
    const ScanArgs& a = s.a;
    const int c = blockIdx.x, g = blockIdx.y;
    const int4 ch = chunk_of(a, c);
    if (ch.z < 0) return;
    const int64_t step = (int64_t)a.nchunks * a.G * 2 * kChunk * kN;
    const int i = blockIdx.z * 256 + threadIdx.x;
    const int which = i / (kChunk * kN / 4), row = i / (kN / 4) % kChunk, n = i % (kN / 4) * 4;
    if (row >= ch.y) return;
    const float* const from = s.slabs + (((int64_t)c * a.G + g) * 2 + which) * kChunk * kN + row * kN + n;
    v4f v = *reinterpret_cast<const v4f*>(from);
#pragma unroll 4
    for (int k = 1; k < s.slices; ++k) v += *reinterpret_cast<const v4f*>(from + k * step);
    if (which == 0) E::store4(static_cast<T*>(s.dB) + (int64_t)(ch.x + row) * s.lddb + g * kN + n, v);
    else E::store4(static_cast<T*>(s.dC) + (int64_t)(ch.x + row) * s.lddc + g * kN + n, v);
}

// The parameters' gradients of a head: the chunks' sums, each thread every 256th, then the threads in a tree.
__global__ __launch_bounds__(256) void join_sums_kernel(ScanArgs a, const float* __restrict__ sums, float* __restrict__ dA_log,
                                                        float* __restrict__ dD, float* __restrict__ ddt_bias) {
    __shared__ v4f part[256];
    const int head = blockIdx.x, tid = threadIdx.x;
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = tid; c < a.nchunks; c += 256) {
        if (a.chunks) {   // (the table's unused entries and empty chunks have no sums)
            const int4 ch = a.chunks[c];
            if (ch.z < 0 || ch.y <= 0) continue;
        }
        v += *reinterpret_cast<const v4f*>(sums + ((int64_t)c * a.H + head) * kSums);
    }
    part[tid] = v;
    __syncthreads();
    for (int d = 128; d > 0; d >>= 1) {
        if (tid < d) part[tid] += part[tid + d];
        __syncthreads();
    }
    if (tid == 0) {
        dA_log[head] = part[0].x;
        dD[head] = part[0].y;
        ddt_bias[head] = part[0].z;
    }
}

struct GradParts {
    float *starts, *ends, *sums, *slabs;
    size_t bytes;
};

GradParts grad_parts(ScanArgs& a, SweepArgs& s, uint8_t* ws, int64_t T, int64_t S, int64_t H, int64_t G, int N, int group_bytes) {
    GradParts p{};
    size_t at = scan_workspace(a, s, ws, T, S, H, G, N, group_bytes);
    auto take = [&](int64_t bytes) {
        float* const q = reinterpret_cast<float*>(ws + at);
        at += (size_t)(bytes + 255) / 256 * 256;
        return q;
    };
    const int64_t chunks = T / kChunk + S;
    p.starts = take(chunks * H * kP * N * 4);
    p.ends = take(chunks * H * kP * N * 4);
    p.sums = take(chunks * H * kSums * 4);
    // (a group's slices are no more than its heads)
    const int64_t slabs = chunks * H < kMaxSlabs ? chunks * H : kMaxSlabs;
    p.slabs = take(slabs * 2 * kChunk * N * 4);
    p.bytes = at;
    return p;
}

}  // namespace

size_t mamba2_scan_backward_workspace_bytes(int64_t T, int64_t S, int64_t H, int64_t N, int64_t G) {
    ScanArgs a{};
    SweepArgs s{};
    return grad_parts(a, s, nullptr, T, S, H, G, (int)N, scan_group_bytes(false, (int)N, true)).bytes;
}

hipError_t launch_mamba2_scan_backward(ScanArgs a, bool bf16, int N, const float* state_in, const void* dy, int64_t lddy,
                                       const float* dstate_out, void* dx, int64_t lddx, float* ddt, int64_t ldddt, void* dB,
                                       int64_t lddb, void* dC, int64_t lddc, float* dA_log, float* dD, float* ddt_bias,
                                       float* dstate_in, void* workspace, hipStream_t stream) {
    const ScanPlan plan = scan_plan(a.seq, a.H, a.G);
    SweepArgs s{};
    s.group_bytes = scan_group_bytes(bf16, N, true);
    const GradParts parts = grad_parts(a, s, static_cast<uint8_t*>(workspace), a.seq.T, a.seq.S, a.H, a.G, N, s.group_bytes);
    if (!a.seq.cu) a.chunks = a.segments = nullptr;
    if (!plan.segmented) s.segment_states = nullptr;
    a.nchunks = plan.nchunks;
    a.nsegments = plan.nsegments;
    a.per_segment = plan.per_segment;
    if (hipError_t err = launch_scan_prepare(a, bf16, N, true, stream)) return err;
    return with_kind(bf16, N, [&](auto b, auto n) {
        using Block = GroupBlock<n.value, b.value ? 1 : 3>;
        s.a = a;
        s.v = a.x;
        s.ldv = a.ldx;
        s.key = Block::kAcross;
        s.start = state_in;
        s.starts = parts.starts;
        if (hipError_t err = launch_sweep(s, plan, bf16, N, kStarts, stream)) return err;
        s.v = dy;
        s.ldv = lddy;
        s.key = Block::kCross;
        s.reverse = true;
        s.start = dstate_out;
        s.end = dstate_in;
        s.starts = parts.ends;
        if (hipError_t err = launch_sweep(s, plan, bf16, N, kStarts, stream)) return err;
        ScanGradArgs g{a, dy, lddy, parts.starts, parts.ends, dx, dB, dC, lddx, lddb, lddc, ddt, ldddt, parts.sums, nullptr, 1, 0,
                       s.group_bytes};
        const int per_group = a.H / a.G;
        const int64_t units = (int64_t)a.nchunks * a.G;
        const int64_t wanted = units >= kGradGroups ? 1 : (kGradGroups + units - 1) / units;
        g.per_slice = (int)((per_group + wanted - 1) / wanted);
        g.slices = (per_group + g.per_slice - 1) / g.per_slice;
        if (g.slices > 1) g.slabs = parts.slabs;
        scan_grad_kernel<b.value, n.value><<<dim3((unsigned)a.nchunks, (unsigned)(a.G * g.slices)), kThreads, 0, stream>>>(g);
        if (hipError_t err = hipGetLastError()) return err;
        if (g.slices > 1) {
            join_slabs_kernel<b.value, n.value><<<dim3((unsigned)a.nchunks, (unsigned)a.G, kChunk * n.value / 512), 256, 0, stream>>>(g);
            if (hipError_t err = hipGetLastError()) return err;
        }
        join_sums_kernel<<<dim3((unsigned)a.H), 256, 0, stream>>>(a, parts.sums, dA_log, dD, ddt_bias);
        return hipGetLastError();
    });
}

}  // namespace dfssm
