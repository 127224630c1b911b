// mamba2_conv.hip -- the causal convolution in front of the Mamba-2 scan, over packed sequences, and its
// gradients (gfx950).
//
//   pre_t = b + sum_j w_j u_{t-3+j},  out_t = silu(pre_t) = pre_t / (1 + exp(-pre_t)),  u = the window, then the rows
//   dpre_t = dout_t sig_t (1 + pre_t (1 - sig_t)),  du_t = sum_j w_j dpre_{t+3-j},
//   dw_j = sum_t dpre_t u_{t-3+j},  db = sum_t dpre_t
//
// Channels are independent and a row's neighbours are wanted four times, so a lane owns kVec neighbouring channels and walks
// over a run of rows with its last three inputs in registers: each row is read once, and 3 rows more a run (the
// backward pass 6, and recomputes pre).  A wave's lanes lie along a row: whole lines are read and written.  A run
// that crosses into the next sequence takes that one's window.  The windows themselves (16 bytes a channel and
// sequence) are the business of workgroups of their own, behind those of the runs.
//
// dw and db: each run's sums go to the workspace and are added in the order of the runs, so equal inputs give equal bits.
#include <math.h>

#include <type_traits>

#include "sequences.h"

namespace dfssm {

namespace {

constexpr int kWaves = 4;       // runs a workgroup walks, one a wave
// Rows of a run: 2048 x 4352 fp32 15.8 us, 18.2 with 16 (fewer waves), 24 with 32 (before sigmoid() below: 14.6 now, 4.9 TB/s of
// the 71 MB it cannot do without, which is what bounds it).  Backward a run costs six rows more: 32.
constexpr int kRun = 8, kGradRun = 32;

struct ConvArgs {
    Sequences seq;
    const void* u;
    int64_t ldu;
    int ch, runs;
    const float* w;      // [ch][4]
    const float* b;
    const float* win;    // [S][ch][4], or NULL: zeros
    float* wout;         // or NULL
    void* out;
    int64_t ldo;
};

struct ConvGradArgs {
    ConvArgs f;
    const void* dout;
    int64_t ldd;
    const float* dwout;  // [S][ch][4], or NULL: zeros
    void* du;
    int64_t lddu;
    float* part;         // [runs][5][ch]: dw_0 .. dw_3, db of each run; or NULL
    float* dwin;         // or NULL
};

// 1 / (1 + exp(-v)) to about two steps of fp32: the exponential in base 2 with the rounding of v log2 e made up for, and the
// hardware's reciprocal (expf and a correctly rounded division take three times the instructions, which then bound the
// kernel: 4158 x 4352 fp32 to bf16 27 us).  The argument is cut before anything is formed of it, so that the exponential and the
// correction stay finite: above 126 the result is 1; below -87 it is 0 (in truth below 2^-125, where the reciprocal ends), so
// that the product with any v, and the slope's, vanishes as it should.
__device__ __forceinline__ float sigmoid(float v) {
    constexpr float kLog2e = 1.44269504088896340736f, kLog2eRest = 1.92596299e-8f, kLn2 = 0.693147180559945f, kLeast = -87.0f;
    const float c = fminf(fmaxf(v, kLeast), 126.0f);   // (a NaN comes back with the product or the slope)
    const float t = -c * kLog2e, rest = fmaf(-c, kLog2e, -t) - c * kLog2eRest;
    const float e = __builtin_amdgcn_exp2f(t);
    const float s = __builtin_amdgcn_rcpf(fmaf(e, rest * kLn2, e) + 1.0f);
    return v < kLeast ? 0.0f : s;
}

// kVec channels' values of a row.
template <bool kBf16, int kVec>
__device__ __forceinline__ void load_row(float (&v)[kVec], const void* base, int64_t ld, int t, int c) {
    const auto* p = static_cast<const typename Elem<kBf16>::type*>(base) + t * ld + c;
    if constexpr (kVec == 4) {
        const v4f q = Elem<kBf16>::load4(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = q[i];
    } else {
        v[0] = Elem<kBf16>::load(p);
    }
}
template <bool kBf16, int kVec>
__device__ __forceinline__ void store_row(const float (&v)[kVec], void* base, int64_t ld, int t, int c) {
    auto* p = static_cast<typename Elem<kBf16>::type*>(base) + t * ld + c;
    if constexpr (kVec == 4) Elem<kBf16>::store4(p, v4f{v[0], v[1], v[2], v[3]});
    else Elem<kBf16>::store(p, v[0]);
}

// The input at row t of the sequence that starts at `begin`: a row, or a place of the window.
template <bool kBf16, int kVec>
__device__ __forceinline__ void input_at(float (&v)[kVec], const ConvArgs& a, int s, int begin, int t, int c) {
    if (t >= begin) {
        load_row<kBf16, kVec>(v, a.u, a.ldu, t, c);
        return;
    }
    const int at = t - begin + 4;
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = a.win ? a.win[((int64_t)s * a.ch + c + i) * 4 + (at < 0 ? 0 : at)] : 0.0f;
}

// Weights and biases of kVec channels.
template <int kVec>
struct Taps {
    float w[4][kVec], b[kVec];
    __device__ __forceinline__ Taps(const ConvArgs& a, int c) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const v4f q = *reinterpret_cast<const v4f*>(a.w + (int64_t)(c + i) * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j][i] = q[j];
            b[i] = a.b[c + i];
        }
    }
    // the same order of operations as the decode step's convolution
    __device__ __forceinline__ float pre(int i, float u0, float u1, float u2, float u3) const {
        return fmaf(w[3][i], u3, fmaf(w[2][i], u2, fmaf(w[1][i], u1, fmaf(w[0][i], u0, b[i]))));
    }
};

// A sequence's new window: its last four inputs.
template <bool kIn>
__device__ void advance_window(const ConvArgs& a, int s, int c) {
    const Span p = span_of(a.seq, s);
    v4f v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float x[1];
        input_at<kIn, 1>(x, a, s, p.begin, p.end - 4 + j, c);
        v[j] = x[0];
    }
    *reinterpret_cast<v4f*>(a.wout + ((int64_t)s * a.ch + c) * 4) = v;
}

template <bool kIn, bool kOut, int kVec>
__global__ __launch_bounds__(kWaves * 64) void conv_kernel(ConvArgs a) {
    const int groups = (a.runs + kWaves - 1) / kWaves;
    if ((int)blockIdx.y >= groups) {
        for (int s = blockIdx.y - groups; s < a.seq.S; s += gridDim.y - groups)
            for (int i = threadIdx.x; i < 64 * kVec; i += kWaves * 64)
                if (const int c = blockIdx.x * 64 * kVec + i; c < a.ch) advance_window<kIn>(a, s, c);
        return;
    }
    const int run = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * kWaves + threadIdx.x / 64));
    const int c = (blockIdx.x * 64 + (threadIdx.x & 63)) * kVec;
    if (run >= a.runs || c >= a.ch) return;
    const Taps<kVec> taps(a, c);
    int t = run * kRun;
    const int stop = t + kRun < a.seq.T ? t + kRun : a.seq.T;
    for (int s = sequence_at(a.seq, t); s < a.seq.S && t < stop; ++s) {
        const Span p = span_of(a.seq, s);
        if (p.begin >= stop) break;
        if (t < p.begin) t = p.begin;
        const int end = p.end < stop ? p.end : stop;
        if (t >= end) continue;
        float u[4][kVec];
#pragma unroll
        for (int j = 0; j < 3; ++j) input_at<kIn, kVec>(u[j], a, s, p.begin, t - 3 + j, c);
        // (unrolled: the loads of several rows are in flight together)
#pragma unroll 4
        for (; t < end; ++t) {
            load_row<kIn, kVec>(u[3], a.u, a.ldu, t, c);
            float o[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float pre = taps.pre(i, u[0][i], u[1][i], u[2][i], u[3][i]);
                o[i] = pre * sigmoid(pre);
#pragma unroll
                for (int j = 0; j < 3; ++j) u[j][i] = u[j + 1][i];
            }
            store_row<kOut, kVec>(o, a.out, a.ldo, t, c);
        }
    }
}

// dpre at row t of a sequence (a lone channel, for the windows' gradients).
template <bool kIn, bool kOut>
__device__ float dpre_at(const ConvGradArgs& a, const Taps<1>& taps, int s, const Span& p, int t, int c) {
    if (t < p.begin || t >= p.end) return 0.0f;
    float u[4][1], d[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) input_at<kIn, 1>(u[j], a.f, s, p.begin, t - 3 + j, c);
    load_row<kOut, 1>(d, a.dout, a.ldd, t, c);
    const float pre = taps.pre(0, u[0][0], u[1][0], u[2][0], u[3][0]), sig = sigmoid(pre);
    return d[0] * (sig * fmaf(pre, 1.0f - sig, 1.0f));
}

// The gradient of a sequence's window: what its first three rows take from it, and what a sequence of fewer than
// four rows leaves of it in the new window.
template <bool kIn, bool kOut>
__device__ void window_gradient(const ConvGradArgs& a, int s, int c) {
    const Span p = span_of(a.f.seq, s);
    const Taps<1> taps(a.f, c);
    float d[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) d[i] = dpre_at<kIn, kOut>(a, taps, s, p, p.begin + i, c);
    const int64_t at = ((int64_t)s * a.f.ch + c) * 4;
    const int len = p.end - p.begin;
    v4f v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float g = a.dwout && i >= len ? a.dwout[at + i - len] : 0.0f;
#pragma unroll
        for (int k = 0; k < i; ++k) g = fmaf(taps.w[i - 1 - k][0], d[k], g);
        v[i] = g;
    }
    *reinterpret_cast<v4f*>(a.dwin + at) = v;
}

template <bool kIn, bool kOut, int kVec>
__global__ __launch_bounds__(kWaves * 64) void conv_grad_kernel(ConvGradArgs a) {
    const ConvArgs& f = a.f;
    const int groups = (f.runs + kWaves - 1) / kWaves;
    if ((int)blockIdx.y >= groups) {
        for (int s = blockIdx.y - groups; s < f.seq.S; s += gridDim.y - groups)
            for (int i = threadIdx.x; i < 64 * kVec; i += kWaves * 64)
                if (const int c = blockIdx.x * 64 * kVec + i; c < f.ch) window_gradient<kIn, kOut>(a, s, c);
        return;
    }
    const int run = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * kWaves + threadIdx.x / 64));
    const int c = (blockIdx.x * 64 + (threadIdx.x & 63)) * kVec;
    if (run >= f.runs || c >= f.ch) return;
    const Taps<kVec> taps(f, c);
    float dw[4][kVec] = {}, db[kVec] = {};
    int t = run * kGradRun;
    const int stop = t + kGradRun < f.seq.T ? t + kGradRun : f.seq.T;
    for (int s = sequence_at(f.seq, t); s < f.seq.S && t < stop; ++s) {
        const Span p = span_of(f.seq, s);
        if (p.begin >= stop) break;
        if (t < p.begin) t = p.begin;
        const int end = p.end < stop ? p.end : stop;
        if (t >= end) continue;
        float u[4][kVec], d[4][kVec] = {};   // d[j]: dpre at row t - 3 + j
#pragma unroll
        for (int j = 0; j < 3; ++j) input_at<kIn, kVec>(u[j], f, s, p.begin, t - 3 + j, c);
        const int first = t;
        // row t + 3's dpre completes row t's du; past the sequence dpre is zero
#pragma unroll 4
        for (; t < end + 3; ++t) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) d[3][i] = 0.0f;
            if (t < p.end) {
                float g[kVec];
                load_row<kIn, kVec>(u[3], f.u, f.ldu, t, c);
                load_row<kOut, kVec>(g, a.dout, a.ldd, t, c);
                const float own = t < end ? 1.0f : 0.0f;  // (the rows behind belong to the next run's sums)
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float pre = taps.pre(i, u[0][i], u[1][i], u[2][i], u[3][i]), sig = sigmoid(pre);
                    d[3][i] = g[i] * (sig * fmaf(pre, 1.0f - sig, 1.0f));
                    const float mine = own * d[3][i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) dw[j][i] = fmaf(mine, u[j][i], dw[j][i]);
                    db[i] += mine;
#pragma unroll
                    for (int j = 0; j < 3; ++j) u[j][i] = u[j + 1][i];
                }
            }
            const int row = t - 3;
            if (row >= first) {
                float g[kVec];
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    g[i] = fmaf(taps.w[3][i], d[0][i],
                                fmaf(taps.w[2][i], d[1][i], fmaf(taps.w[1][i], d[2][i], taps.w[0][i] * d[3][i])));
                    if (a.dwout && row >= p.end - 4)
                        g[i] += a.dwout[((int64_t)s * f.ch + c + i) * 4 + (row - p.end + 4)];
                }
                store_row<kIn, kVec>(g, a.du, a.lddu, row, c);
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i)
#pragma unroll
                for (int j = 0; j < 3; ++j) d[j][i] = d[j + 1][i];
        }
        t = end;
    }
    if (!a.part) return;
    float* const part = a.part + (int64_t)run * 5 * f.ch + c;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) part[(int64_t)j * f.ch + i] = dw[j][i];
        part[(int64_t)4 * f.ch + i] = db[i];
    }
}

// dw and db: the runs' sums, each of 16 waves a sixteenth of the runs in order, then the waves in order.
__global__ __launch_bounds__(1024) void conv_grad_join_kernel(const float* __restrict__ part, int runs, int ch,
                                                              float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = (int64_t)5 * ch, i = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (i < n) {
        const int from = (int)((int64_t)runs * wave / 16), to = (int)((int64_t)runs * (wave + 1) / 16);
#pragma unroll 8
        for (int r = from; r < to; ++r) s += part[r * n + i];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || i >= n) return;
    s = sums[0][lane];
#pragma unroll
    for (int k = 1; k < 16; ++k) s += sums[k][lane];
    const int64_t j = i / ch, c = i - j * ch;
    if (j < 4) dw[c * 4 + j] = s;
    else db[c] = s;
}

bool vectors(const void* p, int64_t ld, bool bf16) {
    const uintptr_t bytes = bf16 ? 8 : 16;
    return (uintptr_t)p % bytes == 0 && ld % 4 == 0;
}

template <class F>
hipError_t with_types(bool in, bool out, bool vec, F f) {
    using True = std::true_type;
    using False = std::false_type;
    auto wide = [&](auto i, auto o) { return vec ? f(i, o, std::integral_constant<int, 4>()) : f(i, o, std::integral_constant<int, 1>()); };
    if (in) return out ? wide(True(), True()) : wide(True(), False());
    return out ? wide(False(), True()) : wide(False(), False());
}

// Workgroups: columns of 64 kVec channels, then runs in fours, then (if wanted) some for the windows.
dim3 conv_grid(const ConvArgs& a, int vec, bool windows) {
    const int groups = (a.runs + kWaves - 1) / kWaves;
    return dim3((unsigned)((a.ch + 64 * vec - 1) / (64 * vec)),
                (unsigned)(groups + (windows ? (a.seq.S < 1024 ? a.seq.S : 1024) : 0)));
}

}  // namespace

int64_t mamba2_conv_max_tokens() { return (int64_t)1 << 20; }

hipError_t launch_mamba2_conv(const Sequences& seq, const void* u, int64_t ldu, bool bf16_in, int ch, const float* w,
                              const float* b, const float* win, float* wout, void* out, int64_t ldo, bool bf16_out,
                              hipStream_t stream) {
    const ConvArgs a{seq, u, ldu, ch, (seq.T + kRun - 1) / kRun, w, b, win, wout, out, ldo};
    const bool vec = ch % 4 == 0 && vectors(u, ldu, bf16_in) && vectors(out, ldo, bf16_out);
    return with_types(bf16_in, bf16_out, vec, [&](auto in, auto o, auto v) {
        conv_kernel<in.value, o.value, v.value><<<conv_grid(a, v.value, wout != nullptr), kWaves * 64, 0, stream>>>(a);
        return hipGetLastError();
    });
}

size_t mamba2_conv_backward_workspace_bytes(int64_t T, int64_t ch) {
    return (size_t)((T + kGradRun - 1) / kGradRun * 5 * ch * 4);
}

hipError_t launch_mamba2_conv_backward(const Sequences& seq, const void* u, int64_t ldu, bool bf16_in, int ch, const float* w,
                                       const float* b, const float* win, const void* dout, int64_t ldd, bool bf16_out,
                                       const float* dwout, void* du, int64_t lddu, float* dw, float* db, float* dwin,
                                       void* workspace, hipStream_t stream) {
    ConvGradArgs a{{seq, u, ldu, ch, (seq.T + kGradRun - 1) / kGradRun, w, b, win, nullptr, nullptr, 0},
                   dout, ldd, dwout, du, lddu, dw ? static_cast<float*>(workspace) : nullptr, dwin};
    const bool vec = ch % 4 == 0 && vectors(u, ldu, bf16_in) && vectors(du, lddu, bf16_in) && vectors(dout, ldd, bf16_out);
    const hipError_t err = with_types(bf16_in, bf16_out, vec, [&](auto in, auto o, auto v) {
        conv_grad_kernel<in.value, o.value, v.value><<<conv_grid(a.f, v.value, dwin != nullptr), kWaves * 64, 0, stream>>>(a);
        return hipGetLastError();
    });
    if (err != hipSuccess || !dw) return err;
    conv_grad_join_kernel<<<dim3((unsigned)((5 * (int64_t)ch + 63) / 64)), 1024, 0, stream>>>(a.part, a.f.runs, ch, dw, db);
    return hipGetLastError();
}

}  // namespace dfssm
