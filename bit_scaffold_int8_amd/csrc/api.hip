// api.hip -- the C ABI (include/dfssm.h): host-side validation and kernel dispatch.
//
// Every entry point validates its arguments before enqueuing anything, launches on
// the caller's stream, never synchronizes and allocates nothing.
#include "dfssm.h"

#include <hip/hip_runtime.h>
#include <stdlib.h>

#include <initializer_list>

#include "scan.h"

namespace dfssm {
hipError_t launch_quantize_act(const float* x, int64_t M, int64_t K, int8_t* x_q, float* s_x,
                               hipStream_t stream);
int quantize_lora_tokens_per_group(int64_t K);
hipError_t launch_quantize_lora_down(const float* x, int64_t M, int64_t K, const int8_t* w_b, int rank,
                                     int8_t* x_q, float* s_x, int32_t* t, int64_t batch, hipStream_t stream);
hipError_t launch_lora_down(const int8_t* x_q, int64_t M, int64_t K, const int8_t* w_b, int32_t* t,
                            int64_t batch, hipStream_t stream);
hipError_t launch_gemv(const int8_t* x_q, const float* s_x, int M, int64_t N, int64_t K,
                       const uint8_t* w_bits, const float* s_w, const int8_t* w_a, const float* s_a,
                       const int8_t* w_b, const float* s_b, const int32_t* t, int32_t* t_out, int rank, float* y,
                       int32_t* acc_dbg, int64_t batch, hipStream_t stream);
hipError_t launch_gemm_mfma(const int8_t* x_q, const float* s_x, int64_t M, int64_t N, int64_t K,
                            const uint8_t* w_bits, const float* s_w, const int8_t* w_a, const float* s_a,
                            const int8_t* w_b, const float* s_b, const int32_t* t, int32_t* t_out, int rank,
                            float* y, int32_t* acc_dbg, int64_t batch, hipStream_t stream);
bool decode_fused_supported(int64_t M, int64_t K);
hipError_t launch_decode_fused(const float* x, int M, int64_t N, int64_t K, const uint8_t* w_bits,
                               const float* s_w, const int8_t* w_a, const float* s_a, const int8_t* w_b,
                               const float* s_b, int rank, int8_t* x_q, float* s_x, int32_t* t, float* y,
                               int32_t* acc_dbg, int64_t batch, hipStream_t stream);
bool int8_head_supported(int64_t M, int64_t K);
hipError_t launch_int8_head(const int8_t* x_q, const float* s_x, int M, int64_t N, int64_t K, const int8_t* e,
                            const float* s_e, float* y, int32_t* acc_dbg, int64_t batch, hipStream_t stream);
hipError_t launch_embedding_lookup(const int32_t* tokens, int64_t T, const int8_t* e, const float* s_e, int64_t V,
                                   int64_t K, float* out, hipStream_t stream);
bool mamba2_step_supported(int64_t nheads, int64_t headdim, int64_t d_state);
hipError_t launch_mamba2_step(const float* zxbcdt, int64_t S, int nheads, const float* conv_in, float* conv_out,
                              float* ssm_state, const float* conv_w, const float* conv_b, const float* dt_bias,
                              const float* A_log, const float* D, const float* norm_w, float eps, float* out,
                              hipStream_t stream);
bool density_field_supported(int64_t d_state);
hipError_t launch_density_encode(const float* state, int64_t R, int64_t D, uint32_t* field, float* scale,
                                 float* state_out, hipStream_t stream);
hipError_t launch_density_decode(const uint32_t* field, const float* scale, int64_t R, int64_t D, float* state,
                                 hipStream_t stream);
size_t decode_layers_workspace_bytes();
uint32_t* decode_layers_scratch(hipStream_t stream);
int64_t decode_layers_trace_words();
int64_t decode_layers_max_layers();
bool prefill_supported(int64_t M, int64_t N, int64_t K);
int prefill_num_cfgs();
void prefill_plan_query(int64_t M, int64_t N, int64_t K, int64_t batch, int* main_cfg, int* tail_cfg,
                        int64_t* n_split);
hipError_t launch_gemm_prefill(const int8_t* x_q, const float* s_x, int64_t M, int64_t N, int64_t K,
                               const uint8_t* w_bits, const float* s_w, const int8_t* w_a, const float* s_a,
                               const int8_t* w_b, const float* s_b, const int32_t* t, int32_t* t_out, int rank,
                               float* y, int32_t* acc_dbg, int64_t batch, int force_cfg, int force_tail,
                               hipStream_t stream);
hipError_t launch_int8_gemm(const int8_t* x_q, int64_t ldx, const float* s_x, int64_t M, int64_t N, int64_t K,
                            const int8_t* w, int64_t ldw, const float* s_w, void* y, int64_t ldy, bool bf16,
                            hipStream_t stream);
size_t cross_entropy_workspace_bytes(int64_t M, int64_t V, int64_t K);
hipError_t launch_cross_entropy(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K, const int8_t* e,
                                const float* s_e, const int32_t* targets, float* loss, float* lse, void* workspace,
                                hipStream_t stream);
size_t cross_entropy_backward_workspace_bytes(int64_t M, int64_t V, int64_t K, bool bf16, bool want_dx, bool want_de);
hipError_t launch_cross_entropy_backward(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K,
                                         const int8_t* e, const float* s_e, const int32_t* targets, const float* lse,
                                         const float* dloss, void* dx, void* de, bool bf16, bool accumulate,
                                         void* workspace, hipStream_t stream);
hipError_t launch_embedding_lookup_scaled(const int32_t* tokens, int64_t T, const int8_t* e, const float* s_e,
                                          int64_t V, int64_t K, float scale, void* out, int64_t ldo, bool bf16,
                                          hipStream_t stream);
size_t embedding_backward_workspace_bytes(int64_t T, int64_t V, int64_t K);
hipError_t launch_embedding_backward(const int32_t* tokens, int64_t T, const void* dout, int64_t ldd, bool dout_bf16,
                                     int64_t V, int64_t K, float scale, void* de, bool de_bf16, bool accumulate,
                                     void* workspace, hipStream_t stream);
hipError_t launch_mamba2_conv(const Sequences& seq, const void* u, int64_t ldu, bool bf16_in, int ch, const float* w,
                              const float* b, const float* win, float* wout, void* out, int64_t ldo, bool bf16_out,
                              hipStream_t stream);
size_t mamba2_conv_backward_workspace_bytes(int64_t T, int64_t ch);
hipError_t launch_mamba2_conv_backward(const Sequences& seq, const void* u, int64_t ldu, bool bf16_in, int ch, const float* w,
                                       const float* b, const float* win, const void* dout, int64_t ldd, bool bf16_out,
                                       const float* dwout, void* du, int64_t lddu, float* dw, float* db, float* dwin,
                                       void* workspace, hipStream_t stream);
size_t mamba2_scan_workspace_bytes(int64_t T, int64_t S, int64_t H, int64_t N, int64_t G);
hipError_t launch_mamba2_scan(ScanArgs a, bool bf16, int N, const float* state_in, float* state_out, void* y, int64_t ldy,
                              void* workspace, hipStream_t stream);
int64_t distillation_max_top();
size_t distillation_workspace_bytes(int64_t M, int64_t V, int64_t K);
hipError_t launch_distillation(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K, const int8_t* e,
                               const float* s_e, const int32_t* ids, const float* top, int64_t k, float temperature,
                               float* loss, float* lse, float* logp, void* workspace, hipStream_t stream);
size_t distillation_backward_workspace_bytes(int64_t M, int64_t V, int64_t K, int64_t k, bool bf16, bool want_dx, bool want_de);
hipError_t launch_distillation_backward(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K,
                                        const int8_t* e, const float* s_e, const int32_t* ids, const float* top, int64_t k,
                                        float temperature, const float* lse, const float* logp, const float* dloss,
                                        void* dx, void* de, bool bf16, bool accumulate, void* workspace,
                                        hipStream_t stream);
size_t mamba2_scan_backward_workspace_bytes(int64_t T, int64_t S, int64_t H, int64_t N, int64_t G);
hipError_t launch_mamba2_scan_backward(ScanArgs a, bool bf16, int N, const float* state_in, const void* dy, int64_t lddy,
                                       const float* dstate_out, void* dx, int64_t lddx, float* ddt, int64_t ldddt, void* dB,
                                       int64_t lddb, void* dC, int64_t lddc, float* dA_log, float* dD, float* ddt_bias,
                                       float* dstate_in, void* workspace, hipStream_t stream);
}  // namespace dfssm

#include "decode_args.h"

namespace {

constexpr int64_t kMaxDecodeM = 16;
constexpr int64_t kGemvMaxK = 8 * 4 * 4 * 128;  // decode kernel: 8 waves x 4 lane groups x 4 chunks x 128 k
// |t| <= 127 * 127 * K must fit int32 (and |acc| <= 127 * K with it)
constexpr int64_t kMaxK = 131072;
constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxBatch = 65535;  // problems ride gridDim.y
constexpr int64_t kRankBytes = 16;     // one row of W_A (int8, rank 16)

// Operands read with 16-byte vector loads (x, x_q, w_bits, w_a, w_b) must be 16-byte
// aligned; scale vectors, t, y and acc_dbg only need their element alignment.
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool aligned4_or_null(const void* p) { return p == nullptr || aligned4(p); }

dfssm_status check_rank(int32_t rank) {
    return (rank == 0 || rank == 16) ? DFSSM_OK : DFSSM_ERR_UNSUPPORTED;
}

dfssm_status check_sizes(int64_t M, int64_t K, int64_t batch) {
    if (M <= 0 || K <= 0 || batch <= 0 || M >= kMaxRows) return DFSSM_ERR_INVALID_ARG;
    if (batch > kMaxBatch) return DFSSM_ERR_UNSUPPORTED;
    return DFSSM_OK;
}

dfssm_status lora_down_impl(const int8_t* x_q, int64_t M, int64_t K, const int8_t* w_b, int32_t rank, int32_t* t,
                            int64_t batch, hipStream_t stream) {
    if (!x_q || !w_b || !t) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = check_sizes(M, K, batch)) return st;
    if (!aligned16(x_q) || !aligned16(w_b) || !aligned4(t)) return DFSSM_ERR_INVALID_ARG;
    if (rank != 16) return DFSSM_ERR_UNSUPPORTED;
    if (K > kMaxK) return DFSSM_ERR_UNSUPPORTED;
    return dfssm::launch_lora_down(x_q, M, K, w_b, t, batch, stream) == hipSuccess ? DFSSM_OK : DFSSM_ERR_HIP;
}

dfssm_status quantize_lora_down_impl(const float* x, int64_t M, int64_t K, const int8_t* w_b, int32_t rank,
                                     int8_t* x_q, float* s_x, int32_t* t, int64_t batch, hipStream_t stream) {
    if (!x || !x_q || !s_x) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = check_sizes(M, K, batch)) return st;
    if (!aligned16(x) || !aligned16(x_q) || !aligned4(s_x)) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = check_rank(rank)) return st;
    if (rank == 16) {
        if (!w_b || !t) return DFSSM_ERR_INVALID_ARG;
        if (!aligned16(w_b) || !aligned4(t)) return DFSSM_ERR_INVALID_ARG;
        if (K > kMaxK) return DFSSM_ERR_UNSUPPORTED;
    }
    if (M * batch >= kMaxRows) return DFSSM_ERR_INVALID_ARG;
    hipError_t e;
    if (K % 4 == 0 && dfssm::quantize_lora_tokens_per_group(K) > 0) {
        e = dfssm::launch_quantize_lora_down(x, M, K, w_b, rank, x_q, s_x, t, batch, stream);
    } else {
        // rows not 16-byte aligned, or longer than the fused kernel's LDS holds: two kernels
        e = dfssm::launch_quantize_act(x, M * batch, K, x_q, s_x, stream);
        if (e == hipSuccess && rank == 16) e = dfssm::launch_lora_down(x_q, M, K, w_b, t, batch, stream);
    }
    return e == hipSuccess ? DFSSM_OK : DFSSM_ERR_HIP;
}

// The scaffold product with the scale + LoRA-up epilogue.  Exactly one of t (given,
// from a LoRA-down call) and w_b (t = W_B x_q computed by the kernel; t_out, when not
// NULL, receives it) is used at rank 16.
dfssm_status gemm_impl(const int8_t* x_q, const float* s_x, int64_t M, int64_t N, int64_t K,
                       const uint8_t* w_bits, const float* s_w, const int8_t* w_a, const float* s_a,
                       const int8_t* w_b, const float* s_b, const int32_t* t, int32_t* t_out, int32_t rank, float* y,
                       int32_t* acc_dbg, int64_t batch, hipStream_t stream) {
    if (!x_q || !s_x || !w_bits || !s_w || !y) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = check_sizes(M, K, batch)) return st;
    if (N <= 0 || N >= kMaxRows || (K % 8) != 0) return DFSSM_ERR_INVALID_ARG;
    if (!aligned16(x_q) || !aligned4(s_x) || !aligned16(w_bits) || !aligned4(s_w) || !aligned4(y) ||
        !aligned4_or_null(acc_dbg) || !aligned4_or_null(t_out))
        return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = check_rank(rank)) return st;
    if (rank == 16) {
        if (!w_a || !s_a || !s_b || (!t && !w_b)) return DFSSM_ERR_INVALID_ARG;
        if (!aligned16(w_a) || !aligned4(s_a) || !aligned4(s_b)) return DFSSM_ERR_INVALID_ARG;
        if ((t && !aligned4(t)) || (w_b && !aligned16(w_b))) return DFSSM_ERR_INVALID_ARG;
    }
    if (K > kMaxK) return DFSSM_ERR_UNSUPPORTED;
    if (rank == 0) {
        w_b = nullptr;
        t = nullptr;
        t_out = nullptr;
    } else if (t) {
        w_b = nullptr;  // the given-t form
        t_out = nullptr;
    }
    hipError_t e;
    // the decode kernel addresses one problem's signs, LoRA rows and outputs with 32-bit
    // offsets
    const bool gemv_fits = N * (K / 8) < ((int64_t)1 << 31) && M * N * 4 < ((int64_t)1 << 31) &&
                           N * kRankBytes < ((int64_t)1 << 31);
    if (M <= kMaxDecodeM && K <= kGemvMaxK && gemv_fits) {
        e = dfssm::launch_gemv(x_q, s_x, (int)M, N, K, w_bits, s_w, w_a, s_a, w_b, s_b, t, t_out, rank, y, acc_dbg,
                               batch, stream);
    } else {
        // DFSSM_PREFILL_CFG pins the many-token kernel's tile configuration (0 ..
        // prefill_num_cfgs() - 1) or, with -2, the generic fallback kernel; unset or -1
        // lets the cost model choose.  DFSSM_PREFILL_TAIL adds a narrower configuration
        // for the columns past the pinned one's main part, where the pinned one is built
        // with that tail.  Testing and tuning knobs.
        int force = -1, force_tail = -1;
        if (const char* f = getenv("DFSSM_PREFILL_CFG")) force = atoi(f);
        if (const char* f = getenv("DFSSM_PREFILL_TAIL")) force_tail = atoi(f);
        const bool prefill = force != -2 && dfssm::prefill_supported(M, N, K) && aligned16(w_bits) &&
                             (rank == 0 || aligned16(w_a));
        if (prefill) {
            e = dfssm::launch_gemm_prefill(x_q, s_x, M, N, K, w_bits, s_w, w_a, s_a, w_b, s_b, t, t_out, rank, y,
                                           acc_dbg, batch, force, force_tail, stream);
        } else {
            e = dfssm::launch_gemm_mfma(x_q, s_x, M, N, K, w_bits, s_w, w_a, s_a, w_b, s_b, t, t_out, rank, y,
                                        acc_dbg, batch, stream);
        }
    }
    return e == hipSuccess ? DFSSM_OK : DFSSM_ERR_HIP;
}

dfssm_status forward_impl(const float* x, int64_t M, int64_t N, int64_t K, const uint8_t* w_bits,
                          const float* s_w, const int8_t* w_a, const float* s_a, const int8_t* w_b,
                          const float* s_b, int32_t rank, int8_t* x_q, float* s_x, int32_t* t, float* y,
                          int32_t* acc_dbg, int64_t batch, hipStream_t stream) {
    // the two calls' checks, in full, before anything is launched
    if (!x || !x_q || !s_x || !w_bits || !s_w || !y) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = check_sizes(M, K, batch)) return st;
    if (N <= 0 || N >= kMaxRows || (K % 8) != 0) return DFSSM_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(x_q) || !aligned4(s_x) || !aligned16(w_bits) || !aligned4(s_w) ||
        !aligned4(y) || !aligned4_or_null(acc_dbg))
        return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = check_rank(rank)) return st;
    if (rank == 16) {
        if (!w_a || !s_a || !w_b || !s_b || !t) return DFSSM_ERR_INVALID_ARG;
        if (!aligned16(w_a) || !aligned4(s_a) || !aligned16(w_b) || !aligned4(s_b) || !aligned4(t))
            return DFSSM_ERR_INVALID_ARG;
    }
    if (K > kMaxK) return DFSSM_ERR_UNSUPPORTED;
    if (M * batch >= kMaxRows) return DFSSM_ERR_INVALID_ARG;
    const bool gemv_fits = N * (K / 8) < ((int64_t)1 << 31) && M * N * 4 < ((int64_t)1 << 31) &&
                           N * kRankBytes < ((int64_t)1 << 31);
    if (gemv_fits && dfssm::decode_fused_supported(M, K)) {
        const hipError_t e = dfssm::launch_decode_fused(x, (int)M, N, K, w_bits, s_w, w_a, s_a, w_b, s_b, rank, x_q,
                                                        s_x, t, y, acc_dbg, batch, stream);
        if (e != hipErrorNotSupported) return e == hipSuccess ? DFSSM_OK : DFSSM_ERR_HIP;
        // the launch plan has several groups per problem at a throughput batch: two kernels
    }
    // Many-token projections with under 2^24 outputs per launch: the plain quantizer, then
    // the MFMA kernel computing t from the code chunks it already stages (its first column
    // tile writes t out).  Against quantize + LoRA-down followed by the product given t it
    // measured 1.2-2 us faster from 17 to 2048 tokens for N = 2048, K = 4096, and level or
    // up to 2.9 us faster from 17 to 1536 tokens for N = 8512, K = 2048.  At 2048 tokens of
    // the latter (2^24 outputs and more) the product is MFMA-bound and the W_B chunks every
    // column tile recomputes cost more than the separate LoRA-down pass (1.1 us slower).
    // The bytes written are the same either way.
    const bool decode_kernel = M <= kMaxDecodeM && K <= kGemvMaxK && gemv_fits;
    if (rank == 16 && !decode_kernel && M * N * batch < ((int64_t)1 << 24) && dfssm::prefill_supported(M, N, K)) {
        if (dfssm::launch_quantize_act(x, M * batch, K, x_q, s_x, stream) != hipSuccess) return DFSSM_ERR_HIP;
        return gemm_impl(x_q, s_x, M, N, K, w_bits, s_w, w_a, s_a, w_b, s_b, nullptr, t, rank, y, acc_dbg, batch,
                         stream);
    }
    if (dfssm_status st = quantize_lora_down_impl(x, M, K, w_b, rank, x_q, s_x, t, batch, stream)) return st;
    return gemm_impl(x_q, s_x, M, N, K, w_bits, s_w, w_a, s_a, nullptr, s_b, t, nullptr, rank, y, acc_dbg, batch,
                     stream);
}

dfssm_status int8_head_impl(const int8_t* x_q, const float* s_x, int64_t M, int64_t N, int64_t K, const int8_t* e,
                           const float* s_e, float* y, int32_t* acc_dbg, int64_t batch, hipStream_t stream) {
    if (!x_q || !s_x || !e || !s_e || !y) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = check_sizes(M, K, batch)) return st;
    if (N <= 0 || N >= kMaxRows || (K % 16) != 0) return DFSSM_ERR_INVALID_ARG;
    if (!aligned16(x_q) || !aligned4(s_x) || !aligned16(e) || !aligned4(s_e) || !aligned4(y) ||
        !aligned4_or_null(acc_dbg))
        return DFSSM_ERR_INVALID_ARG;
    // one problem's matrix and outputs are addressed with 32-bit offsets (plus one
    // stage of rows past N)
    if ((N + 128) * K >= ((int64_t)1 << 31) || M * N * 4 >= ((int64_t)1 << 31)) return DFSSM_ERR_UNSUPPORTED;
    if (!dfssm::int8_head_supported(M, K)) return DFSSM_ERR_UNSUPPORTED;
    return dfssm::launch_int8_head(x_q, s_x, (int)M, N, K, e, s_e, y, acc_dbg, batch, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

dfssm_status decode_layers_impl(const dfssm_decode_layer_weights* w, int64_t n_layers, const float* x_in,
                                float* x_out, const float* conv_in, float* conv_out, float* ssm_state, float eps,
                                void* workspace, size_t workspace_bytes, int32_t* status, uint32_t* trace,
                                int64_t spin_limit, uint32_t flags, hipStream_t stream, bool validate_only = false) {
    if (!w || !x_in || !x_out || !conv_in || !conv_out || !ssm_state || !workspace || !status)
        return DFSSM_ERR_INVALID_ARG;
    if (!w->in_w_bits || !w->in_s_w || !w->in_w_a || !w->in_s_a || !w->in_w_b || !w->in_s_b || !w->conv_w ||
        !w->conv_b || !w->dt_bias || !w->A_log || !w->D || !w->norm_w || !w->out_w_bits || !w->out_s_w ||
        !w->out_w_a || !w->out_s_a || !w->out_w_b || !w->out_s_b)
        return DFSSM_ERR_INVALID_ARG;
    if (n_layers < 1 || n_layers > dfssm::decode_layers_max_layers()) return DFSSM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || eps > 1e30f) return DFSSM_ERR_INVALID_ARG;
    if (workspace_bytes < dfssm::decode_layers_workspace_bytes()) return DFSSM_ERR_INVALID_ARG;
    if (flags & ~DFSSM_DECODE_UNREACHABLE_WAITS) return DFSSM_ERR_INVALID_ARG;
    if (!aligned16(w->in_w_bits) || !aligned16(w->in_w_a) || !aligned16(w->in_w_b) || !aligned16(w->conv_w) ||
        !aligned16(w->norm_w) || !aligned16(w->out_w_bits) || !aligned16(w->out_w_a) || !aligned16(w->out_w_b) ||
        !aligned4(w->in_s_w) || !aligned4(w->in_s_a) || !aligned4(w->in_s_b) || !aligned4(w->conv_b) ||
        !aligned4(w->dt_bias) || !aligned4(w->A_log) || !aligned4(w->D) || !aligned4(w->out_s_w) ||
        !aligned4(w->out_s_a) || !aligned4(w->out_s_b) || !aligned16(x_in) || !aligned4(x_out) ||
        !aligned16(conv_in) || !aligned16(conv_out) || !aligned16(ssm_state) || !aligned16(workspace) ||
        !aligned4(status) || !aligned4_or_null(trace))
        return DFSSM_ERR_INVALID_ARG;
    const int64_t conv_bytes = n_layers * 4352 * 16;
    const uintptr_t ci = (uintptr_t)conv_in, co = (uintptr_t)conv_out;
    if (ci < co + (uintptr_t)conv_bytes && co < ci + (uintptr_t)conv_bytes) return DFSSM_ERR_INVALID_ARG;
    if (validate_only) return DFSSM_OK;
    const dfssm::decode::Args a{w->in_w_bits, w->in_s_w, w->in_w_a, w->in_s_a, w->in_w_b, w->in_s_b,
                                w->conv_w, w->conv_b, w->dt_bias, w->A_log, w->D, w->norm_w,
                                w->out_w_bits, w->out_s_w, w->out_w_a, w->out_s_a, w->out_w_b, w->out_s_b,
                                conv_in, conv_out, ssm_state, x_in, x_out, trace,
                                static_cast<uint32_t*>(workspace), status, (int)n_layers, eps,
                                spin_limit > 0 ? spin_limit : ((int64_t)1 << 22),
                                (flags & DFSSM_DECODE_UNREACHABLE_WAITS) ? (1u << 30) : 0u};
    const hipError_t e = dfssm::launch_decode_layers(a, stream);
    if (e == hipErrorNotSupported) return DFSSM_ERR_UNSUPPORTED;
    return e == hipSuccess ? DFSSM_OK : DFSSM_ERR_HIP;
}

// ---- the operators over an int8 matrix with fp32 or bf16 results
constexpr int64_t kMaxStride = (int64_t)1 << 22;     // row strides of the int8 operands: a tile's 256 rows stay below 2^30
constexpr int64_t kMaxBlocks = (int64_t)1 << 30;       // 32 x 32 blocks of one product's output
// (a launch holds fewer than 2^32 threads)
constexpr int64_t kMaxLossTokens = (int64_t)1 << 25, kMaxLossRows = (int64_t)1 << 28;  // of one forward call
constexpr int64_t kMaxLossLogits = (int64_t)1 << 38;
constexpr int64_t kMaxTeacherEntries = (int64_t)1 << 28;  // (eight of them take a wave)
constexpr int64_t kMaxLossGradTokens = (int64_t)1 << 18;  // of one backward call
constexpr int64_t kMaxGradTokens = (int64_t)1 << 24, kMaxGradRows = (int64_t)1 << 28;  // of one embedding gradient

bool type_ok(int32_t t) { return t == DFSSM_F32 || t == DFSSM_BF16; }
bool aligned_type(const void* p, int32_t t) { return ((uintptr_t)p & (t == DFSSM_BF16 ? 1u : 3u)) == 0; }

// Sizes of the cross entropy over [V][K] for M tokens.
dfssm_status loss_sizes(int64_t M, int64_t V, int64_t K) {
    if (M <= 0 || V <= 0 || K <= 0 || M >= kMaxRows || V >= kMaxRows || K % 16 != 0) return DFSSM_ERR_INVALID_ARG;
    if (K > kMaxK || M > kMaxLossTokens || V > kMaxLossRows || M * V > kMaxLossLogits) return DFSSM_ERR_UNSUPPORTED;
    return DFSSM_OK;
}

dfssm_status distillation_sizes(int64_t M, int64_t V, int64_t K, int64_t top) {
    if (top <= 0) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = loss_sizes(M, V, K)) return st;
    return top > dfssm::distillation_max_top() || M * top > kMaxTeacherEntries ? DFSSM_ERR_UNSUPPORTED : DFSSM_OK;
}

bool temperature_ok(float t) { return t >= 0x1p-60f && t <= 0x1p60f; }

dfssm_status embedding_sizes(int64_t T, int64_t V, int64_t K) {
    if (T <= 0 || V <= 0 || K <= 0 || T >= kMaxRows || V >= kMaxRows) return DFSSM_ERR_INVALID_ARG;
    if (K > kMaxK) return DFSSM_ERR_UNSUPPORTED;
    return DFSSM_OK;
}

dfssm_status density_checks(int64_t rows, int64_t d_state) {
    if (rows <= 0 || d_state <= 0) return DFSSM_ERR_INVALID_ARG;
    if (!dfssm::density_field_supported(d_state)) return DFSSM_ERR_UNSUPPORTED;
    if (rows >= ((int64_t)1 << 40) / d_state) return DFSSM_ERR_INVALID_ARG;
    return DFSSM_OK;
}

// ---- packed sequences
constexpr int64_t kMaxTokens = (int64_t)1 << 20, kMaxChannels = (int64_t)1 << 18, kMaxLd = (int64_t)1 << 31;

bool overlapping(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

dfssm_status sequence_sizes(int64_t T, int64_t S, bool offsets) {
    if (T <= 0 || S <= 0 || T >= kMaxRows || S >= kMaxRows || (!offsets && T % S != 0)) return DFSSM_ERR_INVALID_ARG;
    if (T > kMaxTokens || S > kMaxBatch) return DFSSM_ERR_UNSUPPORTED;
    return DFSSM_OK;
}

dfssm_status conv_sizes(int64_t T, int64_t S, int64_t ch, bool offsets) {
    if (ch <= 0 || ch >= kMaxRows) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = sequence_sizes(T, S, offsets)) return st;
    return ch > kMaxChannels || T * ch > ((int64_t)1 << 34) ? DFSSM_ERR_UNSUPPORTED : DFSSM_OK;
}

// A matrix's stride: what is shorter than a row is wrong, 2^31 and more is refused.
dfssm_status stride_ok(int64_t ld, int64_t row) {
    return ld < row ? DFSSM_ERR_INVALID_ARG : ld >= kMaxLd ? DFSSM_ERR_UNSUPPORTED : DFSSM_OK;
}

dfssm::Sequences sequences(const int32_t* cu, int64_t T, int64_t S) { return {cu, (int)T, (int)S, (int)(T / S)}; }

dfssm_status scan_sizes(int64_t T, int64_t S, int64_t H, int64_t P, int64_t N, int64_t G, bool offsets) {
    if (H <= 0 || P <= 0 || N <= 0 || G <= 0 || H >= kMaxRows || P >= kMaxRows || N >= kMaxRows || H % G != 0)
        return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = sequence_sizes(T, S, offsets)) return st;
    if (P != dfssm::kP || (N != 64 && N != 128) || H > 1024 || S * H > ((int64_t)1 << 21) ||
        (T / dfssm::kChunk + S) * (H + 4 * G) > ((int64_t)1 << 25) ||
        (T / dfssm::kChunk + S) * G > ((int64_t)1 << 21))    // (1024 threads and more a chunk and group: below 2^32 in a launch)
        return DFSSM_ERR_UNSUPPORTED;
    return DFSSM_OK;
}

// Rows that are read in pieces of 16 bytes; 64 of them stay below 2^31 bytes.
dfssm_status wide_rows(const void* p, int64_t ld, int64_t row, int32_t type) {
    if (!aligned16(p) || ld % (type == DFSSM_BF16 ? 8 : 4) != 0 || ld < row) return DFSSM_ERR_INVALID_ARG;
    return ld > kMaxStride ? DFSSM_ERR_UNSUPPORTED : DFSSM_OK;
}

dfssm_status scan_operands(const dfssm_mamba2_scan_operands* op, dfssm::ScanArgs& a) {
    if (!op || !op->x || !op->B || !op->C || !op->dt || !op->A_log || !op->D || !op->dt_bias) return DFSSM_ERR_INVALID_ARG;
    if (!type_ok(op->type)) return DFSSM_ERR_INVALID_ARG;
    const int64_t bc = op->ngroups * op->d_state;
    const bool sized = op->nheads > 0 && op->nheads < kMaxRows && op->ngroups > 0 && op->ngroups < kMaxRows && op->d_state > 0 &&
                       op->d_state < kMaxRows;
    if (!sized) return DFSSM_ERR_INVALID_ARG;
    if (!aligned16(op->state_in) || !aligned4(op->dt) || !aligned4(op->A_log) || !aligned4(op->D) ||
        !aligned4(op->dt_bias) || !aligned4(op->cu_seqlens))
        return DFSSM_ERR_INVALID_ARG;
    // (what is wrong comes before what is not supported)
    dfssm_status worst = scan_sizes(op->T, op->S, op->nheads, op->headdim, op->d_state, op->ngroups, op->cu_seqlens != nullptr);
    for (dfssm_status st : {wide_rows(op->x, op->ldx, op->nheads * dfssm::kP, op->type), wide_rows(op->B, op->ldb, bc, op->type),
                            wide_rows(op->C, op->ldc, bc, op->type), stride_ok(op->lddt, op->nheads)})
        if (worst != DFSSM_ERR_INVALID_ARG && st != DFSSM_OK) worst = st;
    if (worst != DFSSM_OK) return worst;
    a = dfssm::ScanArgs{};
    a.seq = sequences(op->cu_seqlens, op->T, op->S);
    a.H = (int)op->nheads;
    a.G = (int)op->ngroups;
    a.x = op->x, a.B = op->B, a.C = op->C, a.dt = op->dt;
    a.ldx = op->ldx, a.lddt = op->lddt, a.ldb = op->ldb, a.ldc = op->ldc;
    a.A_log = op->A_log, a.D = op->D, a.dt_bias = op->dt_bias;
    return DFSSM_OK;
}

}  // namespace

extern "C" {

const char* dfssm_status_string(dfssm_status status) {
    switch (status) {
        case DFSSM_OK: return "DFSSM_OK";
        case DFSSM_ERR_INVALID_ARG: return "DFSSM_ERR_INVALID_ARG";
        case DFSSM_ERR_UNSUPPORTED: return "DFSSM_ERR_UNSUPPORTED";
        case DFSSM_ERR_HIP: return "DFSSM_ERR_HIP";
    }
    return "DFSSM_ERR_UNKNOWN";
}

int32_t dfssm_version(void) { return 402; }

dfssm_status dfssm_prefill_plan(int64_t M, int64_t N, int64_t K, int64_t batch, int32_t* main_cfg,
                                int32_t* tail_cfg, int64_t* n_split) {
    if (!main_cfg || !tail_cfg || !n_split) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = check_sizes(M, K, batch)) return st;
    if (N <= 0 || N >= kMaxRows || (K % 8) != 0) return DFSSM_ERR_INVALID_ARG;
    if (K > kMaxK) return DFSSM_ERR_UNSUPPORTED;
    // the same tests as dfssm_scaffold_lora_gemm[_strided_batched]: the decode kernel, or
    // the generic kernel, takes the shape
    const bool gemv_fits = N * (K / 8) < ((int64_t)1 << 31) && M * N * 4 < ((int64_t)1 << 31) &&
                           N * kRankBytes < ((int64_t)1 << 31);
    if (M <= kMaxDecodeM && K <= kGemvMaxK && gemv_fits) return DFSSM_ERR_UNSUPPORTED;
    if (!dfssm::prefill_supported(M, N, K)) return DFSSM_ERR_UNSUPPORTED;
    int mc = 0, tc = -1;
    int64_t ns = N;
    dfssm::prefill_plan_query(M, N, K, batch, &mc, &tc, &ns);
    *main_cfg = mc;
    *tail_cfg = tc;
    *n_split = ns;
    return DFSSM_OK;
}

dfssm_status dfssm_quantize_act(const float* x, int64_t M, int64_t K, int8_t* x_q, float* s_x,
                                hipStream_t stream) {
    if (!x || !x_q || !s_x) return DFSSM_ERR_INVALID_ARG;
    if (M <= 0 || K <= 0 || M >= kMaxRows) return DFSSM_ERR_INVALID_ARG;
    if (!aligned4(x) || !aligned4(s_x)) return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_quantize_act(x, M, K, x_q, s_x, stream) == hipSuccess ? DFSSM_OK : DFSSM_ERR_HIP;
}

dfssm_status dfssm_lora_down(const int8_t* x_q, int64_t M, int64_t K, const int8_t* w_b, int32_t rank, int32_t* t,
                             hipStream_t stream) {
    return lora_down_impl(x_q, M, K, w_b, rank, t, 1, stream);
}

dfssm_status dfssm_lora_down_strided_batched(const int8_t* x_q, int64_t M, int64_t K, const int8_t* w_b,
                                             int32_t rank, int32_t* t, int64_t batch, hipStream_t stream) {
    return lora_down_impl(x_q, M, K, w_b, rank, t, batch, stream);
}

dfssm_status dfssm_quantize_lora_down(const float* x, int64_t M, int64_t K, const int8_t* w_b, int32_t rank,
                                      int8_t* x_q, float* s_x, int32_t* t, hipStream_t stream) {
    return quantize_lora_down_impl(x, M, K, w_b, rank, x_q, s_x, t, 1, stream);
}

dfssm_status dfssm_quantize_lora_down_strided_batched(const float* x, int64_t M, int64_t K, const int8_t* w_b,
                                                      int32_t rank, int8_t* x_q, float* s_x, int32_t* t,
                                                      int64_t batch, hipStream_t stream) {
    return quantize_lora_down_impl(x, M, K, w_b, rank, x_q, s_x, t, batch, stream);
}

dfssm_status dfssm_scaffold_lora_gemm(const int8_t* x_q, const float* s_x, int64_t M, int64_t N, int64_t K,
                                      const uint8_t* w_bits, const float* s_w, const int8_t* w_a,
                                      const float* s_a, const int8_t* w_b, const float* s_b, int32_t rank,
                                      float* y, int32_t* acc_dbg, int32_t* t_dbg, hipStream_t stream) {
    if (rank != 0 && !w_b) return DFSSM_ERR_INVALID_ARG;
    return gemm_impl(x_q, s_x, M, N, K, w_bits, s_w, w_a, s_a, w_b, s_b, nullptr, t_dbg, rank, y, acc_dbg, 1,
                     stream);
}

dfssm_status dfssm_scaffold_lora_gemm_strided_batched(const int8_t* x_q, const float* s_x, int64_t M, int64_t N,
                                                      int64_t K, const uint8_t* w_bits, const float* s_w,
                                                      const int8_t* w_a, const float* s_a, const int8_t* w_b,
                                                      const float* s_b, int32_t rank, float* y, int32_t* acc_dbg,
                                                      int32_t* t_dbg, int64_t batch, hipStream_t stream) {
    if (rank != 0 && !w_b) return DFSSM_ERR_INVALID_ARG;
    return gemm_impl(x_q, s_x, M, N, K, w_bits, s_w, w_a, s_a, w_b, s_b, nullptr, t_dbg, rank, y, acc_dbg, batch,
                     stream);
}

dfssm_status dfssm_scaffold_lora_gemm_given_t(const int8_t* x_q, const float* s_x, int64_t M, int64_t N, int64_t K,
                                              const uint8_t* w_bits, const float* s_w, const int8_t* w_a,
                                              const float* s_a, const float* s_b, const int32_t* t, int32_t rank,
                                              float* y, int32_t* acc_dbg, hipStream_t stream) {
    if (rank != 0 && !t) return DFSSM_ERR_INVALID_ARG;
    return gemm_impl(x_q, s_x, M, N, K, w_bits, s_w, w_a, s_a, nullptr, s_b, t, nullptr, rank, y, acc_dbg, 1,
                     stream);
}

dfssm_status dfssm_scaffold_lora_gemm_given_t_strided_batched(const int8_t* x_q, const float* s_x, int64_t M,
                                                              int64_t N, int64_t K, const uint8_t* w_bits,
                                                              const float* s_w, const int8_t* w_a, const float* s_a,
                                                              const float* s_b, const int32_t* t, int32_t rank,
                                                              float* y, int32_t* acc_dbg, int64_t batch,
                                                              hipStream_t stream) {
    if (rank != 0 && !t) return DFSSM_ERR_INVALID_ARG;
    return gemm_impl(x_q, s_x, M, N, K, w_bits, s_w, w_a, s_a, nullptr, s_b, t, nullptr, rank, y, acc_dbg, batch,
                     stream);
}

dfssm_status dfssm_scaffold_lora_forward(const float* x, int64_t M, int64_t N, int64_t K, const uint8_t* w_bits,
                                         const float* s_w, const int8_t* w_a, const float* s_a, const int8_t* w_b,
                                         const float* s_b, int32_t rank, int8_t* x_q, float* s_x, int32_t* t,
                                         float* y, int32_t* acc_dbg, hipStream_t stream) {
    return forward_impl(x, M, N, K, w_bits, s_w, w_a, s_a, w_b, s_b, rank, x_q, s_x, t, y, acc_dbg, 1, stream);
}

dfssm_status dfssm_scaffold_lora_forward_strided_batched(const float* x, int64_t M, int64_t N, int64_t K,
                                                         const uint8_t* w_bits, const float* s_w, const int8_t* w_a,
                                                         const float* s_a, const int8_t* w_b, const float* s_b,
                                                         int32_t rank, int8_t* x_q, float* s_x, int32_t* t,
                                                         float* y, int32_t* acc_dbg, int64_t batch,
                                                         hipStream_t stream) {
    return forward_impl(x, M, N, K, w_bits, s_w, w_a, s_a, w_b, s_b, rank, x_q, s_x, t, y, acc_dbg, batch, stream);
}

dfssm_status dfssm_int8_rowscale_gemm(const int8_t* x_q, const float* s_x, int64_t M, int64_t N, int64_t K,
                                      const int8_t* e, const float* s_e, float* y, int32_t* acc_dbg,
                                      hipStream_t stream) {
    return int8_head_impl(x_q, s_x, M, N, K, e, s_e, y, acc_dbg, 1, stream);
}

dfssm_status dfssm_int8_rowscale_gemm_strided_batched(const int8_t* x_q, const float* s_x, int64_t M, int64_t N,
                                                      int64_t K, const int8_t* e, const float* s_e, float* y,
                                                      int32_t* acc_dbg, int64_t batch, hipStream_t stream) {
    return int8_head_impl(x_q, s_x, M, N, K, e, s_e, y, acc_dbg, batch, stream);
}

dfssm_status dfssm_embedding_lookup(const int32_t* tokens, int64_t T, const int8_t* e, const float* s_e, int64_t V,
                                    int64_t K, float* out, hipStream_t stream) {
    if (!tokens || !e || !s_e || !out) return DFSSM_ERR_INVALID_ARG;
    if (T <= 0 || V <= 0 || K <= 0 || T >= kMaxRows) return DFSSM_ERR_INVALID_ARG;
    if (!aligned4(tokens) || !aligned4(s_e) || !aligned4(out)) return DFSSM_ERR_INVALID_ARG;
    if (V * K >= ((int64_t)1 << 40) || T * K >= ((int64_t)1 << 40)) return DFSSM_ERR_UNSUPPORTED;
    return dfssm::launch_embedding_lookup(tokens, T, e, s_e, V, K, out, stream) == hipSuccess ? DFSSM_OK
                                                                                            : DFSSM_ERR_HIP;
}

dfssm_status dfssm_density_field_encode(const float* state, int64_t rows, int64_t d_state, uint32_t* field,
                                        float* scale, hipStream_t stream) {
    if (!state || !field || !scale) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = density_checks(rows, d_state)) return st;
    if (!aligned16(state) || !aligned16(field) || !aligned4(scale)) return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_density_encode(state, rows, d_state, field, scale, nullptr, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

dfssm_status dfssm_density_field_decode(const uint32_t* field, const float* scale, int64_t rows, int64_t d_state,
                                        float* state, hipStream_t stream) {
    if (!state || !field || !scale) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = density_checks(rows, d_state)) return st;
    if (!aligned16(state) || !aligned4(field) || !aligned4(scale)) return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_density_decode(field, scale, rows, d_state, state, stream) == hipSuccess ? DFSSM_OK
                                                                                                 : DFSSM_ERR_HIP;
}

dfssm_status dfssm_density_field_requantize(float* state, int64_t rows, int64_t d_state, uint32_t* field,
                                            float* scale, hipStream_t stream) {
    if (!state) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = density_checks(rows, d_state)) return st;
    if (!aligned16(state) || !aligned4_or_null(field) || !aligned4_or_null(scale)) return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_density_encode(state, rows, d_state, field, scale, state, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

size_t dfssm_decode_layers_workspace_bytes(void) { return dfssm::decode_layers_workspace_bytes(); }

int64_t dfssm_decode_layers_trace_words(void) { return dfssm::decode_layers_trace_words(); }

dfssm_status dfssm_decode_layers_noalloc(const dfssm_decode_layer_weights* w, int64_t n_layers, const float* x_in,
                                         float* x_out, const float* conv_state_in, float* conv_state_out,
                                         float* ssm_state, float eps, int32_t* status, uint32_t* trace,
                                         int64_t spin_limit, uint32_t flags, hipStream_t stream) {
    // the same checks as dfssm_decode_layers, with the library's array standing in for
    // the workspace (a stand-in address passes them; the real one is fetched after)
    alignas(16) static char probe[16];
    if (dfssm_status st = decode_layers_impl(w, n_layers, x_in, x_out, conv_state_in, conv_state_out, ssm_state, eps,
                                             probe, dfssm::decode_layers_workspace_bytes(), status, trace, spin_limit,
                                             flags, stream, /*validate_only=*/true))
        return st;
    uint32_t* ws = dfssm::decode_layers_scratch(stream);
    if (ws == nullptr) return DFSSM_ERR_HIP;
    return decode_layers_impl(w, n_layers, x_in, x_out, conv_state_in, conv_state_out, ssm_state, eps, ws,
                              dfssm::decode_layers_workspace_bytes(), status, trace, spin_limit, flags, stream, false);
}

dfssm_status dfssm_decode_layers(const dfssm_decode_layer_weights* w, int64_t n_layers, const float* x_in,
                                 float* x_out, const float* conv_state_in, float* conv_state_out, float* ssm_state,
                                 float eps, void* workspace, size_t workspace_bytes, int32_t* status, uint32_t* trace,
                                 int64_t spin_limit, uint32_t flags, hipStream_t stream) {
    return decode_layers_impl(w, n_layers, x_in, x_out, conv_state_in, conv_state_out, ssm_state, eps, workspace,
                              workspace_bytes, status, trace, spin_limit, flags, stream);
}

dfssm_status dfssm_mamba2_decode_step(const float* zxbcdt, int64_t S, int64_t nheads, int64_t headdim,
                                      int64_t d_state, const float* conv_state_in, float* conv_state_out,
                                      float* ssm_state, const float* conv_w, const float* conv_b,
                                      const float* dt_bias, const float* A_log, const float* D,
                                      const float* norm_w, float eps, float* out, hipStream_t stream) {
    if (!zxbcdt || !conv_state_in || !conv_state_out || !ssm_state || !conv_w || !conv_b || !dt_bias || !A_log ||
        !D || !norm_w || !out)
        return DFSSM_ERR_INVALID_ARG;
    if (S <= 0 || S > kMaxBatch || nheads <= 0 || headdim <= 0 || d_state <= 0) return DFSSM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || eps > 1e30f) return DFSSM_ERR_INVALID_ARG;
    if (!aligned16(conv_state_in) || !aligned16(conv_state_out) || !aligned16(ssm_state) || !aligned16(conv_w) ||
        !aligned16(norm_w) || !aligned16(out) || !aligned4(zxbcdt) || !aligned4(conv_b) || !aligned4(dt_bias) ||
        !aligned4(A_log) || !aligned4(D))
        return DFSSM_ERR_INVALID_ARG;
    if (!dfssm::mamba2_step_supported(nheads, headdim, d_state)) return DFSSM_ERR_UNSUPPORTED;
    const int64_t d_inner = nheads * headdim, conv_dim = d_inner + 2 * d_state;
    auto overlap = [](const void* a, int64_t na, const void* b, int64_t nb) {
        const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
        return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
    };
    if (overlap(conv_state_in, S * conv_dim * 16, conv_state_out, S * conv_dim * 16) ||
        overlap(out, S * d_inner * 4, zxbcdt, S * (d_inner + conv_dim + nheads) * 4))
        return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_mamba2_step(zxbcdt, S, (int)nheads, conv_state_in, conv_state_out, ssm_state, conv_w, conv_b,
                                     dt_bias, A_log, D, norm_w, eps, out, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

dfssm_status dfssm_int8_gemm(const int8_t* x_q, int64_t ldx, const float* s_x, int64_t M, int64_t N, int64_t K,
                             const int8_t* w, int64_t ldw, const float* s_w, void* y, int64_t ldy, int32_t y_type,
                             hipStream_t stream) {
    if (!x_q || !s_x || !w || !s_w || !y) return DFSSM_ERR_INVALID_ARG;
    if (M <= 0 || N <= 0 || K <= 0 || M >= kMaxRows || N >= kMaxRows) return DFSSM_ERR_INVALID_ARG;
    if (ldx < K || ldw < K || ldy < N || !type_ok(y_type)) return DFSSM_ERR_INVALID_ARG;
    if (!aligned4(s_x) || !aligned4(s_w) || !aligned_type(y, y_type)) return DFSSM_ERR_INVALID_ARG;
    if (K > kMaxK || ldx > kMaxStride || ldw > kMaxStride || ldy >= ((int64_t)1 << 40) ||
        ((N + 31) / 32) * ((M + 31) / 32) > kMaxBlocks)
        return DFSSM_ERR_UNSUPPORTED;
    return dfssm::launch_int8_gemm(x_q, ldx, s_x, M, N, K, w, ldw, s_w, y, ldy, y_type == DFSSM_BF16, stream) ==
                   hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

size_t dfssm_cross_entropy_workspace_bytes(int64_t M, int64_t V, int64_t K) {
    return loss_sizes(M, V, K) == DFSSM_OK ? dfssm::cross_entropy_workspace_bytes(M, V, K) : 0;
}

dfssm_status dfssm_cross_entropy(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K,
                                 const int8_t* e, const float* s_e, const int32_t* targets, float* loss, float* lse,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!x_q || !s_x || !e || !s_e || !targets || !loss || !lse || !workspace) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = loss_sizes(M, V, K)) return st;
    if (!aligned16(x_q) || !aligned16(e) || !aligned16(workspace) || !aligned4(s_x) || !aligned4(s_e) ||
        !aligned4(targets) || !aligned4(loss) || !aligned4(lse))
        return DFSSM_ERR_INVALID_ARG;
    if (workspace_bytes < dfssm::cross_entropy_workspace_bytes(M, V, K)) return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_cross_entropy(x_q, s_x, M, V, K, e, s_e, targets, loss, lse, workspace, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

size_t dfssm_cross_entropy_backward_workspace_bytes(int64_t M, int64_t V, int64_t K, int32_t grad_type,
                                                    int32_t want_dx, int32_t want_de) {
    if (loss_sizes(M, V, K) != DFSSM_OK || M > kMaxLossGradTokens || !type_ok(grad_type) || (!want_dx && !want_de)) return 0;
    return dfssm::cross_entropy_backward_workspace_bytes(M, V, K, grad_type == DFSSM_BF16, want_dx != 0, want_de != 0);
}

dfssm_status dfssm_cross_entropy_backward(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K,
                                          const int8_t* e, const float* s_e, const int32_t* targets, const float* lse,
                                          const float* dloss, void* dx, void* de, int32_t grad_type,
                                          int32_t accumulate_de, void* workspace, size_t workspace_bytes,
                                          hipStream_t stream) {
    if (!x_q || !s_x || !e || !s_e || !targets || !lse || !dloss || (!dx && !de) || !workspace)
        return DFSSM_ERR_INVALID_ARG;
    if (!type_ok(grad_type) || (accumulate_de != 0 && accumulate_de != 1)) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = loss_sizes(M, V, K)) return st;
    if (!aligned16(x_q) || !aligned16(e) || !aligned16(workspace) || !aligned16(dx) || !aligned16(de) ||
        !aligned4(s_x) || !aligned4(s_e) || !aligned4(targets) || !aligned4(lse) || !aligned4(dloss))
        return DFSSM_ERR_INVALID_ARG;
    if (M > kMaxLossGradTokens) return DFSSM_ERR_UNSUPPORTED;
    const bool bf16 = grad_type == DFSSM_BF16;
    if (workspace_bytes < dfssm::cross_entropy_backward_workspace_bytes(M, V, K, bf16, dx != nullptr, de != nullptr))
        return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_cross_entropy_backward(x_q, s_x, M, V, K, e, s_e, targets, lse, dloss, dx, de, bf16,
                                                accumulate_de != 0, workspace, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

size_t dfssm_distillation_workspace_bytes(int64_t M, int64_t V, int64_t K, int64_t top) {
    return distillation_sizes(M, V, K, top) == DFSSM_OK ? dfssm::distillation_workspace_bytes(M, V, K) : 0;
}

dfssm_status dfssm_distillation(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K, const int8_t* e,
                                const float* s_e, const int32_t* top_ids, const float* top_logits, int64_t top,
                                float temperature, float* loss, float* lse, float* logp, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
    if (!x_q || !s_x || !e || !s_e || !top_ids || !top_logits || !loss || !lse || !logp || !workspace) return DFSSM_ERR_INVALID_ARG;
    if (!temperature_ok(temperature)) return DFSSM_ERR_INVALID_ARG;
    if (!aligned16(x_q) || !aligned16(e) || !aligned16(workspace) || !aligned4(s_x) || !aligned4(s_e) ||
        !aligned4(top_ids) || !aligned4(top_logits) || !aligned4(loss) || !aligned4(lse) || !aligned4(logp))
        return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = distillation_sizes(M, V, K, top)) return st;
    if (workspace_bytes < dfssm::distillation_workspace_bytes(M, V, K)) return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_distillation(x_q, s_x, M, V, K, e, s_e, top_ids, top_logits, top, temperature, loss, lse, logp,
                                      workspace, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

size_t dfssm_distillation_backward_workspace_bytes(int64_t M, int64_t V, int64_t K, int64_t top, int32_t grad_type,
                                                   int32_t want_dx, int32_t want_de) {
    if (distillation_sizes(M, V, K, top) != DFSSM_OK || M > kMaxLossGradTokens || !type_ok(grad_type) || (!want_dx && !want_de))
        return 0;
    return dfssm::distillation_backward_workspace_bytes(M, V, K, top, grad_type == DFSSM_BF16, want_dx != 0, want_de != 0);
}

dfssm_status dfssm_distillation_backward(const int8_t* x_q, const float* s_x, int64_t M, int64_t V, int64_t K,
                                         const int8_t* e, const float* s_e, const int32_t* top_ids,
                                         const float* top_logits, int64_t top, float temperature, const float* lse,
                                         const float* logp, const float* dloss, void* dx, void* de, int32_t grad_type,
                                         int32_t accumulate_de, void* workspace, size_t workspace_bytes,
                                         hipStream_t stream) {
    if (!x_q || !s_x || !e || !s_e || !top_ids || !top_logits || !lse || !logp || !dloss || (!dx && !de) || !workspace)
        return DFSSM_ERR_INVALID_ARG;
    if (!type_ok(grad_type) || (accumulate_de != 0 && accumulate_de != 1) || !temperature_ok(temperature)) return DFSSM_ERR_INVALID_ARG;
    if (!aligned16(x_q) || !aligned16(e) || !aligned16(workspace) || !aligned16(dx) || !aligned16(de) ||
        !aligned4(s_x) || !aligned4(s_e) || !aligned4(top_ids) || !aligned4(top_logits) || !aligned4(lse) || !aligned4(logp) ||
        !aligned4(dloss))
        return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = distillation_sizes(M, V, K, top)) return st;
    if (M > kMaxLossGradTokens) return DFSSM_ERR_UNSUPPORTED;
    const bool bf16 = grad_type == DFSSM_BF16;
    if (workspace_bytes < dfssm::distillation_backward_workspace_bytes(M, V, K, top, bf16, dx != nullptr, de != nullptr))
        return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_distillation_backward(x_q, s_x, M, V, K, e, s_e, top_ids, top_logits, top, temperature, lse, logp, dloss,
                                               dx, de, bf16, accumulate_de != 0, workspace, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

dfssm_status dfssm_embedding_lookup_scaled(const int32_t* tokens, int64_t T, const int8_t* e, const float* s_e,
                                           int64_t V, int64_t K, float scale, void* out, int64_t ldo,
                                           int32_t out_type, hipStream_t stream) {
    if (!tokens || !e || !s_e || !out || !type_ok(out_type)) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = embedding_sizes(T, V, K)) return st;
    if (!aligned4(tokens) || !aligned4(s_e) || !aligned_type(out, out_type) || ldo < K) return DFSSM_ERR_INVALID_ARG;
    if (ldo >= ((int64_t)1 << 31)) return DFSSM_ERR_UNSUPPORTED;
    return dfssm::launch_embedding_lookup_scaled(tokens, T, e, s_e, V, K, scale, out, ldo, out_type == DFSSM_BF16,
                                                 stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

size_t dfssm_embedding_backward_workspace_bytes(int64_t T, int64_t V, int64_t K) {
    if (embedding_sizes(T, V, K) != DFSSM_OK || T > kMaxGradTokens || V > kMaxGradRows) return 0;
    return dfssm::embedding_backward_workspace_bytes(T, V, K);
}

dfssm_status dfssm_embedding_backward(const int32_t* tokens, int64_t T, const void* dout, int64_t ldd,
                                      int32_t dout_type, int64_t V, int64_t K, float scale, void* de,
                                      int32_t de_type, int32_t accumulate, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
    if (!tokens || !dout || !de || !workspace || !type_ok(dout_type) || !type_ok(de_type)) return DFSSM_ERR_INVALID_ARG;
    if (accumulate != 0 && accumulate != 1) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = embedding_sizes(T, V, K)) return st;
    if (!aligned4(tokens) || !aligned_type(dout, dout_type) || !aligned_type(de, de_type) || !aligned16(workspace) ||
        ldd < K)
        return DFSSM_ERR_INVALID_ARG;
    if (T > kMaxGradTokens || V > kMaxGradRows || ldd >= ((int64_t)1 << 31)) return DFSSM_ERR_UNSUPPORTED;
    if (workspace_bytes < dfssm::embedding_backward_workspace_bytes(T, V, K)) return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_embedding_backward(tokens, T, dout, ldd, dout_type == DFSSM_BF16, V, K, scale, de,
                                            de_type == DFSSM_BF16, accumulate != 0, workspace, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

dfssm_status dfssm_mamba2_conv(const void* xbc, int64_t ldx, int32_t in_type, int64_t T, int64_t S, int64_t ch,
                               const int32_t* cu_seqlens, const float* conv_w, const float* conv_b,
                               const float* window_in, float* window_out, void* out, int64_t ldo, int32_t out_type,
                               hipStream_t stream) {
    if (!xbc || !conv_w || !conv_b || !out || !type_ok(in_type) || !type_ok(out_type)) return DFSSM_ERR_INVALID_ARG;
    if (!aligned_type(xbc, in_type) || !aligned_type(out, out_type) || !aligned16(conv_w) || !aligned4(conv_b) ||
        !aligned16(window_in) || !aligned16(window_out) || !aligned4(cu_seqlens) || ldx < ch || ldo < ch)
        return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = conv_sizes(T, S, ch, cu_seqlens != nullptr)) return st;
    if (overlapping(window_in, S * ch * 16, window_out, S * ch * 16)) return DFSSM_ERR_INVALID_ARG;
    if (ldx >= kMaxLd || ldo >= kMaxLd) return DFSSM_ERR_UNSUPPORTED;
    return dfssm::launch_mamba2_conv(sequences(cu_seqlens, T, S), xbc, ldx, in_type == DFSSM_BF16, (int)ch, conv_w, conv_b,
                                     window_in, window_out, out, ldo, out_type == DFSSM_BF16, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

size_t dfssm_mamba2_conv_backward_workspace_bytes(int64_t T, int64_t S, int64_t ch) {
    return conv_sizes(T, S, ch, true) == DFSSM_OK ? dfssm::mamba2_conv_backward_workspace_bytes(T, ch) : 0;
}

dfssm_status dfssm_mamba2_conv_backward(const void* xbc, int64_t ldx, int32_t in_type, int64_t T, int64_t S, int64_t ch,
                                        const int32_t* cu_seqlens, const float* conv_w, const float* conv_b,
                                        const float* window_in, const void* dout, int64_t ldd, int32_t out_type,
                                        const float* dwindow_out, void* dxbc, int64_t lddx, float* dconv_w,
                                        float* dconv_b, float* dwindow_in, void* workspace, size_t workspace_bytes,
                                        hipStream_t stream) {
    if (!xbc || !conv_w || !conv_b || !dout || !dxbc || !type_ok(in_type) || !type_ok(out_type)) return DFSSM_ERR_INVALID_ARG;
    if ((dconv_w == nullptr) != (dconv_b == nullptr) || (dconv_w && !workspace)) return DFSSM_ERR_INVALID_ARG;
    if (!aligned_type(xbc, in_type) || !aligned_type(dxbc, in_type) || !aligned_type(dout, out_type) || !aligned16(conv_w) ||
        !aligned4(conv_b) || !aligned16(window_in) || !aligned16(dwindow_out) || !aligned16(dwindow_in) ||
        !aligned16(dconv_w) || !aligned4(dconv_b) || !aligned16(workspace) || !aligned4(cu_seqlens) || ldx < ch || ldd < ch || lddx < ch)
        return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = conv_sizes(T, S, ch, cu_seqlens != nullptr)) return st;
    if (overlapping(dwindow_in, S * ch * 16, dwindow_out, S * ch * 16) || overlapping(dwindow_in, S * ch * 16, window_in, S * ch * 16))
        return DFSSM_ERR_INVALID_ARG;
    if (dconv_w && workspace_bytes < dfssm::mamba2_conv_backward_workspace_bytes(T, ch)) return DFSSM_ERR_INVALID_ARG;
    if (ldx >= kMaxLd || ldd >= kMaxLd || lddx >= kMaxLd) return DFSSM_ERR_UNSUPPORTED;
    return dfssm::launch_mamba2_conv_backward(sequences(cu_seqlens, T, S), xbc, ldx, in_type == DFSSM_BF16, (int)ch, conv_w,
                                              conv_b, window_in, dout, ldd, out_type == DFSSM_BF16, dwindow_out, dxbc, lddx,
                                              dconv_w, dconv_b, dwindow_in, workspace, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

size_t dfssm_mamba2_scan_workspace_bytes(int64_t T, int64_t S, int64_t nheads, int64_t headdim, int64_t d_state,
                                         int64_t ngroups) {
    if (scan_sizes(T, S, nheads, headdim, d_state, ngroups, true) != DFSSM_OK) return 0;
    return dfssm::mamba2_scan_workspace_bytes(T, S, nheads, d_state, ngroups);
}

dfssm_status dfssm_mamba2_scan(const dfssm_mamba2_scan_operands* op, void* y, int64_t ldy, float* state_out,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
    dfssm::ScanArgs a;
    if (!y || !workspace || !aligned16(workspace) || !aligned16(state_out)) return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = scan_operands(op, a)) return st;
    if (dfssm_status st = wide_rows(y, ldy, op->nheads * dfssm::kP, op->type)) return st;
    const int64_t states = op->S * op->nheads * dfssm::kP * op->d_state * 4;
    if (state_out != op->state_in && overlapping(state_out, states, op->state_in, states)) return DFSSM_ERR_INVALID_ARG;
    if (workspace_bytes < dfssm::mamba2_scan_workspace_bytes(op->T, op->S, op->nheads, op->d_state, op->ngroups))
        return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_mamba2_scan(a, op->type == DFSSM_BF16, (int)op->d_state, op->state_in, state_out, y, ldy, workspace,
                                     stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

size_t dfssm_mamba2_scan_backward_workspace_bytes(int64_t T, int64_t S, int64_t nheads, int64_t headdim,
                                                  int64_t d_state, int64_t ngroups) {
    if (scan_sizes(T, S, nheads, headdim, d_state, ngroups, true) != DFSSM_OK) return 0;
    return dfssm::mamba2_scan_backward_workspace_bytes(T, S, nheads, d_state, ngroups);
}

dfssm_status dfssm_mamba2_scan_backward(const dfssm_mamba2_scan_operands* op, const dfssm_mamba2_scan_gradients* grad,
                                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
    dfssm::ScanArgs a;
    if (!grad || !grad->dy || !grad->dx || !grad->dB || !grad->dC || !grad->ddt || !grad->dA_log || !grad->dD || !grad->ddt_bias ||
        !workspace)
        return DFSSM_ERR_INVALID_ARG;
    if (!aligned16(workspace) || !aligned16(grad->dstate_out) || !aligned16(grad->dstate_in) || !aligned4(grad->ddt) ||
        !aligned4(grad->dA_log) || !aligned4(grad->dD) || !aligned4(grad->ddt_bias))
        return DFSSM_ERR_INVALID_ARG;
    if (dfssm_status st = scan_operands(op, a)) return st;
    const int64_t row = op->nheads * dfssm::kP, bc = op->ngroups * op->d_state;
    dfssm_status worst = DFSSM_OK;
    for (dfssm_status st : {wide_rows(grad->dy, grad->lddy, row, op->type), wide_rows(grad->dx, grad->lddx, row, op->type),
                            wide_rows(grad->dB, grad->lddb, bc, op->type), wide_rows(grad->dC, grad->lddc, bc, op->type),
                            stride_ok(grad->ldddt, op->nheads)})
        if (worst != DFSSM_ERR_INVALID_ARG && st != DFSSM_OK) worst = st;
    if (worst != DFSSM_OK) return worst;
    const int64_t states = op->S * op->nheads * dfssm::kP * op->d_state * 4;
    if ((grad->dstate_in != grad->dstate_out && overlapping(grad->dstate_in, states, grad->dstate_out, states)) ||
        overlapping(grad->dstate_in, states, op->state_in, states))
        return DFSSM_ERR_INVALID_ARG;
    if (workspace_bytes < dfssm::mamba2_scan_backward_workspace_bytes(op->T, op->S, op->nheads, op->d_state, op->ngroups))
        return DFSSM_ERR_INVALID_ARG;
    return dfssm::launch_mamba2_scan_backward(a, op->type == DFSSM_BF16, (int)op->d_state, op->state_in, grad->dy, grad->lddy,
                                              grad->dstate_out, grad->dx, grad->lddx, grad->ddt, grad->ldddt, grad->dB, grad->lddb,
                                              grad->dC, grad->lddc, grad->dA_log, grad->dD, grad->ddt_bias, grad->dstate_in,
                                              workspace, stream) == hipSuccess
               ? DFSSM_OK
               : DFSSM_ERR_HIP;
}

}  // extern "C"
