"""ctypes binding of libdfssm.so (include/dfssm.h) -- argument marshalling only.

Every function here has the C entry point's name and forwards raw device pointers,
sizes and the current HIP stream; all arithmetic happens in the HIP kernels.  If
the shared library is missing the import fails loudly: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdfssm.so")

DFSSM_OK = 0
DFSSM_ERR_INVALID_ARG = 1
DFSSM_ERR_UNSUPPORTED = 2
DFSSM_ERR_HIP = 3

# every symbol include/dfssm.h declares
EXPORTED = ("dfssm_status_string", "dfssm_version", "dfssm_quantize_act", "dfssm_lora_down",
            "dfssm_lora_down_strided_batched", "dfssm_quantize_lora_down",
            "dfssm_quantize_lora_down_strided_batched", "dfssm_scaffold_lora_gemm",
            "dfssm_scaffold_lora_gemm_strided_batched", "dfssm_scaffold_lora_gemm_given_t",
            "dfssm_scaffold_lora_gemm_given_t_strided_batched", "dfssm_scaffold_lora_forward",
            "dfssm_scaffold_lora_forward_strided_batched", "dfssm_int8_rowscale_gemm",
            "dfssm_int8_rowscale_gemm_strided_batched", "dfssm_embedding_lookup", "dfssm_mamba2_decode_step",
            "dfssm_prefill_plan", "dfssm_decode_layers_workspace_bytes", "dfssm_decode_layers_trace_words",
            "dfssm_decode_layers", "dfssm_decode_layers_noalloc", "dfssm_density_field_encode",
            "dfssm_density_field_decode", "dfssm_density_field_requantize", "dfssm_int8_gemm",
            "dfssm_cross_entropy_workspace_bytes", "dfssm_cross_entropy",
            "dfssm_cross_entropy_backward_workspace_bytes", "dfssm_cross_entropy_backward",
            "dfssm_embedding_lookup_scaled", "dfssm_embedding_backward_workspace_bytes", "dfssm_embedding_backward",
            "dfssm_distillation_workspace_bytes", "dfssm_distillation",
            "dfssm_distillation_backward_workspace_bytes", "dfssm_distillation_backward",
            "dfssm_mamba2_conv", "dfssm_mamba2_conv_backward_workspace_bytes", "dfssm_mamba2_conv_backward",
            "dfssm_mamba2_scan_workspace_bytes", "dfssm_mamba2_scan", "dfssm_mamba2_scan_backward_workspace_bytes",
            "dfssm_mamba2_scan_backward")

# dfssm_type: the element type of a result or a gradient
DFSSM_F32 = 0
DFSSM_BF16 = 1

DFSSM_DECODE_STATUS_TIMEOUT = 1
DFSSM_DECODE_STATUS_GAVE_UP = 2
DFSSM_DECODE_UNREACHABLE_WAITS = 1

# dfssm_decode_layer_weights: the stacked per-layer weights of dfssm_decode_layers
DECODE_WEIGHT_FIELDS = ("in_w_bits", "in_s_w", "in_w_a", "in_s_a", "in_w_b", "in_s_b", "conv_w", "conv_b",
                        "dt_bias", "A_log", "D", "norm_w", "out_w_bits", "out_s_w", "out_w_a", "out_s_a",
                        "out_w_b", "out_s_b")


class DecodeLayerWeights(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in DECODE_WEIGHT_FIELDS]


# dfssm_mamba2_scan_operands: pointers, then sizes, then the type
SCAN_POINTERS = ("x", "B", "C", "dt", "A_log", "D", "dt_bias", "state_in", "cu_seqlens")
SCAN_SIZES = ("ldx", "ldb", "ldc", "lddt", "T", "S", "nheads", "headdim", "d_state", "ngroups")


class ScanOperands(ctypes.Structure):
    _fields_ = ([(name, ctypes.c_void_p) for name in SCAN_POINTERS] + [(name, ctypes.c_int64) for name in SCAN_SIZES]
                + [("type", ctypes.c_int32)])


# dfssm_mamba2_scan_gradients
SCAN_GRADIENTS = ("dy", "dstate_out", "dx", "dB", "dC", "ddt", "dA_log", "dD", "ddt_bias", "dstate_in")
SCAN_GRADIENT_SIZES = ("lddy", "lddx", "lddb", "lddc", "ldddt")


class ScanGradients(ctypes.Structure):
    _fields_ = ([(name, ctypes.c_void_p) for name in SCAN_GRADIENTS]
                + [(name, ctypes.c_int64) for name in SCAN_GRADIENT_SIZES])


class DfssmError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {status_string(status)} ({status})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m bit_scaffold_int8_amd.build`")
    # torch ships its own HIP runtime and loads it by path.  Loaded first, the library
    # would bring in the system's copy as well, and device pointers from torch would not
    # be valid in the library's runtime; with torch loaded first, the library's
    # dependency resolves to torch's runtime (same soname).
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.dfssm_status_string.argtypes = [ctypes.c_int]
    lib.dfssm_status_string.restype = ctypes.c_char_p
    lib.dfssm_version.argtypes = []
    lib.dfssm_version.restype = i32
    lib.dfssm_decode_layers_workspace_bytes.argtypes = []
    lib.dfssm_decode_layers_workspace_bytes.restype = ctypes.c_size_t
    lib.dfssm_decode_layers_trace_words.argtypes = []
    lib.dfssm_decode_layers_trace_words.restype = i64
    sigs = {
        "dfssm_quantize_act": [P, i64, i64, P, P, P],
        "dfssm_lora_down": [P, i64, i64, P, i32, P, P],
        "dfssm_lora_down_strided_batched": [P, i64, i64, P, i32, P, i64, P],
        "dfssm_quantize_lora_down": [P, i64, i64, P, i32, P, P, P, P],
        "dfssm_quantize_lora_down_strided_batched": [P, i64, i64, P, i32, P, P, P, i64, P],
        "dfssm_scaffold_lora_gemm": [P, P, i64, i64, i64, P, P, P, P, P, P, i32, P, P, P, P],
        "dfssm_scaffold_lora_gemm_strided_batched": [P, P, i64, i64, i64, P, P, P, P, P, P, i32, P, P, P, i64, P],
        "dfssm_scaffold_lora_gemm_given_t": [P, P, i64, i64, i64, P, P, P, P, P, P, i32, P, P, P],
        "dfssm_scaffold_lora_gemm_given_t_strided_batched": [P, P, i64, i64, i64, P, P, P, P, P, P, i32, P, P, i64,
                                                             P],
        "dfssm_scaffold_lora_forward": [P, i64, i64, i64, P, P, P, P, P, P, i32, P, P, P, P, P, P],
        "dfssm_scaffold_lora_forward_strided_batched": [P, i64, i64, i64, P, P, P, P, P, P, i32, P, P, P, P, P,
                                                        i64, P],
        "dfssm_int8_rowscale_gemm": [P, P, i64, i64, i64, P, P, P, P, P],
        "dfssm_int8_rowscale_gemm_strided_batched": [P, P, i64, i64, i64, P, P, P, P, i64, P],
        "dfssm_embedding_lookup": [P, i64, P, P, i64, i64, P, P],
        "dfssm_mamba2_decode_step": [P, i64, i64, i64, i64, P, P, P, P, P, P, P, P, P, ctypes.c_float, P, P],
        "dfssm_prefill_plan": [i64, i64, i64, i64, P, P, P],
        "dfssm_decode_layers": [P, i64, P, P, P, P, P, ctypes.c_float, P, ctypes.c_size_t, P, P, i64, ctypes.c_uint32,
                                P],
        "dfssm_decode_layers_noalloc": [P, i64, P, P, P, P, P, ctypes.c_float, P, P, i64, ctypes.c_uint32, P],
        "dfssm_density_field_encode": [P, i64, i64, P, P, P],
        "dfssm_density_field_decode": [P, P, i64, i64, P, P],
        "dfssm_density_field_requantize": [P, i64, i64, P, P, P],
        "dfssm_int8_gemm": [P, i64, P, i64, i64, i64, P, i64, P, P, i64, i32, P],
        "dfssm_cross_entropy": [P, P, i64, i64, i64, P, P, P, P, P, P, ctypes.c_size_t, P],
        "dfssm_cross_entropy_backward": [P, P, i64, i64, i64, P, P, P, P, P, P, P, i32, i32, P, ctypes.c_size_t, P],
        "dfssm_embedding_lookup_scaled": [P, i64, P, P, i64, i64, ctypes.c_float, P, i64, i32, P],
        "dfssm_embedding_backward": [P, i64, P, i64, i32, i64, i64, ctypes.c_float, P, i32, i32, P, ctypes.c_size_t,
                                     P],
        "dfssm_distillation": [P, P, i64, i64, i64, P, P, P, P, i64, ctypes.c_float, P, P, P, P, ctypes.c_size_t, P],
        "dfssm_distillation_backward": [P, P, i64, i64, i64, P, P, P, P, i64, ctypes.c_float, P, P, P, P, P, i32, i32, P,
                                        ctypes.c_size_t, P],
        "dfssm_mamba2_conv": [P, i64, i32, i64, i64, i64, P, P, P, P, P, P, i64, i32, P],
        "dfssm_mamba2_conv_backward": [P, i64, i32, i64, i64, i64, P, P, P, P, P, i64, i32, P, P, i64, P, P, P, P,
                                       ctypes.c_size_t, P],
        "dfssm_mamba2_scan": [P, P, i64, P, P, ctypes.c_size_t, P],
        "dfssm_mamba2_scan_backward": [P, P, P, ctypes.c_size_t, P],
    }
    for name, argtypes in (("dfssm_cross_entropy_workspace_bytes", [i64, i64, i64]),
                           ("dfssm_cross_entropy_backward_workspace_bytes", [i64, i64, i64, i32, i32, i32]),
                           ("dfssm_embedding_backward_workspace_bytes", [i64, i64, i64]),
                           ("dfssm_distillation_workspace_bytes", [i64] * 4),
                           ("dfssm_distillation_backward_workspace_bytes", [i64] * 4 + [i32] * 3),
                           ("dfssm_mamba2_conv_backward_workspace_bytes", [i64, i64, i64]),
                           ("dfssm_mamba2_scan_workspace_bytes", [i64] * 6),
                           ("dfssm_mamba2_scan_backward_workspace_bytes", [i64] * 6)):
        getattr(lib, name).argtypes = argtypes
        getattr(lib, name).restype = ctypes.c_size_t
    for name, argtypes in sigs.items():
        f = getattr(lib, name)
        f.argtypes = argtypes
        f.restype = ctypes.c_int
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.dfssm_status_string(int(status)).decode()


def dfssm_version() -> int:
    return int(lib.dfssm_version())


def dfssm_prefill_plan(M: int, N: int, K: int, batch: int = 1):
    """(main configuration, tail configuration or -1, first tail column) the MFMA
    kernel's cost model picks for this shape; host only."""
    mc, tc, ns = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int64(0)
    _call("dfssm_prefill_plan", M, N, K, batch, ctypes.addressof(mc), ctypes.addressof(tc), ctypes.addressof(ns))
    return mc.value, tc.value, ns.value


def _ptr(t):
    """Device pointer of a tensor, an int address, or None (NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def raw(name: str, *args) -> int:
    """Pointer-level call of any entry point; returns the status code unchanged."""
    return getattr(lib, name)(*args)


def _call(name, *args):
    st = getattr(lib, name)(*args)
    if st != DFSSM_OK:
        raise DfssmError(st, name)


def dfssm_quantize_act(x, x_q, s_x, stream=None) -> None:
    """x fp32 [M, K] -> x_q int8 [M, K], s_x fp32 [M]."""
    M, K = x.shape
    _call("dfssm_quantize_act", _ptr(x), M, K, _ptr(x_q), _ptr(s_x), _stream(stream))


def dfssm_lora_down(x_q, w_b, t, stream=None) -> None:
    """t int32 [M, 16] = W_B [16, K] x_q [M, K]^T."""
    M, K = x_q.shape
    _call("dfssm_lora_down", _ptr(x_q), M, K, _ptr(w_b), int(w_b.shape[0]), _ptr(t), _stream(stream))


def dfssm_lora_down_strided_batched(x_q, w_b, t, stream=None) -> None:
    """x_q [B, M, K], w_b [B, 16, K] -> t [B, M, 16]."""
    B, M, K = x_q.shape
    _call("dfssm_lora_down_strided_batched", _ptr(x_q), M, K, _ptr(w_b), int(w_b.shape[1]), _ptr(t), B,
          _stream(stream))


def dfssm_quantize_lora_down(x, w_b, x_q, s_x, t, stream=None) -> None:
    """x fp32 [M, K] -> x_q, s_x and (w_b given) t = W_B x_q; w_b = None for rank 0."""
    M, K = x.shape
    rank = 0 if w_b is None else int(w_b.shape[0])
    _call("dfssm_quantize_lora_down", _ptr(x), M, K, _ptr(w_b), rank, _ptr(x_q), _ptr(s_x), _ptr(t),
          _stream(stream))


def dfssm_quantize_lora_down_strided_batched(x, w_b, x_q, s_x, t, stream=None) -> None:
    """x [B, M, K], w_b [B, 16, K] -> x_q [B, M, K], s_x [B, M], t [B, M, 16]."""
    B, M, K = x.shape
    rank = 0 if w_b is None else int(w_b.shape[1])
    _call("dfssm_quantize_lora_down_strided_batched", _ptr(x), M, K, _ptr(w_b), rank, _ptr(x_q), _ptr(s_x),
          _ptr(t), B, _stream(stream))


def dfssm_scaffold_lora_gemm(x_q, s_x, w_bits, s_w, w_a, s_a, w_b, s_b, y, acc_dbg=None, t_dbg=None,
                             stream=None) -> None:
    """y fp32 [M, N] from x_q [M, K], s_x [M], w_bits [N, K/8], s_w [N] and the LoRA pair
    w_a [N, 16], s_a [N], w_b [16, K], s_b [16] (all None for rank 0); t = W_B x_q is
    computed by the kernel (t_dbg [M, 16], when given, receives it)."""
    M, K = x_q.shape
    N = w_bits.shape[0]
    rank = 0 if w_a is None else int(w_a.shape[1])
    _call("dfssm_scaffold_lora_gemm", _ptr(x_q), _ptr(s_x), M, N, K, _ptr(w_bits), _ptr(s_w), _ptr(w_a),
          _ptr(s_a), _ptr(w_b), _ptr(s_b), rank, _ptr(y), _ptr(acc_dbg), _ptr(t_dbg), _stream(stream))


def dfssm_scaffold_lora_gemm_strided_batched(x_q, s_x, w_bits, s_w, w_a, s_a, w_b, s_b, y, acc_dbg=None,
                                             t_dbg=None, stream=None) -> None:
    """Batched form: x_q [B, M, K], s_x [B, M], w_bits [B, N, K/8], s_w [B, N], w_a [B, N, 16],
    s_a [B, N], w_b [B, 16, K], s_b [B, 16], y [B, M, N], t_dbg [B, M, 16]."""
    B, M, K = x_q.shape
    N = w_bits.shape[1]
    rank = 0 if w_a is None else int(w_a.shape[2])
    _call("dfssm_scaffold_lora_gemm_strided_batched", _ptr(x_q), _ptr(s_x), M, N, K, _ptr(w_bits), _ptr(s_w),
          _ptr(w_a), _ptr(s_a), _ptr(w_b), _ptr(s_b), rank, _ptr(y), _ptr(acc_dbg), _ptr(t_dbg), B,
          _stream(stream))


def dfssm_scaffold_lora_gemm_given_t(x_q, s_x, w_bits, s_w, w_a, s_a, s_b, t, y, acc_dbg=None,
                                     stream=None) -> None:
    """The product with t [M, 16] given (from dfssm_lora_down / dfssm_quantize_lora_down):
    y fp32 [M, N] from x_q, s_x, w_bits, s_w and w_a, s_a, s_b, t (all None for rank 0)."""
    M, K = x_q.shape
    N = w_bits.shape[0]
    rank = 0 if w_a is None else int(w_a.shape[1])
    _call("dfssm_scaffold_lora_gemm_given_t", _ptr(x_q), _ptr(s_x), M, N, K, _ptr(w_bits), _ptr(s_w), _ptr(w_a),
          _ptr(s_a), _ptr(s_b), _ptr(t), rank, _ptr(y), _ptr(acc_dbg), _stream(stream))


def dfssm_scaffold_lora_gemm_given_t_strided_batched(x_q, s_x, w_bits, s_w, w_a, s_a, s_b, t, y, acc_dbg=None,
                                                     stream=None) -> None:
    """Batched form of dfssm_scaffold_lora_gemm_given_t: every operand with a leading [B]."""
    B, M, K = x_q.shape
    N = w_bits.shape[1]
    rank = 0 if w_a is None else int(w_a.shape[2])
    _call("dfssm_scaffold_lora_gemm_given_t_strided_batched", _ptr(x_q), _ptr(s_x), M, N, K, _ptr(w_bits),
          _ptr(s_w), _ptr(w_a), _ptr(s_a), _ptr(s_b), _ptr(t), rank, _ptr(y), _ptr(acc_dbg), B, _stream(stream))


def dfssm_scaffold_lora_forward(x, w_bits, s_w, w_a, s_a, w_b, s_b, x_q, s_x, t, y, acc_dbg=None,
                                stream=None) -> None:
    """The whole projection in one call: x fp32 [M, K] -> x_q, s_x, t and y [M, N]
    (LoRA operands all None for rank 0)."""
    M, K = x.shape
    N = w_bits.shape[0]
    rank = 0 if w_a is None else int(w_a.shape[1])
    _call("dfssm_scaffold_lora_forward", _ptr(x), M, N, K, _ptr(w_bits), _ptr(s_w), _ptr(w_a), _ptr(s_a),
          _ptr(w_b), _ptr(s_b), rank, _ptr(x_q), _ptr(s_x), _ptr(t), _ptr(y), _ptr(acc_dbg), _stream(stream))


def dfssm_scaffold_lora_forward_strided_batched(x, w_bits, s_w, w_a, s_a, w_b, s_b, x_q, s_x, t, y,
                                                acc_dbg=None, stream=None) -> None:
    """Batched form of dfssm_scaffold_lora_forward: every operand with a leading [B]."""
    B, M, K = x.shape
    N = w_bits.shape[1]
    rank = 0 if w_a is None else int(w_a.shape[2])
    _call("dfssm_scaffold_lora_forward_strided_batched", _ptr(x), M, N, K, _ptr(w_bits), _ptr(s_w), _ptr(w_a),
          _ptr(s_a), _ptr(w_b), _ptr(s_b), rank, _ptr(x_q), _ptr(s_x), _ptr(t), _ptr(y), _ptr(acc_dbg), B,
          _stream(stream))


def dfssm_int8_rowscale_gemm(x_q, s_x, e, s_e, y, acc_dbg=None, stream=None) -> None:
    """int8 LM head: y [M, N] = s_x (s_e (E x_q)) from x_q [M, K], s_x [M], e [N, K], s_e [N]."""
    M, K = x_q.shape
    N = e.shape[0]
    _call("dfssm_int8_rowscale_gemm", _ptr(x_q), _ptr(s_x), M, N, K, _ptr(e), _ptr(s_e), _ptr(y), _ptr(acc_dbg),
          _stream(stream))


def dfssm_int8_rowscale_gemm_strided_batched(x_q, s_x, e, s_e, y, acc_dbg=None, stream=None) -> None:
    """Batched form: x_q [B, M, K], s_x [B, M], e [B, N, K], s_e [B, N], y [B, M, N]."""
    B, M, K = x_q.shape
    N = e.shape[1]
    _call("dfssm_int8_rowscale_gemm_strided_batched", _ptr(x_q), _ptr(s_x), M, N, K, _ptr(e), _ptr(s_e), _ptr(y),
          _ptr(acc_dbg), B, _stream(stream))


def dfssm_embedding_lookup(tokens, e, s_e, out, stream=None) -> None:
    """out [T, K] = s_e[id] E[id] for the int32 ids `tokens` [T] (ids outside [0, V): zeros)."""
    T = tokens.shape[0]
    V, K = e.shape
    _call("dfssm_embedding_lookup", _ptr(tokens), T, _ptr(e), _ptr(s_e), V, K, _ptr(out), _stream(stream))


def dfssm_mamba2_decode_step(zxbcdt, conv_state_in, conv_state_out, ssm_state, conv_w, conv_b, dt_bias, A_log, D,
                             norm_w, eps, out, stream=None) -> None:
    """Mamba-2 step for S sequences: zxbcdt [S, 2 d_inner + 2 d_state + nheads] (in_proj
    output) -> out [S, d_inner] (out_proj input); conv_state_in -> conv_state_out
    [S, conv_dim, 4]; ssm_state [S, nheads, headdim, d_state] updated in place."""
    S = zxbcdt.shape[0]
    _, nheads, headdim, d_state = ssm_state.shape
    _call("dfssm_mamba2_decode_step", _ptr(zxbcdt), S, nheads, headdim, d_state, _ptr(conv_state_in),
          _ptr(conv_state_out), _ptr(ssm_state), _ptr(conv_w), _ptr(conv_b), _ptr(dt_bias), _ptr(A_log), _ptr(D),
          _ptr(norm_w), float(eps), _ptr(out), _stream(stream))


def dfssm_decode_layers_workspace_bytes() -> int:
    return int(lib.dfssm_decode_layers_workspace_bytes())


def dfssm_decode_layers_trace_words() -> int:
    return int(lib.dfssm_decode_layers_trace_words())


def dfssm_decode_layers(weights: dict, n_layers, x_in, x_out, conv_state_in, conv_state_out, ssm_state, eps,
                        workspace, status, trace=None, spin_limit: int = 0, flags: int = 0, stream=None) -> None:
    """The decode step of n_layers stacked layers for one sequence, one launch.  `weights`
    maps every name of DECODE_WEIGHT_FIELDS to a device tensor (stacked over layers);
    workspace is a zeroed device buffer of dfssm_decode_layers_workspace_bytes() bytes,
    status a device int32 the kernel ORs failure bits into."""
    w = DecodeLayerWeights(*[_ptr(weights[name]) for name in DECODE_WEIGHT_FIELDS])
    nbytes = workspace.numel() * workspace.element_size()
    _call("dfssm_decode_layers", ctypes.addressof(w), int(n_layers), _ptr(x_in), _ptr(x_out), _ptr(conv_state_in),
          _ptr(conv_state_out), _ptr(ssm_state), float(eps), _ptr(workspace), nbytes, _ptr(status), _ptr(trace),
          int(spin_limit), int(flags), _stream(stream))


def dfssm_decode_layers_noalloc(weights: dict, n_layers, x_in, x_out, conv_state_in, conv_state_out, ssm_state,
                                eps, status, trace=None, spin_limit: int = 0, flags: int = 0, stream=None) -> None:
    """dfssm_decode_layers with the library's own per-GPU array as the workspace: nothing
    is allocated; calls that overlap on one GPU race."""
    w = DecodeLayerWeights(*[_ptr(weights[name]) for name in DECODE_WEIGHT_FIELDS])
    _call("dfssm_decode_layers_noalloc", ctypes.addressof(w), int(n_layers), _ptr(x_in), _ptr(x_out),
          _ptr(conv_state_in), _ptr(conv_state_out), _ptr(ssm_state), float(eps), _ptr(status), _ptr(trace),
          int(spin_limit), int(flags), _stream(stream))


def dfssm_density_field_encode(state, field, scale, stream=None) -> None:
    """state fp32 [R, d] -> field uint32 [R, d / 8], scale fp32 [R] (density-field codec)."""
    R, d = state.shape
    _call("dfssm_density_field_encode", _ptr(state), R, d, _ptr(field), _ptr(scale), _stream(stream))


def dfssm_density_field_decode(field, scale, state, stream=None) -> None:
    """field uint32 [R, d / 8], scale fp32 [R] -> state fp32 [R, d] (popcount readout)."""
    R, d = state.shape
    _call("dfssm_density_field_decode", _ptr(field), _ptr(scale), R, d, _ptr(state), _stream(stream))


def dfssm_density_field_requantize(state, field=None, scale=None, stream=None) -> None:
    """The round trip in place: state [R, d] <- its field's readout (field, scale optional)."""
    R, d = state.shape
    _call("dfssm_density_field_requantize", _ptr(state), R, d, _ptr(field), _ptr(scale), _stream(stream))



# ---- operators with fp32 or bf16 results: these functions also check what the C ABI cannot see
# (element types, shapes, strides, devices; ValueError) and run on the tensors' own device.

def _type(what, t) -> int:
    """dfssm_type of a tensor."""
    import torch
    if t.dtype is torch.float32:
        return DFSSM_F32
    if t.dtype is torch.bfloat16:
        return DFSSM_BF16
    raise ValueError(f"{what}: fp32 or bf16 expected, got {t.dtype}")


def _rows(what, t, shape, dtype=None) -> int:
    """Checks a matrix with contiguous rows; its row stride in elements."""
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{what}: {dtype} expected, got {t.dtype}")
    M, K = shape
    sm, sk = t.stride()
    if (sk != 1 and K > 1) or (sm < K and M > 1):
        raise ValueError(f"{what}: rows must be contiguous and must not overlap, got strides {t.stride()}")
    return sm if M > 1 else K


def _dense(what, t, shape, dtype) -> None:
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous {dtype} {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)} "
                         f"with strides {t.stride()}")


def _matrix(what, t) -> tuple:
    if t.dim() != 2:
        raise ValueError(f"{what}: a matrix expected, got shape {tuple(t.shape)}")
    return t.shape


def _run_on(name, tensors, stream, *args) -> None:
    """Calls an entry point on the device that holds the tensors (and on its current stream)."""
    import torch
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev or dev < 0:
            raise ValueError(f"{name}: all tensors must be on one GPU, got {[str(t.device) for t in tensors]}")
    if stream is None:
        # the current stream's handle without the Stream object, whose making takes longer than a launch
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        _call(name, *args, stream)
        return
    with torch.cuda.device(dev):
        _call(name, *args, stream)


def _bytes(t) -> int:
    if not t.is_contiguous():
        raise ValueError("workspace: a contiguous tensor expected")
    return t.numel() * t.element_size()


def dfssm_int8_gemm(x_q, s_x, w, s_w, y, stream=None) -> None:
    """y [M, N] (fp32 or bf16) = s_x (s_w (W x_q)) from x_q int8 [M, K], s_x [M], w int8 [N, K], s_w [N]; the rows
    of x_q, w and y may be strided."""
    import torch
    M, K = _matrix("x_q", x_q)
    N = _matrix("w", w)[0]
    ldx, ldw = _rows("x_q", x_q, (M, K), torch.int8), _rows("w", w, (N, K), torch.int8)
    ldy = _rows("y", y, (M, N))
    _dense("s_x", s_x, (M,), torch.float32)
    _dense("s_w", s_w, (N,), torch.float32)
    _run_on("dfssm_int8_gemm", (x_q, s_x, w, s_w, y), stream, x_q.data_ptr(), ldx, s_x.data_ptr(), M, N, K,
            w.data_ptr(), ldw, s_w.data_ptr(), y.data_ptr(), ldy, _type("y", y))


def _head(x_q, s_x, e, s_e, targets=None) -> tuple:
    """Checks the head's operands; (M, V, K)."""
    import torch
    M, K = _matrix("x_q", x_q)
    V = _matrix("e", e)[0]
    _dense("x_q", x_q, (M, K), torch.int8)
    _dense("s_x", s_x, (M,), torch.float32)
    _dense("e", e, (V, K), torch.int8)
    _dense("s_e", s_e, (V,), torch.float32)
    if targets is not None:
        _dense("targets", targets, (M,), torch.int32)
    return M, V, K


def dfssm_cross_entropy_workspace_bytes(M: int, V: int, K: int) -> int:
    return int(lib.dfssm_cross_entropy_workspace_bytes(M, V, K))


def dfssm_cross_entropy(x_q, s_x, e, s_e, targets, loss, lse, workspace, stream=None) -> None:
    """loss, lse fp32 [M] of the head's logits (x_q int8 [M, K], s_x [M], e int8 [V, K], s_e [V]) for the
    int32 targets [M] (outside [0, V): the position does not count); workspace: a tensor of
    dfssm_cross_entropy_workspace_bytes(M, V, K) bytes."""
    import torch
    M, V, K = _head(x_q, s_x, e, s_e, targets)
    _dense("loss", loss, (M,), torch.float32)
    _dense("lse", lse, (M,), torch.float32)
    _run_on("dfssm_cross_entropy", (x_q, s_x, e, s_e, targets, loss, lse, workspace), stream, x_q.data_ptr(),
            s_x.data_ptr(), M, V, K, e.data_ptr(), s_e.data_ptr(), targets.data_ptr(), loss.data_ptr(),
            lse.data_ptr(), workspace.data_ptr(), _bytes(workspace))


def dfssm_cross_entropy_backward_workspace_bytes(M: int, V: int, K: int, dx, de) -> int:
    """For the gradients dx and de (tensors, or None for one that is not wanted)."""
    if dx is None and de is None:
        raise ValueError("dfssm_cross_entropy_backward_workspace_bytes: dx or de expected")
    t = _type("dx, de", de if dx is None else dx)
    return int(lib.dfssm_cross_entropy_backward_workspace_bytes(M, V, K, t, dx is not None, de is not None))


def dfssm_cross_entropy_backward(x_q, s_x, e, s_e, targets, lse, dloss, dx, de, workspace, accumulate: bool = False,
                                 stream=None) -> None:
    """dx [M, K] and de [V, K] (both fp32 or both bf16; None for one that is not wanted) from the forward
    call's operands, its lse, and dloss fp32 [M]; accumulate adds to de.  workspace: a tensor of
    dfssm_cross_entropy_backward_workspace_bytes(M, V, K, dx, de) bytes."""
    import torch
    M, V, K = _head(x_q, s_x, e, s_e, targets)
    _dense("lse", lse, (M,), torch.float32)
    _dense("dloss", dloss, (M,), torch.float32)
    outs = [t for t in (dx, de) if t is not None]
    if not outs:
        raise ValueError("dfssm_cross_entropy_backward: dx or de expected")
    t = _type("dx, de", outs[0])
    if dx is not None:
        _dense("dx", dx, (M, K), outs[0].dtype)
    if de is not None:
        _dense("de", de, (V, K), outs[0].dtype)
    _run_on("dfssm_cross_entropy_backward", (x_q, s_x, e, s_e, targets, lse, dloss, workspace, *outs), stream,
            x_q.data_ptr(), s_x.data_ptr(), M, V, K, e.data_ptr(), s_e.data_ptr(), targets.data_ptr(),
            lse.data_ptr(), dloss.data_ptr(), _ptr(dx), _ptr(de), t, int(bool(accumulate)), workspace.data_ptr(),
            _bytes(workspace))


def _teacher(x_q, s_x, e, s_e, top_ids, top_logits) -> tuple:
    """Checks the head's and the teacher's operands; (M, V, K, top)."""
    import torch
    M, V, K = _head(x_q, s_x, e, s_e)
    top = _matrix("top_ids", top_ids)[1]
    _dense("top_ids", top_ids, (M, top), torch.int32)
    _dense("top_logits", top_logits, (M, top), torch.float32)
    return M, V, K, top


def dfssm_distillation_workspace_bytes(M: int, V: int, K: int, top: int) -> int:
    return int(lib.dfssm_distillation_workspace_bytes(M, V, K, top))


def dfssm_distillation(x_q, s_x, e, s_e, top_ids, top_logits, temperature, loss, lse, logp, workspace, stream=None) -> None:
    """loss, lse fp32 [M] and logp fp32 [M, top]: the divergence of the head's distribution (x_q int8 [M, K], s_x [M],
    e int8 [V, K], s_e [V]) from a teacher's, given by its largest logits (top_ids int32, top_logits fp32, both
    [M, top]; ids outside [0, V): no entry) at a temperature; workspace: a tensor of
    dfssm_distillation_workspace_bytes(M, V, K, top) bytes."""
    import torch
    M, V, K, top = _teacher(x_q, s_x, e, s_e, top_ids, top_logits)
    _dense("loss", loss, (M,), torch.float32)
    _dense("lse", lse, (M,), torch.float32)
    _dense("logp", logp, (M, top), torch.float32)
    _run_on("dfssm_distillation", (x_q, s_x, e, s_e, top_ids, top_logits, loss, lse, logp, workspace), stream,
            x_q.data_ptr(), s_x.data_ptr(), M, V, K, e.data_ptr(), s_e.data_ptr(), top_ids.data_ptr(),
            top_logits.data_ptr(), top, float(temperature), loss.data_ptr(), lse.data_ptr(), logp.data_ptr(),
            workspace.data_ptr(), _bytes(workspace))


def dfssm_distillation_backward_workspace_bytes(M: int, V: int, K: int, top: int, dx, de) -> int:
    """For the gradients dx and de (tensors, or None for one that is not wanted)."""
    if dx is None and de is None:
        raise ValueError("dfssm_distillation_backward_workspace_bytes: dx or de expected")
    t = _type("dx, de", de if dx is None else dx)
    return int(lib.dfssm_distillation_backward_workspace_bytes(M, V, K, top, t, dx is not None, de is not None))


def dfssm_distillation_backward(x_q, s_x, e, s_e, top_ids, top_logits, temperature, lse, logp, dloss, dx, de, workspace,
                                accumulate: bool = False, stream=None) -> None:
    """dx [M, K] and de [V, K] (both fp32 or both bf16; None for one that is not wanted) from the forward call's
    operands, its lse and logp, and dloss fp32 [M]; accumulate adds to de.  workspace: a tensor of
    dfssm_distillation_backward_workspace_bytes(M, V, K, top, dx, de) bytes."""
    import torch
    M, V, K, top = _teacher(x_q, s_x, e, s_e, top_ids, top_logits)
    _dense("lse", lse, (M,), torch.float32)
    _dense("logp", logp, (M, top), torch.float32)
    _dense("dloss", dloss, (M,), torch.float32)
    outs = [t for t in (dx, de) if t is not None]
    if not outs:
        raise ValueError("dfssm_distillation_backward: dx or de expected")
    t = _type("dx, de", outs[0])
    if dx is not None:
        _dense("dx", dx, (M, K), outs[0].dtype)
    if de is not None:
        _dense("de", de, (V, K), outs[0].dtype)
    _run_on("dfssm_distillation_backward", (x_q, s_x, e, s_e, top_ids, top_logits, lse, logp, dloss, workspace, *outs),
            stream, x_q.data_ptr(), s_x.data_ptr(), M, V, K, e.data_ptr(), s_e.data_ptr(), top_ids.data_ptr(),
            top_logits.data_ptr(), top, float(temperature), lse.data_ptr(), logp.data_ptr(), dloss.data_ptr(), _ptr(dx),
            _ptr(de), t, int(bool(accumulate)), workspace.data_ptr(), _bytes(workspace))


def dfssm_embedding_lookup_scaled(tokens, e, s_e, scale, out, stream=None) -> None:
    """out [T, K] (fp32 or bf16, rows may be strided) = scale s_e[id] E[id] for the int32 ids `tokens` [T]
    (ids outside [0, V): zeros)."""
    import torch
    V, K = _matrix("e", e)
    T = tokens.numel()
    _dense("tokens", tokens, (T,), torch.int32)
    _dense("e", e, (V, K), torch.int8)
    _dense("s_e", s_e, (V,), torch.float32)
    ldo = _rows("out", out, (T, K))
    _run_on("dfssm_embedding_lookup_scaled", (tokens, e, s_e, out), stream, tokens.data_ptr(), T, e.data_ptr(),
            s_e.data_ptr(), V, K, float(scale), out.data_ptr(), ldo, _type("out", out))


def dfssm_embedding_backward_workspace_bytes(T: int, V: int, K: int) -> int:
    return int(lib.dfssm_embedding_backward_workspace_bytes(T, V, K))


def dfssm_embedding_backward(tokens, dout, scale, de, workspace, accumulate: bool = False, stream=None) -> None:
    """de [V, K] = scale times the sum of dout's rows (fp32 or bf16 [T, K], rows may be strided) of each id
    of the int32 `tokens` [T]; accumulate adds to de instead (rows without tokens stay as they are).
    workspace: a tensor of dfssm_embedding_backward_workspace_bytes(T, V, K) bytes."""
    import torch
    V, K = _matrix("de", de)
    T = tokens.numel()
    _dense("tokens", tokens, (T,), torch.int32)
    ldd = _rows("dout", dout, (T, K))
    _dense("de", de, (V, K), de.dtype)
    _run_on("dfssm_embedding_backward", (tokens, dout, de, workspace), stream, tokens.data_ptr(), T, dout.data_ptr(),
            ldd, _type("dout", dout), V, K, float(scale), de.data_ptr(), _type("de", de), int(bool(accumulate)),
            workspace.data_ptr(), _bytes(workspace))


# ---- the Mamba-2 operators over packed sequences.  cu_seqlens: int32 offsets [S + 1] on the same device, or None for
# sequences of equal length (their number is that of the states or windows, or `sequences`).

def _sequences(name, T, cu_seqlens, states, sequences) -> int:
    """The number of sequences, agreed on by everything that tells it."""
    if cu_seqlens is None and sequences is None:   # (the common case, without the list)
        S = 0
        for t in states:
            if t is not None:
                if S not in (0, t.shape[0]):
                    raise ValueError(f"{name}: the numbers of sequences differ: {S}, {t.shape[0]}")
                S = t.shape[0]
        if T % (S or 1):
            raise ValueError(f"{name}: {T} rows are not {S} sequences of equal length")
        return S or 1
    import torch
    told = [t.shape[0] for t in states if t is not None]
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError(f"{name}: cu_seqlens: S + 1 offsets expected, got shape {tuple(cu_seqlens.shape)}")
        _dense("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32)
        told.append(cu_seqlens.numel() - 1)
    if sequences is not None:
        told.append(int(sequences))
    S = told[0] if told else 1
    if any(n != S for n in told):
        raise ValueError(f"{name}: the numbers of sequences differ: {told}")
    if cu_seqlens is None and (S <= 0 or T % S != 0):
        raise ValueError(f"{name}: {T} rows are not {S} sequences of equal length")
    return S


def _optional(what, t, shape):
    import torch
    if t is not None:
        _dense(what, t, shape, torch.float32)


def _present(*tensors):
    return [t for t in tensors if t is not None]


def _conv_operands(name, xbc, conv_w, conv_b, windows, cu_seqlens, sequences) -> tuple:
    import torch
    T, ch = _matrix("xbc", xbc)
    ldx = _rows("xbc", xbc, (T, ch))
    _dense("conv_w", conv_w, (ch, 4), torch.float32)
    _dense("conv_b", conv_b, (ch,), torch.float32)
    S = _sequences(name, T, cu_seqlens, windows.values(), sequences)
    for what, t in windows.items():
        _optional(what, t, (S, ch, 4))
    return ldx, _type("xbc", xbc), T, S, ch


def dfssm_mamba2_conv(xbc, conv_w, conv_b, window_in, window_out, out, cu_seqlens=None, sequences=None, stream=None) -> None:
    """out [T, ch] = silu of the causal convolution of xbc [T, ch] (each fp32 or bf16, rows may be strided) with
    conv_w [ch, 4], conv_b [ch]; window_in / window_out fp32 [S, ch, 4] or None (zeros / not wanted)."""
    ldx, tx, T, S, ch = _conv_operands("dfssm_mamba2_conv", xbc, conv_w, conv_b,
                                       {"window_in": window_in, "window_out": window_out}, cu_seqlens, sequences)
    ldo = _rows("out", out, (T, ch))
    _run_on("dfssm_mamba2_conv", _present(xbc, conv_w, conv_b, out, window_in, window_out, cu_seqlens), stream,
            xbc.data_ptr(), ldx, tx, T, S, ch, _ptr(cu_seqlens), conv_w.data_ptr(), conv_b.data_ptr(), _ptr(window_in),
            _ptr(window_out), out.data_ptr(), ldo, _type("out", out))


def dfssm_mamba2_conv_backward_workspace_bytes(T: int, S: int, ch: int) -> int:
    return int(lib.dfssm_mamba2_conv_backward_workspace_bytes(T, S, ch))


def dfssm_mamba2_conv_backward(xbc, conv_w, conv_b, window_in, dout, dwindow_out, dxbc, dconv_w, dconv_b, dwindow_in,
                               workspace, cu_seqlens=None, sequences=None, stream=None) -> None:
    """dxbc [T, ch] (xbc's type), dconv_w, dconv_b (both None: frozen) and dwindow_in (or None) from the forward call's
    operands, dout [T, ch] and dwindow_out (or None: zeros); workspace: a tensor of
    dfssm_mamba2_conv_backward_workspace_bytes(T, S, ch) bytes, or None with frozen weights."""
    windows = {"window_in": window_in, "dwindow_out": dwindow_out, "dwindow_in": dwindow_in}
    ldx, tx, T, S, ch = _conv_operands("dfssm_mamba2_conv_backward", xbc, conv_w, conv_b, windows, cu_seqlens, sequences)
    ldd, lddx = _rows("dout", dout, (T, ch)), _rows("dxbc", dxbc, (T, ch), xbc.dtype)
    _optional("dconv_w", dconv_w, (ch, 4))
    _optional("dconv_b", dconv_b, (ch,))
    _run_on("dfssm_mamba2_conv_backward",
            _present(xbc, conv_w, conv_b, dout, dxbc, *windows.values(), dconv_w, dconv_b, workspace, cu_seqlens), stream,
            xbc.data_ptr(), ldx, tx, T, S, ch, _ptr(cu_seqlens), conv_w.data_ptr(), conv_b.data_ptr(), _ptr(window_in),
            dout.data_ptr(), ldd, _type("dout", dout), _ptr(dwindow_out), dxbc.data_ptr(), lddx, _ptr(dconv_w),
            _ptr(dconv_b), _ptr(dwindow_in), _ptr(workspace), 0 if workspace is None else _bytes(workspace))


def _heads(what, t, T, dtype) -> tuple:
    """Checks rows of parts [T, A, B] whose parts lie side by side; (stride of a row, A, B)."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != T:
        raise ValueError(f"{what}: shape ({T}, ., .) expected, got {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {dtype} expected, got {t.dtype}")
    _, A, B = shape
    st, sa, sb = t.stride()
    if (sb != 1 and B > 1) or (sa != B and A > 1) or (st < A * B and T > 1):
        raise ValueError(f"{what}: rows must be contiguous and must not overlap, got strides {t.stride()}")
    return (st if T > 1 else A * B), A, B


# dfssm_mamba2_scan_operands and dfssm_mamba2_scan_gradients as bytes (packed faster than a ctypes structure is made)
_pack_operands = struct.Struct(f"{len(SCAN_POINTERS)}Q{len(SCAN_SIZES)}qi4x").pack
_pack_gradients = struct.Struct(f"{len(SCAN_GRADIENTS)}Q{len(SCAN_GRADIENT_SIZES)}q").pack


def _scan_operands(name, x, dt, B, C, A_log, D, dt_bias, state_in, states, cu_seqlens, sequences):
    """Checks the scan's operands; (dfssm_mamba2_scan_operands, its tensors, T, H, P, G, N)."""
    import torch
    T = x.shape[0] if x.dim() else 0
    ldx, H, P = _heads("x", x, T, x.dtype)
    ldb, G, N = _heads("B", B, T, x.dtype)
    ldc, Gc, Nc = _heads("C", C, T, x.dtype)
    if Gc != G or Nc != N:
        raise ValueError(f"C: shape {tuple(B.shape)} expected, got {tuple(C.shape)}")
    lddt = _rows("dt", dt, (T, H), torch.float32)
    f32, row = torch.float32, (H,)
    _dense("A_log", A_log, row, f32)
    _dense("D", D, row, f32)
    _dense("dt_bias", dt_bias, row, f32)
    S = _sequences(name, T, cu_seqlens, (state_in, *states), sequences)
    tensors = [x, dt, B, C, A_log, D, dt_bias]
    state = (S, H, P, N)
    for t in (state_in, *states):
        if t is not None:
            _dense("state", t, state, f32)
            tensors.append(t)
    if cu_seqlens is not None:
        tensors.append(cu_seqlens)
    op = _pack_operands(x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), A_log.data_ptr(), D.data_ptr(),
                        dt_bias.data_ptr(), 0 if state_in is None else state_in.data_ptr(),
                        0 if cu_seqlens is None else cu_seqlens.data_ptr(), ldx, ldb, ldc, lddt, T, S, H, P, N, G,
                        _type("x", x))
    return op, tensors, T, H, P, G, N


def dfssm_mamba2_scan_workspace_bytes(T: int, S: int, nheads: int, headdim: int, d_state: int, ngroups: int = 1) -> int:
    return int(lib.dfssm_mamba2_scan_workspace_bytes(T, S, nheads, headdim, d_state, ngroups))


def dfssm_mamba2_scan(x, dt, B, C, A_log, D, dt_bias, state_in, state_out, y, workspace, cu_seqlens=None, sequences=None,
                      stream=None) -> None:
    """y [T, H, 64] and state_out of the scan over x [T, H, 64], dt fp32 [T, H] (raw), B, C [T, G, N], A_log, D,
    dt_bias [H] (x, B, C, y all fp32 or all bf16, rows may be strided); state_in / state_out fp32 [S, H, 64, N] or None
    (zeros / not wanted), the same tensor for an update in place; workspace: a tensor of
    dfssm_mamba2_scan_workspace_bytes(T, S, H, 64, N, G) bytes."""
    op, tensors, T, H, P, _, _ = _scan_operands("dfssm_mamba2_scan", x, dt, B, C, A_log, D, dt_bias, state_in,
                                                (state_out,), cu_seqlens, sequences)
    ldy, Hy, Py = _heads("y", y, T, x.dtype)
    if Hy != H or Py != P:
        raise ValueError(f"y: shape {tuple(x.shape)} expected, got {tuple(y.shape)}")
    tensors += (y, workspace)
    _run_on("dfssm_mamba2_scan", tensors, stream, op, y.data_ptr(), ldy, _ptr(state_out), workspace.data_ptr(),
            _bytes(workspace))


def dfssm_mamba2_scan_backward_workspace_bytes(T: int, S: int, nheads: int, headdim: int, d_state: int,
                                               ngroups: int = 1) -> int:
    return int(lib.dfssm_mamba2_scan_backward_workspace_bytes(T, S, nheads, headdim, d_state, ngroups))


def dfssm_mamba2_scan_backward(x, dt, B, C, A_log, D, dt_bias, state_in, dy, dstate_out, dx, ddt, dB, dC, dA_log, dD, ddt_bias,
                               dstate_in, workspace, cu_seqlens=None, sequences=None, stream=None) -> None:
    """The gradients of dfssm_mamba2_scan from its operands, dy [T, H, 64] and dstate_out (fp32 [S, H, 64, N] or None:
    zeros): dx, dB, dC (their operands' type and shape), ddt fp32 [T, H], dA_log, dD, ddt_bias fp32 [H], dstate_in (fp32, or
    None: not wanted; dstate_out itself: in place); workspace: a tensor of
    dfssm_mamba2_scan_backward_workspace_bytes(T, S, H, 64, N, G) bytes."""
    import torch
    op, tensors, T, H, _, _, _ = _scan_operands("dfssm_mamba2_scan_backward", x, dt, B, C, A_log, D, dt_bias, state_in,
                                                (dstate_out, dstate_in), cu_seqlens, sequences)
    strides = {}
    for what, t, like in (("dy", dy, x), ("dx", dx, x), ("dB", dB, B), ("dC", dC, C)):
        strides[what], *same = _heads(what, t, T, x.dtype)
        if same != list(like.shape[1:]):
            raise ValueError(f"{what}: shape {tuple(like.shape)} expected, got {tuple(t.shape)}")
    ldddt = _rows("ddt", ddt, (T, H), torch.float32)
    for what, t in (("dA_log", dA_log), ("dD", dD), ("ddt_bias", ddt_bias)):
        _dense(what, t, (H,), torch.float32)
    grad = _pack_gradients(dy.data_ptr(), _ptr(dstate_out) or 0, dx.data_ptr(), dB.data_ptr(), dC.data_ptr(), ddt.data_ptr(),
                           dA_log.data_ptr(), dD.data_ptr(), ddt_bias.data_ptr(), _ptr(dstate_in) or 0, strides["dy"],
                           strides["dx"], strides["dB"], strides["dC"], ldddt)
    _run_on("dfssm_mamba2_scan_backward", [*tensors, dy, dx, dB, dC, ddt, dA_log, dD, ddt_bias, workspace], stream,
            op, grad, workspace.data_ptr(), _bytes(workspace))
