"""ctypes binding to libtemx.so (argument marshalling only).

The ``te_mx_*`` functions take raw integer pointers and mirror include/temx.h;
they raise ``TemxError`` on any status other than TE_MX_OK.  The torch-level
helpers (``quantize``, ``gemm``, ``grouped_gemm``) only allocate outputs with
torch and pass ``data_ptr()`` and the current stream; every step of the
computation runs in the library's CUDA kernels.  There is no fallback: if the
library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtemx.so")

TE_MX_OK = 0
STATUS_NAMES = {0: "TE_MX_OK", 1: "TE_MX_ERR_INVALID_ARG", 2: "TE_MX_ERR_UNSUPPORTED_SHAPE",
                3: "TE_MX_ERR_MISALIGNED", 4: "TE_MX_ERR_WORKSPACE_TOO_SMALL", 5: "TE_MX_ERR_CUDA",
                6: "TE_MX_ERR_DEVICE_TIMEOUT", 7: "TE_MX_ERR_ARCH"}
BF16, FP16, FP32 = 0, 1, 2                       # te_mx_dtype
ACT_SILU, ACT_GELU, ACT_RELU = 0, 1, 2           # te_mx_activation
ACTIVATIONS = {"silu": ACT_SILU, "gelu": ACT_GELU, "relu": ACT_RELU}
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1              # te_mx_scoring
SCORINGS = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}
EPI_NONE, EPI_BIAS, EPI_GELU_AUX, EPI_BIAS_GELU_AUX, EPI_DGELU, EPI_ACCUMULATE_F32 = 0, 1, 2, 3, 4, 5

# (name, restype, argtypes) for every function declared in include/temx.h
_I64, _I32, _P, _SZ = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
SIGNATURES = {
    "te_mx_scale_pitch": (_SZ, [_I64]),
    "te_mx_quantize": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _P]),
    "te_mx_block_quantize": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _P, _I64, _P]),
    "te_mx_block_scale_pitch_fp32": (_I64, [_I64]),
    "te_mx_block_quantize_fp32": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _P, _I64, _P]),
    "te_mx_layernorm_quantize": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, ctypes.c_float, _P, _P, _I64, _P,
                                                _P, _I64, _P, _P, _P]),
    "te_mx_layernorm": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _P, _I32, ctypes.c_float, _P, _I64, _P, _P, _P]),
    "te_mx_layernorm_backward_workspace_size": (_SZ, [_I64, _I64]),
    "te_mx_layernorm_backward": (ctypes.c_int, [_P, _I64, _P, _I64, _I64, _I64, _I32, _P, _I32, _P, _P, _P, _I64, _P,
                                                _P, _P, _SZ, _P]),
    "te_mx_rmsnorm": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _I64, _P, _I32, ctypes.c_float, _P, _I64, _P, _I64, _P,
                                     _P]),
    "te_mx_rmsnorm_quantize": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _I32, ctypes.c_float, _P, _I64, _P, _I64,
                                              _P, _P, _I64, _P, _P, _I64, _P, _P]),
    "te_mx_rmsnorm_backward_workspace_size": (_SZ, [_I64, _I64]),
    "te_mx_rmsnorm_backward": (ctypes.c_int, [_P, _I64, _P, _I64, _I64, _I64, _I32, _P, _I32, _P, _P, _I64, _P, _I64, _P,
                                              _P, _SZ, _P]),
    "te_mx_route": (ctypes.c_int, [_P, _I64, _I32, _I64, _I32, _P, _I32, _I32, _I32, ctypes.c_float, _P, _P, _P]),
    "te_mx_route_backward": (ctypes.c_int, [_P, _P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _I32, ctypes.c_float, _P, _I64,
                                            _P]),
    "te_mx_moe_sort": (ctypes.c_int, [_P, _I64, _I32, _P, _P, _P, _P]),
    "te_mx_moe_dispatch": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I32, _I64, _P, _I64, _P, _I64, _P]),
    "te_mx_moe_combine": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _I64, _I32, _P, _P, _I64, _P, _I64, _P]),
    "te_mx_moe_combine_backward": (ctypes.c_int, [_P, _I64, _P, _I64, _I64, _I64, _I32, _P, _P, _I64, _I32, _P, _I64, _P,
                                                  _P]),
    "te_mx_grouped_code_width": (_I64, [_I64, _I32]),
    "te_mx_grouped_scale_width": (_I64, [_I64, _I32]),
    "te_mx_quantize_colwise_grouped": (ctypes.c_int, [_P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _I64, _P]),
    "te_mx_grouped_gemm_wgrad": (ctypes.c_int, [_I32, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I32, _P,
                                                _P]),
    "te_mx_quantize_dbias_workspace_size": (_SZ, [_I64, _I64]),
    "te_mx_quantize_dbias": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _P, _P, _SZ, _P]),
    "te_mx_quantize_dbias_noalloc": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _P, _P]),
    "te_mx_gemm": (ctypes.c_int, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _P, _I32, _P, _P, _P, _SZ, _P]),
    "te_mx_gated_gemm": (ctypes.c_int, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _P, _I32, _P, _P, _P]),
    "te_mx_grouped_gated_gemm": (ctypes.c_int, [_I32, _P, _I64, _P, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I32, _P, _P,
                                                _P]),
    "te_mx_gated_backward": (ctypes.c_int, [_P, _I64, _P, _I64, _I64, _I64, _I32, _P, _I64, _P, _P, _I64, _P, _I64, _P,
                                            _I64, _P]),
    "te_mx_gemm_fp32_scales": (ctypes.c_int, [_P, _P, _I64, _P, _P, _I64, _I32, _I64, _I64, _I64, _P, _I32, _P, _P,
                                              _P]),
    "te_mx_grouped_gemm": (ctypes.c_int, [_I32, _P, _I64, _P, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I32,
                                          _P, _P, _P, _SZ, _P]),
    "te_mx_gemm_workspace_size": (_SZ, [_I64, _I64, _I64, _I32]),
    "te_mx_device_status": (ctypes.c_int, []),
    "te_mx_selftest_timeout": (ctypes.c_int, [ctypes.c_uint32, _P]),
    "te_mx_last_error": (ctypes.c_char_p, []),
    "te_mx_version": (ctypes.c_char_p, []),
}


class TemxError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libtemx.so (built in-tree by ``_build.build()``); raises if missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m mxfp8_block_scaled_quantize_gb300._build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(l, name)
            f.restype, f.argtypes = res, args
        _lib = l
    return _lib


def _check(status: int) -> None:
    if status != TE_MX_OK:
        raise TemxError(status, lib().te_mx_last_error().decode())


# ---------------------------------------------------------------- raw C ABI

def te_mx_scale_pitch(k: int) -> int:
    return lib().te_mx_scale_pitch(k)


def te_mx_quantize(x, rows, cols, ld_x, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col, stream) -> None:
    _check(lib().te_mx_quantize(x, rows, cols, ld_x, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col, stream))


def te_mx_block_quantize(x, rows, cols, ld_x, block_2d, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col,
                         stream) -> None:
    _check(lib().te_mx_block_quantize(x, rows, cols, ld_x, block_2d, q_row, s_row, ld_s_row, q_col, s_col,
                                      ld_s_col, stream))


def te_mx_layernorm_quantize(x, rows, hidden, ld_x, gamma, beta, eps, q_row, s_row, ld_s_row, q_col, s_col,
                             ld_s_col, mu, rsigma, stream) -> None:
    _check(lib().te_mx_layernorm_quantize(x, rows, hidden, ld_x, gamma, beta, eps, q_row, s_row, ld_s_row, q_col,
                                          s_col, ld_s_col, mu, rsigma, stream))


def te_mx_layernorm(x, rows, hidden, ld_x, dtype, gamma, beta, param_dtype, eps, y, ld_y, mu, rsigma, stream) -> None:
    _check(lib().te_mx_layernorm(x, rows, hidden, ld_x, dtype, gamma, beta, param_dtype, eps, y, ld_y, mu, rsigma,
                                 stream))


def te_mx_layernorm_backward_workspace_size(rows, hidden) -> int:
    return lib().te_mx_layernorm_backward_workspace_size(rows, hidden)


def te_mx_layernorm_backward(dy, ld_dy, x, ld_x, rows, hidden, dtype, gamma, param_dtype, mu, rsigma, dx, ld_dx,
                             dgamma, dbeta, workspace, workspace_bytes, stream) -> None:
    _check(lib().te_mx_layernorm_backward(dy, ld_dy, x, ld_x, rows, hidden, dtype, gamma, param_dtype, mu, rsigma, dx,
                                          ld_dx, dgamma, dbeta, workspace, workspace_bytes, stream))


def te_mx_rmsnorm(x, rows, hidden, ld_x, dtype, residual, ld_residual, gamma, param_dtype, eps, z, ld_z, y, ld_y, rsigma,
                  stream) -> None:
    _check(lib().te_mx_rmsnorm(x, rows, hidden, ld_x, dtype, residual, ld_residual, gamma, param_dtype, eps, z, ld_z, y,
                               ld_y, rsigma, stream))


def te_mx_rmsnorm_quantize(x, rows, hidden, ld_x, residual, ld_residual, gamma, param_dtype, eps, z, ld_z, y, ld_y, q_row,
                           s_row, ld_s_row, q_col, s_col, ld_s_col, rsigma, stream) -> None:
    _check(lib().te_mx_rmsnorm_quantize(x, rows, hidden, ld_x, residual, ld_residual, gamma, param_dtype, eps, z, ld_z, y,
                                        ld_y, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col, rsigma, stream))


def te_mx_rmsnorm_backward_workspace_size(rows, hidden) -> int:
    return lib().te_mx_rmsnorm_backward_workspace_size(rows, hidden)


def te_mx_rmsnorm_backward(dy, ld_dy, z, ld_z, rows, hidden, dtype, gamma, param_dtype, rsigma, dz, ld_dz, dx, ld_dx,
                           dgamma, workspace, workspace_bytes, stream) -> None:
    _check(lib().te_mx_rmsnorm_backward(dy, ld_dy, z, ld_z, rows, hidden, dtype, gamma, param_dtype, rsigma, dz, ld_dz, dx,
                                        ld_dx, dgamma, workspace, workspace_bytes, stream))


def te_mx_route(logits, tokens, experts, ld_logits, dtype, bias, k, scoring, renormalise, scale, index, weight,
                stream) -> None:
    _check(lib().te_mx_route(logits, tokens, experts, ld_logits, dtype, bias, k, scoring, renormalise, scale, index, weight,
                             stream))


def te_mx_route_backward(dweight, logits, ld_logits, index, tokens, experts, dtype, k, scoring, renormalise, scale, dlogits,
                         ld_dlogits, stream) -> None:
    _check(lib().te_mx_route_backward(dweight, logits, ld_logits, index, tokens, experts, dtype, k, scoring, renormalise,
                                      scale, dlogits, ld_dlogits, stream))


def te_mx_moe_sort(index, slots, experts, group_m, row, slot, stream) -> None:
    _check(lib().te_mx_moe_sort(index, slots, experts, group_m, row, slot, stream))


def te_mx_moe_dispatch(x, ld_x, row_bytes, scales, ld_scales, scale_bytes, row, tokens, k, total_rows, out, ld_out,
                       out_scales, ld_out_scales, stream) -> None:
    _check(lib().te_mx_moe_dispatch(x, ld_x, row_bytes, scales, ld_scales, scale_bytes, row, tokens, k, total_rows, out,
                                    ld_out, out_scales, ld_out_scales, stream))


def te_mx_moe_combine(y, ld_y, total_rows, hidden, dtype, row, tokens, k, weight, residual, ld_residual, out, ld_out,
                      stream) -> None:
    _check(lib().te_mx_moe_combine(y, ld_y, total_rows, hidden, dtype, row, tokens, k, weight, residual, ld_residual, out,
                                   ld_out, stream))


def te_mx_moe_combine_backward(dout, ld_dout, y, ld_y, total_rows, hidden, dtype, row, weight, tokens, k, dy, ld_dy,
                               dweight, stream) -> None:
    _check(lib().te_mx_moe_combine_backward(dout, ld_dout, y, ld_y, total_rows, hidden, dtype, row, weight, tokens, k, dy,
                                            ld_dy, dweight, stream))


def te_mx_grouped_code_width(total_m, num_groups) -> int:
    return lib().te_mx_grouped_code_width(total_m, num_groups)


def te_mx_grouped_scale_width(total_m, num_groups) -> int:
    return lib().te_mx_grouped_scale_width(total_m, num_groups)


def te_mx_quantize_colwise_grouped(x, total_m, cols, ld_x, num_groups, group_m, q, ld_q, s, ld_s, stream) -> None:
    _check(lib().te_mx_quantize_colwise_grouped(x, total_m, cols, ld_x, num_groups, group_m, q, ld_q, s, ld_s,
                                                stream))


def te_mx_grouped_gemm_wgrad(num_groups, group_m, total_m, dY, s_dY, X, s_X, M, N, ld_q, ld_s, accumulate, D,
                             stream) -> None:
    _check(lib().te_mx_grouped_gemm_wgrad(num_groups, group_m, total_m, dY, s_dY, X, s_X, M, N, ld_q, ld_s,
                                          accumulate, D, stream))


def te_mx_quantize_dbias_workspace_size(rows, cols) -> int:
    return lib().te_mx_quantize_dbias_workspace_size(rows, cols)


def te_mx_quantize_dbias(x, rows, cols, ld_x, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col, dbias, workspace,
                         workspace_bytes, stream) -> None:
    _check(lib().te_mx_quantize_dbias(x, rows, cols, ld_x, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col, dbias,
                                      workspace, workspace_bytes, stream))


def te_mx_quantize_dbias_noalloc(x, rows, cols, ld_x, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col, dbias,
                                 stream) -> None:
    """Same as te_mx_quantize_dbias, for callers that cannot allocate device
    memory: the scratch is built into the library (TE_MX_NOALLOC_SCRATCH_BYTES)."""
    _check(lib().te_mx_quantize_dbias_noalloc(x, rows, cols, ld_x, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col,
                                              dbias, stream))


def te_mx_gemm(A, sA, ld_sA, B, sB, ld_sB, M, N, K, bias, epilogue, D, aux, workspace, workspace_bytes,
               stream) -> None:
    _check(lib().te_mx_gemm(A, sA, ld_sA, B, sB, ld_sB, M, N, K, bias, epilogue, D, aux, workspace,
                            workspace_bytes, stream))


def te_mx_grouped_gemm(num_groups, group_m, total_m, X, sX, ld_sX, W, sW, ld_sW, N, K, bias, epilogue, D, aux,
                       workspace, workspace_bytes, stream) -> None:
    _check(lib().te_mx_grouped_gemm(num_groups, group_m, total_m, X, sX, ld_sX, W, sW, ld_sW, N, K, bias,
                                    epilogue, D, aux, workspace, workspace_bytes, stream))


def te_mx_gated_gemm(A, sA, ld_sA, W, sW, ld_sW, M, F, K, bias, activation, D, aux, stream) -> None:
    _check(lib().te_mx_gated_gemm(A, sA, ld_sA, W, sW, ld_sW, M, F, K, bias, activation, D, aux, stream))


def te_mx_grouped_gated_gemm(num_groups, group_m, total_m, X, sX, ld_sX, W, sW, ld_sW, F, K, bias, activation, D, aux,
                             stream) -> None:
    _check(lib().te_mx_grouped_gated_gemm(num_groups, group_m, total_m, X, sX, ld_sX, W, sW, ld_sW, F, K, bias,
                                          activation, D, aux, stream))


def te_mx_gated_backward(dh, ld_dh, gate_up, ld_gate_up, rows, F, activation, d_gate_up, ld_d, q_row, s_row, ld_s_row,
                         q_col, ld_q_col, s_col, ld_s_col, stream) -> None:
    _check(lib().te_mx_gated_backward(dh, ld_dh, gate_up, ld_gate_up, rows, F, activation, d_gate_up, ld_d, q_row, s_row,
                                      ld_s_row, q_col, ld_q_col, s_col, ld_s_col, stream))


def te_mx_gemm_workspace_size(M, N, K, num_groups=0) -> int:
    return lib().te_mx_gemm_workspace_size(M, N, K, num_groups)


def te_mx_device_status() -> None:
    _check(lib().te_mx_device_status())


def te_mx_selftest_timeout(limit_us: int, stream=None) -> None:
    _check(lib().te_mx_selftest_timeout(limit_us, 0 if stream is None else stream))


def te_mx_version() -> str:
    return lib().te_mx_version().decode()


# ---------------------------------------------------------------- torch helpers

_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _raw_stream() -> int:
    """The current device's current stream's handle, taken without building a
    Stream object, which costs as much as a small launch (the first call puts the
    function that does so in this one's place)."""
    global _raw_stream
    import torch
    c = torch._C
    if hasattr(c, "_cuda_getCurrentRawStream") and hasattr(c, "_cuda_getDevice"):
        torch.cuda.init()
        current, device = c._cuda_getCurrentRawStream, c._cuda_getDevice
        _raw_stream = lambda: current(device())  # noqa: E731
    else:
        _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


def _current_device() -> int:
    """The current CUDA device's index (the first call puts the function that
    looks it up in this one's place)."""
    global _current_device
    import torch
    torch.cuda.init()
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _current_device()


def _stream_ptr(stream=None) -> int:
    return _raw_stream() if stream is None else stream.cuda_stream


def _on(stream):
    """Context in which what a helper allocates belongs to ``stream`` as its
    launches do (else a temporary could be given out again, on the current
    stream, while the kernel still uses it)."""
    import torch
    return torch.cuda.stream(stream)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def quantize(x, rowwise: bool = True, colwise: bool = False, stream=None, out=None, dbias: bool = False,
             workspace=None):
    """MXFP8-quantise a 2-D bf16 CUDA tensor.  Returns a dict with q_row
    [R,C], s_row [R, pitch(C)] and/or q_col [C,R], s_col [C, pitch(R)] (uint8),
    and with ``dbias`` also "dbias" (bf16 [C], the column sums); the bias
    gradient's scratch is ``workspace`` (uint8 CUDA tensor) or allocated here."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda
    rows, cols = x.shape
    assert x.stride(1) == 1
    o = dict(out or {})
    if rowwise and "q_row" not in o:
        o["q_row"] = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
        o["s_row"] = torch.empty(rows, te_mx_scale_pitch(cols), dtype=torch.uint8, device=x.device)
    if colwise and "q_col" not in o:
        o["q_col"] = torch.empty(cols, rows, dtype=torch.uint8, device=x.device)
        o["s_col"] = torch.empty(cols, te_mx_scale_pitch(rows), dtype=torch.uint8, device=x.device)
    args = (x.data_ptr(), rows, cols, x.stride(0),
            _ptr(o.get("q_row")), _ptr(o.get("s_row")), o["s_row"].stride(0) if "s_row" in o else 0,
            _ptr(o.get("q_col")), _ptr(o.get("s_col")), o["s_col"].stride(0) if "s_col" in o else 0)
    if not dbias:
        te_mx_quantize(*args, _stream_ptr(stream))
        return o
    if "dbias" not in o:
        o["dbias"] = torch.empty(cols, dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(1, te_mx_quantize_dbias_workspace_size(rows, cols)), dtype=torch.uint8,
                                device=x.device)
    te_mx_quantize_dbias(*args, o["dbias"].data_ptr(), workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
    return o


def te_mx_block_scale_pitch_fp32(n) -> int:
    return int(lib().te_mx_block_scale_pitch_fp32(n))


def te_mx_block_quantize_fp32(x, rows, cols, ld_x, block_2d, q_row, s_row, ld_s_row, q_col, s_col, ld_s_col,
                              stream) -> None:
    _check(lib().te_mx_block_quantize_fp32(x, rows, cols, ld_x, block_2d, q_row, s_row, ld_s_row, q_col, s_col,
                                           ld_s_col, stream))


def block_quantize_fp32(x, block_2d: bool = False, rowwise: bool = True, colwise: bool = False, stream=None,
                        out=None):
    """Float8BlockScaling-quantise a 2-D bf16 CUDA tensor keeping FP32 scales:
    E4M3 codes as ``block_quantize`` and fp32 scales, one per block and row
    (``s_row`` [rows, pitch(cols)], ``s_col`` [cols, pitch(rows)]), for
    ``gemm_fp32_scales``."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda
    rows, cols = x.shape
    assert x.stride(1) == 1
    o = dict(out or {})
    if rowwise and "q_row" not in o:
        o["q_row"] = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
        o["s_row"] = torch.empty(rows, te_mx_block_scale_pitch_fp32(cols), dtype=torch.float32, device=x.device)
    if colwise and "q_col" not in o:
        o["q_col"] = torch.empty(cols, rows, dtype=torch.uint8, device=x.device)
        o["s_col"] = torch.empty(cols, te_mx_block_scale_pitch_fp32(rows), dtype=torch.float32, device=x.device)
    te_mx_block_quantize_fp32(x.data_ptr(), rows, cols, x.stride(0), int(bool(block_2d)),
                              _ptr(o.get("q_row")), _ptr(o.get("s_row")), o["s_row"].stride(0) if "s_row" in o else 0,
                              _ptr(o.get("q_col")), _ptr(o.get("s_col")), o["s_col"].stride(0) if "s_col" in o else 0,
                              _stream_ptr(stream))
    return o


def block_quantize(x, block_2d: bool = False, rowwise: bool = True, colwise: bool = False, stream=None, out=None):
    """Float8BlockScaling-quantise a 2-D bf16 CUDA tensor with E8M0-cast
    scales: 1x128 / 128x1 blocks, or 128x128 blocks with ``block_2d``.  The
    outputs have the layout of ``quantize`` (block scales repeated per 32
    elements), so ``gemm`` consumes them as they are."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda
    rows, cols = x.shape
    assert x.stride(1) == 1
    o = dict(out or {})
    if rowwise and "q_row" not in o:
        o["q_row"] = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
        o["s_row"] = torch.empty(rows, te_mx_scale_pitch(cols), dtype=torch.uint8, device=x.device)
    if colwise and "q_col" not in o:
        o["q_col"] = torch.empty(cols, rows, dtype=torch.uint8, device=x.device)
        o["s_col"] = torch.empty(cols, te_mx_scale_pitch(rows), dtype=torch.uint8, device=x.device)
    te_mx_block_quantize(x.data_ptr(), rows, cols, x.stride(0), int(bool(block_2d)),
                         _ptr(o.get("q_row")), _ptr(o.get("s_row")), o["s_row"].stride(0) if "s_row" in o else 0,
                         _ptr(o.get("q_col")), _ptr(o.get("s_col")), o["s_col"].stride(0) if "s_col" in o else 0,
                         _stream_ptr(stream))
    return o


def layernorm_quantize(x, gamma, beta, eps: float = 1e-5, rowwise: bool = True, colwise: bool = False,
                       stream=None, out=None):
    """LayerNorm over the last axis of a 2-D bf16 CUDA tensor fused with its
    MXFP8 quantisation.  Returns a dict with q_row/s_row and/or q_col/s_col
    (as ``quantize``) and "mu" and "rsigma" (fp32 [rows])."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda and x.stride(1) == 1
    assert gamma.dtype == torch.bfloat16 and beta.dtype == torch.bfloat16
    rows, hidden = x.shape
    o = dict(out or {})
    if rowwise and "q_row" not in o:
        o["q_row"] = torch.empty(rows, hidden, dtype=torch.uint8, device=x.device)
        o["s_row"] = torch.empty(rows, te_mx_scale_pitch(hidden), dtype=torch.uint8, device=x.device)
    if colwise and "q_col" not in o:
        o["q_col"] = torch.empty(hidden, rows, dtype=torch.uint8, device=x.device)
        o["s_col"] = torch.empty(hidden, te_mx_scale_pitch(rows), dtype=torch.uint8, device=x.device)
    if "mu" not in o:
        o["mu"] = torch.empty(rows, dtype=torch.float32, device=x.device)
        o["rsigma"] = torch.empty(rows, dtype=torch.float32, device=x.device)
    te_mx_layernorm_quantize(x.data_ptr(), rows, hidden, x.stride(0), gamma.data_ptr(), beta.data_ptr(), float(eps),
                             _ptr(o.get("q_row")), _ptr(o.get("s_row")), o["s_row"].stride(0) if "s_row" in o else 0,
                             _ptr(o.get("q_col")), _ptr(o.get("s_col")), o["s_col"].stride(0) if "s_col" in o else 0,
                             _ptr(o.get("mu")), _ptr(o.get("rsigma")), _stream_ptr(stream))
    return o


class _DtypeCodes(dict):
    """te_mx_dtype by torch dtype, filled in on first use."""

    def __missing__(self, dtype):
        import torch
        self.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32})
        if dtype not in self:
            raise TypeError(f"{dtype} is none of bfloat16, float16 and float32")
        return self[dtype]


_dtype_code = _DtypeCodes()


def _pitch(t) -> int:
    """Row pitch of a 2-D tensor (a single row has no next one, whatever its stride says)."""
    rows, cols = t.shape
    ld, unit = t.stride()
    assert unit == 1 or cols == 1
    return ld if rows > 1 else max(ld, cols)


def _vectors(a, b, n: int, dtype, device: int) -> bool:
    """Whether a, and b if given, are contiguous vectors of n elements of that type on that CUDA device."""
    return all(t is None or (t.shape == (n,) and t.dtype == dtype and t.is_contiguous() and t.get_device() == device)
               for t in (a, b))


def layernorm(x, gamma, beta=None, eps: float = 1e-5, stats: bool = True, stream=None, out=None):
    """LayerNorm over the last axis of a 2-D bf16, fp16 or fp32 CUDA tensor;
    gamma and beta (None: no shift) have its type or fp32.  Returns a dict with
    "y" (the type of x) and, with ``stats``, "mu" and "rsigma" (fp32 [rows])
    for ``layernorm_backward``."""
    if stream is not None:
        with _on(stream):
            return layernorm(x, gamma, beta, eps=eps, stats=stats, out=out)
    torch = _torch or _load_torch()
    shape = x.shape
    rows, hidden = shape
    device = x.get_device()
    assert device >= 0 and gamma.get_device() == device and gamma.shape == shape[1:] and gamma.is_contiguous()
    b = 0
    if beta is not None:
        assert (beta.dtype == gamma.dtype and beta.shape == gamma.shape and beta.is_contiguous()
                and beta.get_device() == device)
        b = beta.data_ptr()
    if out is None:
        y, ld_y = torch.empty_like(x, memory_format=torch.contiguous_format), hidden
        o = {"y": y}
    else:
        o = dict(out)
        if "y" not in o:
            o["y"] = torch.empty_like(x, memory_format=torch.contiguous_format)
        y, ld_y = o["y"], _pitch(o["y"])
        assert y.shape == shape and y.dtype == x.dtype and y.get_device() == device
        assert stats or ("mu" in o) == ("rsigma" in o)     # (a lone one would be left unwritten)
        assert _vectors(o.get("mu"), o.get("rsigma"), rows, torch.float32, device)
    mu = rsigma = 0
    if stats:
        if "mu" not in o:
            o["mu"] = torch.empty(rows, dtype=torch.float32, device=x.device)
        if "rsigma" not in o:
            o["rsigma"] = torch.empty_like(o["mu"])
    if "mu" in o:
        mu, rsigma = o["mu"].data_ptr(), o["rsigma"].data_ptr()
    _check(lib().te_mx_layernorm(x.data_ptr(), rows, hidden, _pitch(x), _dtype_code[x.dtype], gamma.data_ptr(), b,
                                 _dtype_code[gamma.dtype], eps, y.data_ptr(), ld_y, mu, rsigma, _raw_stream()))
    return o


def layernorm_backward(dy, x, gamma, mu, rsigma, dparams: bool = True, stream=None, out=None, workspace=None):
    """Gradients of ``layernorm`` (or of the normalisation in
    ``layernorm_quantize``): dy and x [rows, hidden] of one type, mu and rsigma
    from the forward pass.  Returns a dict with "dx" and, with ``dparams``,
    "dgamma" and "dbeta" (the type of gamma); their scratch is ``workspace``
    (uint8 CUDA tensor) or allocated here."""
    if stream is not None:
        with _on(stream):
            return layernorm_backward(dy, x, gamma, mu, rsigma, dparams=dparams, out=out, workspace=workspace)
    torch = _torch or _load_torch()
    shape, dt = x.shape, _dtype_code[x.dtype]
    rows, hidden = shape
    device = x.get_device()
    assert device >= 0 and dy.get_device() == device and dy.shape == shape and dy.dtype == x.dtype
    assert gamma.shape == shape[1:] and gamma.is_contiguous() and mu.shape == rsigma.shape == shape[:1]
    assert mu.is_contiguous() and rsigma.is_contiguous() and mu.dtype == rsigma.dtype == torch.float32
    assert gamma.get_device() == mu.get_device() == rsigma.get_device() == device
    if out is None:
        dx, ld_dx = torch.empty_like(x, memory_format=torch.contiguous_format), hidden
        o = {"dx": dx}
    else:
        o = dict(out)
        if "dx" not in o:
            o["dx"] = torch.empty_like(x, memory_format=torch.contiguous_format)
        dx, ld_dx = o["dx"], _pitch(o["dx"])
        assert dx.shape == shape and dx.dtype == x.dtype and dx.get_device() == device
        assert dparams or "dgamma" in o or "dbeta" not in o       # (a lone dbeta would be left unwritten)
        assert _vectors(o.get("dgamma"), o.get("dbeta"), hidden, gamma.dtype, device)
    dga = dbe = ws = size = 0
    if dparams:
        if "dgamma" not in o:
            o["dgamma"] = torch.empty_like(gamma)
        if "dbeta" not in o:
            o["dbeta"] = torch.empty_like(gamma)
    if "dgamma" in o:
        dga, dbe = o["dgamma"].data_ptr(), _ptr(o.get("dbeta"))
        if workspace is None:
            workspace = torch.empty(lib().te_mx_layernorm_backward_workspace_size(rows, hidden), dtype=torch.uint8,
                                    device=x.device)
        else:
            assert workspace.get_device() == device and workspace.is_contiguous()
        ws, size = workspace.data_ptr(), workspace.numel()
    _check(lib().te_mx_layernorm_backward(dy.data_ptr(), _pitch(dy), x.data_ptr(), _pitch(x), rows, hidden, dt,
                                          gamma.data_ptr(), _dtype_code[gamma.dtype], mu.data_ptr(), rsigma.data_ptr(),
                                          dx.data_ptr(), ld_dx, dga, dbe, ws, size, _raw_stream()))
    return o


def quantize_colwise_grouped(x, group_m, stream=None, out=None):
    """Per-expert column-wise MXFP8 copy of the token-major bf16 CUDA tensor x
    [total_m, cols] (experts' rows in order, ``group_m``: int32 CUDA tensor of
    token counts).  Returns {"q": uint8 [cols, ld_q], "s": uint8 [cols, ld_s]}
    in the padded per-expert layout (widths from te_mx_grouped_*_width)."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda and x.stride(1) == 1
    assert group_m.dtype == torch.int32 and group_m.is_cuda
    total_m, cols = x.shape
    G = group_m.numel()
    o = dict(out or {})
    if "q" not in o:
        o["q"] = torch.empty(cols, te_mx_grouped_code_width(total_m, G), dtype=torch.uint8, device=x.device)
        o["s"] = torch.empty(cols, te_mx_grouped_scale_width(total_m, G), dtype=torch.uint8, device=x.device)
    te_mx_quantize_colwise_grouped(x.data_ptr(), total_m, cols, x.stride(0), G, group_m.data_ptr(), o["q"].data_ptr(),
                                   o["q"].stride(0), o["s"].data_ptr(), o["s"].stride(0), _stream_ptr(stream))
    return o


def grouped_gemm_wgrad(group_m, total_m, dy, x, stream=None, out=None, accumulate: bool = False):
    """dW_e = dY_e^T X_e for every expert: ``dy`` and ``x`` are the dicts of
    quantize_colwise_grouped of dY [total_m, M] and X [total_m, N] (same
    group_m).  Returns bf16 [G, M, N] (``out`` if given); with ``accumulate``,
    ``out`` is an fp32 [G, M, N] tensor that is added to."""
    import torch
    G = group_m.numel()
    M, N = dy["q"].shape[0], x["q"].shape[0]
    assert dy["q"].stride(0) == x["q"].stride(0) and dy["s"].stride(0) == x["s"].stride(0)
    if accumulate:
        assert out is not None and out.dtype == torch.float32
    d = out if out is not None else torch.empty(G, M, N, dtype=torch.bfloat16, device=dy["q"].device)
    te_mx_grouped_gemm_wgrad(G, group_m.data_ptr(), total_m, dy["q"].data_ptr(), dy["s"].data_ptr(), x["q"].data_ptr(),
                             x["s"].data_ptr(), M, N, dy["q"].stride(0), dy["s"].stride(0), int(bool(accumulate)),
                             d.data_ptr(), _stream_ptr(stream))
    return d


def gemm(qa, sa, qb, sb, bias=None, gelu: bool = False, stream=None, out=None, dgelu_aux=None,
         accumulate=None):
    """D = epilogue(deq(qa) . deq(qb)^T (+ bias)) in bf16; returns (D, aux or None).
    With ``dgelu_aux`` (bf16 [M, N], the forward pre-activation) the epilogue is
    D = bf16(acc * gelu'(dgelu_aux)).  With ``accumulate`` (an fp32 [M, N] CUDA
    tensor) it is accumulate += deq(qa) . deq(qb)^T in fp32."""
    import torch
    M, K = qa.shape
    N = qb.shape[0]
    if accumulate is not None:
        assert accumulate.dtype == torch.float32 and bias is None and not gelu and dgelu_aux is None
        te_mx_gemm(qa.data_ptr(), sa.data_ptr(), sa.stride(0), qb.data_ptr(), sb.data_ptr(), sb.stride(0),
                   M, N, K, 0, EPI_ACCUMULATE_F32, accumulate.data_ptr(), 0, 0, 0, _stream_ptr(stream))
        return accumulate, None
    epi = (EPI_BIAS if bias is not None else EPI_NONE) + (EPI_GELU_AUX if gelu else 0)
    if dgelu_aux is not None:
        assert bias is None and not gelu
        d = torch.empty(M, N, dtype=torch.bfloat16, device=qa.device) if out is None else out[0]
        te_mx_gemm(qa.data_ptr(), sa.data_ptr(), sa.stride(0), qb.data_ptr(), sb.data_ptr(), sb.stride(0),
                   M, N, K, 0, EPI_DGELU, d.data_ptr(), dgelu_aux.data_ptr(), 0, 0, _stream_ptr(stream))
        return d, None
    if out is None:
        d = torch.empty(M, N, dtype=torch.bfloat16, device=qa.device)
        aux = torch.empty(M, N, dtype=torch.bfloat16, device=qa.device) if gelu else None
    else:
        d, aux = out
    te_mx_gemm(qa.data_ptr(), sa.data_ptr(), sa.stride(0), qb.data_ptr(), sb.data_ptr(), sb.stride(0),
               M, N, K, _ptr(bias), epi, d.data_ptr(), _ptr(aux), 0, 0, _stream_ptr(stream))
    return d, aux


def te_mx_gemm_fp32_scales(A, sA, ld_sA, B, sB, ld_sB, b_blocks_2d, M, N, K, bias, epilogue, D, aux,
                           stream) -> None:
    _check(lib().te_mx_gemm_fp32_scales(A, sA, ld_sA, B, sB, ld_sB, b_blocks_2d, M, N, K, bias, epilogue, D, aux,
                                        stream))


def gemm_fp32_scales(qa, sa, qb, sb, b_blocks_2d: bool, bias=None, gelu: bool = False, stream=None, out=None,
                     dgelu_aux=None):
    """Float8BlockScaling GEMM with FP32 scales (``block_quantize_fp32``
    output; ``b_blocks_2d`` for 128x128 weight blocks): D = epilogue(sum over
    128-long K blocks of sA sB A_kb . B_kb^T (+ bias)); returns (D, aux or None).
    With ``dgelu_aux`` the epilogue is the GELU backward (see ``gemm``)."""
    import torch
    M, K = qa.shape
    N = qb.shape[0]
    epi = (EPI_BIAS if bias is not None else EPI_NONE) + (EPI_GELU_AUX if gelu else 0)
    aux = None
    if dgelu_aux is not None:
        assert bias is None and not gelu
        epi = EPI_DGELU
    if out is None:
        d = torch.empty(M, N, dtype=torch.bfloat16, device=qa.device)
        if gelu:
            aux = torch.empty(M, N, dtype=torch.bfloat16, device=qa.device)
    else:
        d, aux = out
    aux_ptr = dgelu_aux.data_ptr() if dgelu_aux is not None else _ptr(aux)
    te_mx_gemm_fp32_scales(qa.data_ptr(), sa.data_ptr(), sa.stride(0), qb.data_ptr(), sb.data_ptr(), sb.stride(0),
                           int(bool(b_blocks_2d)), M, N, K, _ptr(bias), epi, d.data_ptr(), aux_ptr,
                           _stream_ptr(stream))
    return d, (aux if dgelu_aux is None else None)


def grouped_gemm(group_m, qx, sx, qw, sw, bias=None, gelu: bool = False, stream=None, out=None, dgelu_aux=None):
    """Grouped GEMM over experts: group_m int32 [G] on the device, qx [total_m, K],
    qw [G, N, K], sw [G*N, pitch]; returns (D, aux or None) of [total_m, N].
    With ``dgelu_aux`` the epilogue is the GELU backward (see ``gemm``)."""
    import torch
    total_m, K = qx.shape
    G, N, _ = qw.shape
    epi = (EPI_BIAS if bias is not None else EPI_NONE) + (EPI_GELU_AUX if gelu else 0)
    if dgelu_aux is not None:
        assert bias is None and not gelu
        d = torch.empty(total_m, N, dtype=torch.bfloat16, device=qx.device) if out is None else out[0]
        sw2 = sw.reshape(G * N, -1)
        te_mx_grouped_gemm(G, group_m.data_ptr(), total_m, qx.data_ptr(), sx.data_ptr(), sx.stride(0),
                           qw.data_ptr(), sw2.data_ptr(), sw2.stride(0), N, K, 0, EPI_DGELU,
                           d.data_ptr(), dgelu_aux.data_ptr(), 0, 0, _stream_ptr(stream))
        return d, None
    if out is None:
        d = torch.empty(total_m, N, dtype=torch.bfloat16, device=qx.device)
        aux = torch.empty(total_m, N, dtype=torch.bfloat16, device=qx.device) if gelu else None
    else:
        d, aux = out
    sw2 = sw.reshape(G * N, -1)
    te_mx_grouped_gemm(G, group_m.data_ptr(), total_m, qx.data_ptr(), sx.data_ptr(), sx.stride(0),
                       qw.data_ptr(), sw2.data_ptr(), sw2.stride(0), N, K, _ptr(bias), epi,
                       d.data_ptr(), _ptr(aux), 0, 0, _stream_ptr(stream))
    return d, aux


def _mx_operand(q, s, rows: int, cols: int, device: int) -> bool:
    """Whether q and s are an MXFP8 operand's contiguous codes and scale rows (a scale
    per 32 codes, at least) on that CUDA device."""
    n, width = s.shape
    return (n == rows and 32 * width >= cols and q.get_device() == s.get_device() == device
            and q.is_contiguous() and q.element_size() == s.element_size() == 1)


def _matrix(t, rows: int, cols: int, dtype, device: int) -> bool:
    return t is None or (t.shape == (rows, cols) and t.dtype == dtype and t.is_contiguous() and t.get_device() == device)


def _bytes(t, rows: int, cols: int, device: int) -> bool:
    """Whether t, if given, is a matrix of bytes on that CUDA device with that many
    rows and at least so many columns (what it has more is left alone)."""
    return t is None or (t.dim() == 2 and t.shape[0] == rows and t.shape[1] >= cols and t.element_size() == 1
                         and t.get_device() == device)


def _bias(t, n: int, dtype, device: int) -> bool:
    return t.dtype == dtype and t.numel() == n and t.is_contiguous() and t.get_device() == device


def gated_gemm(qx, sx, qw, sw, activation: str = "silu", bias=None, aux: bool = False, stream=None, out=None):
    """Gated feed-forward of MXFP8 operands: qx [M, K] and qw [2F, K] (the gate
    weight's rows, then the up weight's; ``quantize``'s row-wise copies), bias
    bf16 [2F] or None, activation "silu", "gelu" (tanh form) or "relu".
    Returns (h, pre): h = act(gate) * up in bf16 [M, F], and with ``aux`` the
    pre-activations [gate | up] in bf16 [M, 2F] for ``gated_backward``, else None."""
    if stream is not None:
        with _on(stream):
            return gated_gemm(qx, sx, qw, sw, activation=activation, bias=bias, aux=aux, out=out)
    torch = _torch or _load_torch()
    M, K = qx.shape
    F = qw.shape[0] // 2
    device = qx.get_device()
    assert device >= 0 and qw.shape == (2 * F, K) and _mx_operand(qx, sx, M, K, device) and _mx_operand(qw, sw, 2 * F, K, device)
    assert bias is None or _bias(bias, 2 * F, torch.bfloat16, device)
    if out is None:
        h = torch.empty(M, F, dtype=torch.bfloat16, device=qx.device)
        pre = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=qx.device) if aux else None
    else:
        h, pre = out
        assert _matrix(h, M, F, torch.bfloat16, device) and _matrix(pre, M, 2 * F, torch.bfloat16, device)
    te_mx_gated_gemm(qx.data_ptr(), sx.data_ptr(), _pitch(sx), qw.data_ptr(), sw.data_ptr(), _pitch(sw), M, F, K,
                     _ptr(bias), ACTIVATIONS[activation], h.data_ptr(), _ptr(pre), _raw_stream())
    return h, pre


def grouped_gated_gemm(group_m, qx, sx, qw, sw, activation: str = "silu", bias=None, aux: bool = False, stream=None,
                       out=None):
    """``gated_gemm`` over the experts of a mixture: group_m int32 [G] on the
    device, qx [total_m, K] (the experts' rows in order), qw [G, 2F, K], sw
    [G*2F, pitch], bias bf16 [G, 2F] or None.  Returns (h [total_m, F], pre
    [total_m, 2F] or None)."""
    if stream is not None:
        with _on(stream):
            return grouped_gated_gemm(group_m, qx, sx, qw, sw, activation=activation, bias=bias, aux=aux, out=out)
    torch = _torch or _load_torch()
    total_m, K = qx.shape
    G, N, _ = qw.shape
    sw2 = sw.reshape(G * N, -1)
    assert group_m.dtype == torch.int32 and group_m.numel() == G and N % 2 == 0 and qw.shape[2] == K
    device = qx.get_device()
    assert device >= 0 and group_m.get_device() == device and group_m.is_contiguous()
    assert _mx_operand(qx, sx, total_m, K, device) and _mx_operand(qw, sw2, G * N, K, device)
    assert bias is None or _bias(bias, G * N, torch.bfloat16, device)
    if out is None:
        h = torch.empty(total_m, N // 2, dtype=torch.bfloat16, device=qx.device)
        pre = torch.empty(total_m, N, dtype=torch.bfloat16, device=qx.device) if aux else None
    else:
        h, pre = out
        assert _matrix(h, total_m, N // 2, torch.bfloat16, device) and _matrix(pre, total_m, N, torch.bfloat16, device)
    te_mx_grouped_gated_gemm(G, group_m.data_ptr(), total_m, qx.data_ptr(), sx.data_ptr(), _pitch(sx), qw.data_ptr(),
                             sw2.data_ptr(), _pitch(sw2), N // 2, K, _ptr(bias), ACTIVATIONS[activation], h.data_ptr(),
                             _ptr(pre), _raw_stream())
    return h, pre


def gated_backward(dh, gate_up, activation: str = "silu", dense: bool = False, rowwise: bool = True, colwise: bool = True,
                   stream=None, out=None):
    """Gradient of the gated feed-forward's pre-activations: dh bf16 [M, F] and
    gate_up bf16 [M, 2F] (the ``pre`` of ``gated_gemm``).  Returns a dict with
    "d_gate_up" (bf16 [M, 2F], with ``dense``), "q_row"/"s_row" (its row-wise
    MXFP8 copy) and "q_col"/"s_col" (its column-wise copy [2F, Kp], the tokens
    zero-padded to Kp, M rounded up to 128), so that
    dX = gemm(q_row, s_row, W's column-wise copy) and
    dW = gemm(q_col, s_col, X's column-wise copy, padded likewise)."""
    if stream is not None:
        with _on(stream):
            return gated_backward(dh, gate_up, activation=activation, dense=dense, rowwise=rowwise, colwise=colwise,
                                  out=out)
    torch = _torch or _load_torch()
    device = dh.get_device()
    assert dh.dtype == gate_up.dtype == torch.bfloat16 and dh.dim() == gate_up.dim() == 2
    assert device >= 0 and gate_up.get_device() == device
    M, F = dh.shape
    assert gate_up.shape == (M, 2 * F) and dh.stride(1) == gate_up.stride(1) == 1
    o = dict(out or {})
    dev, u8, kp = dh.device, torch.uint8, (M + 127) // 128 * 128
    if o:
        d, q = o.get("d_gate_up"), o.get("q_row")
        assert d is None or (d.shape == (M, 2 * F) and d.dtype == torch.bfloat16 and d.get_device() == device)
        assert q is None or (q.shape == (M, 2 * F) and q.is_contiguous())
        assert _bytes(q, M, 2 * F, device) and _bytes(o.get("s_row"), M, F // 16, device)
        assert _bytes(o.get("q_col"), 2 * F, kp, device) and _bytes(o.get("s_col"), 2 * F, kp // 32, device)
        # (lone codes or scales would be left unwritten)
        assert (rowwise or ("q_row" in o) == ("s_row" in o)) and (colwise or ("q_col" in o) == ("s_col" in o))
    if dense and "d_gate_up" not in o:
        o["d_gate_up"] = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev)
    if rowwise:
        if "q_row" not in o:
            o["q_row"] = torch.empty((M, 2 * F), dtype=u8, device=dev)
        if "s_row" not in o:
            o["s_row"] = torch.empty((M, (F // 16 + 15) // 16 * 16), dtype=u8, device=dev)
    if colwise:
        if "q_col" not in o:
            o["q_col"] = torch.empty((2 * F, kp), dtype=u8, device=dev)
        if "s_col" not in o:
            o["s_col"] = torch.empty((2 * F, (kp // 32 + 15) // 16 * 16), dtype=u8, device=dev)
    d = d_ld = q_row = s_row = s_row_ld = q_col = q_col_ld = s_col = s_col_ld = 0
    if "d_gate_up" in o:
        d, d_ld = o["d_gate_up"].data_ptr(), _pitch(o["d_gate_up"])
    if "q_row" in o:
        q_row, s_row, s_row_ld = o["q_row"].data_ptr(), o["s_row"].data_ptr(), _pitch(o["s_row"])
    if "q_col" in o:
        q_col, q_col_ld = o["q_col"].data_ptr(), _pitch(o["q_col"])
        s_col, s_col_ld = o["s_col"].data_ptr(), _pitch(o["s_col"])
    _check(lib().te_mx_gated_backward(dh.data_ptr(), _pitch(dh), gate_up.data_ptr(), _pitch(gate_up), M, F,
                                      ACTIVATIONS[activation], d, d_ld, q_row, s_row, s_row_ld, q_col, q_col_ld, s_col,
                                      s_col_ld, _raw_stream()))
    return o


def _like(t, shape, dtype, device: int) -> bool:
    """Whether t, if given, is a 2-D tensor of that shape and type, its rows contiguous, on that CUDA device."""
    return t is None or (t.shape == shape and t.dtype == dtype and t.get_device() == device)


def _vector(t, n: int, dtype, device: int) -> bool:
    """Whether t, if given, is a contiguous vector of n elements of that type on that CUDA device."""
    return t is None or (t.shape == (n,) and t.dtype == dtype and t.get_device() == device and t.is_contiguous())


def rmsnorm(x, gamma, eps: float = 1e-5, residual=None, stats: bool = True, stream=None, out=None):
    """RMSNorm over the last axis of a 2-D bf16, fp16 or fp32 CUDA tensor, of
    z = x + residual if one is given; gamma has its type or fp32.  Returns a dict
    with "y" (the type of x), "z" (with a residual; the sum, rounded) and, with
    ``stats``, "rsigma" (fp32 [rows]) for ``rmsnorm_backward``."""
    if stream is not None:
        with _on(stream):
            return rmsnorm(x, gamma, eps=eps, residual=residual, stats=stats, out=out)
    torch = _torch or _load_torch()
    shape, dtype = x.shape, x.dtype
    rows, hidden = shape
    device = x.get_device()
    assert device >= 0 and device == _current_device() and gamma.get_device() == device and gamma.shape == shape[1:] and gamma.is_contiguous()
    o = {} if out is None else dict(out)
    if o:
        assert _like(o.get("y"), shape, dtype, device) and _like(o.get("z"), shape, dtype, device)
        assert _vector(o.get("rsigma"), rows, torch.float32, device)
    if "y" not in o:
        o["y"] = torch.empty_like(x, memory_format=torch.contiguous_format)
    res = ld_res = z = ld_z = rs = 0
    if residual is not None:
        assert _like(residual, shape, dtype, device)
        if "z" not in o:
            o["z"] = torch.empty_like(x, memory_format=torch.contiguous_format)
        v = o["z"]
        res, ld_res = residual.data_ptr(), hidden if residual.is_contiguous() else _pitch(residual)
        z, ld_z = v.data_ptr(), hidden if v.is_contiguous() else _pitch(v)
    else:
        assert "z" not in o                                    # (it would be left unwritten)
    if stats and "rsigma" not in o:
        o["rsigma"] = torch.empty(rows, dtype=torch.float32, device=x.device)
    if "rsigma" in o:
        rs = o["rsigma"].data_ptr()
    y = o["y"]
    _check(lib().te_mx_rmsnorm(x.data_ptr(), rows, hidden, hidden if x.is_contiguous() else _pitch(x), _dtype_code[dtype],
                               res, ld_res, gamma.data_ptr(), _dtype_code[gamma.dtype], eps, z, ld_z, y.data_ptr(),
                               hidden if y.is_contiguous() else _pitch(y), rs, _raw_stream()))
    return o


def rmsnorm_quantize(x, gamma, eps: float = 1e-5, residual=None, rowwise: bool = True, colwise: bool = False,
                     dense: bool = False, stream=None, out=None):
    """``rmsnorm`` of a 2-D bf16 CUDA tensor with its MXFP8 quantisation; gamma
    has bf16 or fp32.  Returns a dict with q_row/s_row and/or q_col/s_col (as
    ``quantize``), "rsigma" (fp32 [rows]), "z" (with a residual) and, with
    ``dense``, "y" in bf16."""
    if stream is not None:
        with _on(stream):
            return rmsnorm_quantize(x, gamma, eps=eps, residual=residual, rowwise=rowwise, colwise=colwise, dense=dense,
                                    out=out)
    torch = _torch or _load_torch()
    shape, bf16, u8, dev = x.shape, torch.bfloat16, torch.uint8, x.device
    rows, hidden = shape
    device = x.get_device()
    assert device >= 0 and device == _current_device() and x.dtype == bf16
    assert gamma.get_device() == device and gamma.shape == shape[1:] and gamma.is_contiguous()
    o = {} if out is None else dict(out)
    if o:
        q = o.get("q_row")
        assert (rowwise or ("q_row" in o) == ("s_row" in o)) and (colwise or ("q_col" in o) == ("s_col" in o))
        assert q is None or (q.shape == shape and q.is_contiguous())
        assert _bytes(q, rows, hidden, device) and _bytes(o.get("s_row"), rows, hidden // 32, device)
        q = o.get("q_col")
        assert q is None or (q.shape == (hidden, rows) and q.is_contiguous())
        assert _bytes(q, hidden, rows, device) and _bytes(o.get("s_col"), hidden, rows // 32, device)
        assert _like(o.get("y"), shape, bf16, device) and _like(o.get("z"), shape, bf16, device)
        assert _vector(o.get("rsigma"), rows, torch.float32, device)
    if rowwise:
        if "q_row" not in o:
            o["q_row"] = torch.empty(shape, dtype=u8, device=dev)
        if "s_row" not in o:
            o["s_row"] = torch.empty((rows, (hidden // 32 + 15) // 16 * 16), dtype=u8, device=dev)
    if colwise:
        if "q_col" not in o:
            o["q_col"] = torch.empty((hidden, rows), dtype=u8, device=dev)
        if "s_col" not in o:
            o["s_col"] = torch.empty((hidden, (rows // 32 + 15) // 16 * 16), dtype=u8, device=dev)
    if dense and "y" not in o:
        o["y"] = torch.empty_like(x, memory_format=torch.contiguous_format)
    if "rsigma" not in o:
        o["rsigma"] = torch.empty(rows, dtype=torch.float32, device=dev)
    res = ld_res = z = ld_z = y = ld_y = q_row = s_row = ld_row = q_col = s_col = ld_col = 0
    if residual is not None:
        assert _like(residual, shape, bf16, device)
        if "z" not in o:
            o["z"] = torch.empty_like(x, memory_format=torch.contiguous_format)
        v = o["z"]
        res, ld_res = residual.data_ptr(), hidden if residual.is_contiguous() else _pitch(residual)
        z, ld_z = v.data_ptr(), hidden if v.is_contiguous() else _pitch(v)
    else:
        assert "z" not in o                                    # (it would be left unwritten)
    if "y" in o:
        v = o["y"]
        y, ld_y = v.data_ptr(), hidden if v.is_contiguous() else _pitch(v)
    if "q_row" in o:
        q_row, s_row, ld_row = o["q_row"].data_ptr(), o["s_row"].data_ptr(), _pitch(o["s_row"])
    if "q_col" in o:
        q_col, s_col, ld_col = o["q_col"].data_ptr(), o["s_col"].data_ptr(), _pitch(o["s_col"])
    _check(lib().te_mx_rmsnorm_quantize(x.data_ptr(), rows, hidden, hidden if x.is_contiguous() else _pitch(x), res, ld_res, gamma.data_ptr(),
                                        _dtype_code[gamma.dtype], eps, z, ld_z, y, ld_y, q_row, s_row, ld_row, q_col,
                                        s_col, ld_col, o["rsigma"].data_ptr(), _raw_stream()))
    return o


def rmsnorm_backward(dy, z, gamma, rsigma, dz=None, dparams: bool = True, stream=None, out=None, workspace=None):
    """Gradients of ``rmsnorm`` and ``rmsnorm_quantize``: dy and z [rows, hidden]
    of one type (z is x where there was no residual), rsigma from the forward
    pass, dz the gradient that reaches z by the residual path (None: zero).
    Returns a dict with "dx" (of x and of the residual alike) and, with
    ``dparams``, "dgamma" (the type of gamma); its scratch is ``workspace`` (uint8
    CUDA tensor) or allocated here."""
    if stream is not None:
        with _on(stream):
            return rmsnorm_backward(dy, z, gamma, rsigma, dz=dz, dparams=dparams, out=out, workspace=workspace)
    torch = _torch or _load_torch()
    shape, dtype = z.shape, z.dtype
    rows, hidden = shape
    device = z.get_device()
    assert device >= 0 and device == _current_device() and _like(dy, shape, dtype, device) and _like(dz, shape, dtype, device)
    assert gamma.shape == shape[1:] and gamma.is_contiguous() and gamma.get_device() == device
    assert _vector(rsigma, rows, torch.float32, device)
    o = {} if out is None else dict(out)
    if o:
        assert _like(o.get("dx"), shape, dtype, device) and _vector(o.get("dgamma"), hidden, gamma.dtype, device)
    if "dx" not in o:
        o["dx"] = torch.empty_like(z, memory_format=torch.contiguous_format)
    if dparams and "dgamma" not in o:
        o["dgamma"] = torch.empty_like(gamma)
    dga = ws = size = 0
    if "dgamma" in o:
        dga = o["dgamma"].data_ptr()
        if workspace is None:
            workspace = torch.empty(lib().te_mx_rmsnorm_backward_workspace_size(rows, hidden), dtype=torch.uint8,
                                    device=z.device)
        else:
            assert workspace.dtype == torch.uint8 and workspace.get_device() == device and workspace.is_contiguous()
        ws, size = workspace.data_ptr(), workspace.numel()
    dx, res, ld_res = o["dx"], 0, 0
    if dz is not None:
        res, ld_res = dz.data_ptr(), hidden if dz.is_contiguous() else _pitch(dz)
    _check(lib().te_mx_rmsnorm_backward(dy.data_ptr(), hidden if dy.is_contiguous() else _pitch(dy), z.data_ptr(),
                                        hidden if z.is_contiguous() else _pitch(z), rows, hidden, _dtype_code[dtype],
                                        gamma.data_ptr(), _dtype_code[gamma.dtype], rsigma.data_ptr(), res, ld_res,
                                        dx.data_ptr(), hidden if dx.is_contiguous() else _pitch(dx), dga, ws, size,
                                        _raw_stream()))
    return o


def route(logits, k: int, scoring: str = "softmax", renormalise: bool = True, scale: float = 1.0, bias=None, stream=None,
          out=None):
    """The k experts of each token (logits [tokens, experts], bf16, fp16 or fp32)
    with the largest logit + bias (bias fp32 [experts] or None; it chooses only),
    ties to the lowest index, and their weights: ``scale`` times the softmax (or
    "sigmoid") of the logits, with ``renormalise`` over the chosen ones.  Returns
    {"index": int32 [tokens, k], "weight": fp32 [tokens, k]}."""
    if stream is not None:
        with _on(stream):
            return route(logits, k, scoring=scoring, renormalise=renormalise, scale=scale, bias=bias, out=out)
    torch = _torch or _load_torch()
    tokens, experts = logits.shape
    device = logits.get_device()
    assert device >= 0 and device == _current_device() and _vector(bias, experts, torch.float32, device)
    o = {} if out is None else dict(out)
    if o:
        assert _matrix(o.get("index"), tokens, k, torch.int32, device)
        assert _matrix(o.get("weight"), tokens, k, torch.float32, device)
    if "index" not in o:
        o["index"] = torch.empty((tokens, k), dtype=torch.int32, device=logits.device)
    if "weight" not in o:
        o["weight"] = torch.empty((tokens, k), dtype=torch.float32, device=logits.device)
    ld = experts if logits.is_contiguous() else _pitch(logits)
    _check(lib().te_mx_route(logits.data_ptr(), tokens, experts, ld, _dtype_code[logits.dtype],
                             0 if bias is None else bias.data_ptr(), k, SCORINGS[scoring], int(bool(renormalise)), scale,
                             o["index"].data_ptr(), o["weight"].data_ptr(), _raw_stream()))
    return o


def route_backward(dweight, logits, index, scoring: str = "softmax", renormalise: bool = True, scale: float = 1.0,
                   stream=None, out=None):
    """The gradient of ``route``'s logits (their type, [tokens, experts]) from that
    of its weights (fp32 [tokens, k]); index and the options as in the forward
    call.  A choice dropped after the weights were made keeps its index here, with
    a dweight of 0 (``moe_combine_backward`` gives it that): its score is part of the
    sum that divided the others.  A negative index is a choice that was never made."""
    if stream is not None:
        with _on(stream):
            return route_backward(dweight, logits, index, scoring=scoring, renormalise=renormalise, scale=scale, out=out)
    torch = _torch or _load_torch()
    tokens, experts = logits.shape
    k = index.shape[1]
    device = logits.get_device()
    assert device >= 0 and device == _current_device()
    assert _matrix(index, tokens, k, torch.int32, device) and _matrix(dweight, tokens, k, torch.float32, device)
    assert _like(out, logits.shape, logits.dtype, device)
    d = torch.empty_like(logits, memory_format=torch.contiguous_format) if out is None else out
    ld = experts if logits.is_contiguous() else _pitch(logits)
    _check(lib().te_mx_route_backward(dweight.data_ptr(), logits.data_ptr(), ld, index.data_ptr(), tokens, experts,
                                      _dtype_code[logits.dtype], k, SCORINGS[scoring], int(bool(renormalise)), scale,
                                      d.data_ptr(), experts if d.is_contiguous() else _pitch(d), _raw_stream()))
    return d


def moe_sort(index, experts: int, stream=None, out=None):
    """Slots sorted by expert: index int32 [tokens, k] (or any shape; a negative
    one has no row).  Returns {"group_m": int32 [experts], the experts' row counts
    (``grouped_gemm``'s group_m), "row": the row of each slot (the shape of index,
    -1 without one), "slot": int32 [slots], the slot of each row (-1 behind the
    last)}."""
    if stream is not None:
        with _on(stream):
            return moe_sort(index, experts, out=out)
    torch = _torch or _load_torch()
    device, n, i32 = index.get_device(), index.numel(), torch.int32
    assert device >= 0 and device == _current_device() and index.dtype == i32 and index.is_contiguous()
    o = {} if out is None else dict(out)
    if o:
        r = o.get("row")
        assert r is None or (r.shape == index.shape and r.dtype == i32 and r.is_contiguous() and r.get_device() == device)
        assert _vector(o.get("group_m"), experts, i32, device) and _vector(o.get("slot"), n, i32, device)
    if "group_m" not in o:
        o["group_m"] = torch.empty(experts, dtype=i32, device=index.device)
    if "row" not in o:
        o["row"] = torch.empty_like(index)
    if "slot" not in o:
        o["slot"] = torch.empty(n, dtype=i32, device=index.device)
    _check(lib().te_mx_moe_sort(index.data_ptr(), n, experts, o["group_m"].data_ptr(), o["row"].data_ptr(),
                                o["slot"].data_ptr(), _raw_stream()))
    return o


def moe_dispatch(x, row, scales=None, total_rows=None, stream=None, out=None):
    """Every token's row copied to the rows of its slots: x [tokens, hidden] of any
    type (or MXFP8 codes, with their ``scales`` [tokens, pitch]), row int32
    [tokens, k] (``moe_sort``).  Returns out [total_rows, hidden] (tokens * k rows
    if not said), or (out, out_scales); rows without a slot are not written.  Its
    gradient is ``moe_combine`` without weights."""
    if stream is not None:
        with _on(stream):
            return moe_dispatch(x, row, scales=scales, total_rows=total_rows, out=out)
    torch = _torch or _load_torch()
    tokens, hidden = x.shape
    k = row.shape[1]
    device, size = x.get_device(), x.element_size()
    assert device >= 0 and device == _current_device() and _matrix(row, tokens, k, torch.int32, device)
    s = ld_s = width = d_s = ld_ds = 0
    if scales is not None:
        width = hidden // 32
        assert size == 1 and hidden % 32 == 0 and _bytes(scales, tokens, width, device)
    if out is None:
        m = tokens * k if total_rows is None else total_rows
        d = torch.empty((m, hidden), dtype=x.dtype, device=x.device)
        ds = None if scales is None else torch.empty((m, (width + 15) // 16 * 16), dtype=scales.dtype, device=x.device)
    else:
        d, ds = out if scales is not None else (out, None)
        m = d.shape[0]
        assert (total_rows is None or total_rows == m) and _like(d, (m, hidden), x.dtype, device)
        assert _bytes(ds, m, width, device)
    if scales is not None:
        s, ld_s, d_s, ld_ds = scales.data_ptr(), _pitch(scales), ds.data_ptr(), _pitch(ds)
    ld_x, ld_d = hidden if x.is_contiguous() else _pitch(x), hidden if d.is_contiguous() else _pitch(d)
    _check(lib().te_mx_moe_dispatch(x.data_ptr(), ld_x * size, hidden * size, s, ld_s, width, row.data_ptr(), tokens, k, m,
                                    d.data_ptr(), ld_d * size, d_s, ld_ds, _raw_stream()))
    return d if scales is None else (d, ds)


def moe_combine(y, row, weight=None, residual=None, stream=None, out=None):
    """out[t] = sum_j weight[t, j] y[row[t, j]] + residual[t]: y [rows, hidden] of
    bf16, fp16 or fp32, row int32 [tokens, k] (a negative one is skipped), weight
    fp32 [tokens, k] or None (all 1: the gradient of ``moe_dispatch``), residual
    [tokens, hidden] or None.  Returns out [tokens, hidden] in the type of y."""
    if stream is not None:
        with _on(stream):
            return moe_combine(y, row, weight=weight, residual=residual, out=out)
    torch = _torch or _load_torch()
    rows, hidden = y.shape
    tokens, k = row.shape
    device = y.get_device()
    assert device >= 0 and device == _current_device()
    assert _matrix(row, tokens, k, torch.int32, device) and _matrix(weight, tokens, k, torch.float32, device)
    assert _like(residual, (tokens, hidden), y.dtype, device) and _like(out, (tokens, hidden), y.dtype, device)
    d = torch.empty((tokens, hidden), dtype=y.dtype, device=y.device) if out is None else out
    w = res = ld_res = 0
    if weight is not None:
        w = weight.data_ptr()
    if residual is not None:
        res, ld_res = residual.data_ptr(), hidden if residual.is_contiguous() else _pitch(residual)
    _check(lib().te_mx_moe_combine(y.data_ptr(), hidden if y.is_contiguous() else _pitch(y), rows, hidden, _dtype_code[y.dtype],
                                   row.data_ptr(), tokens, k, w, res, ld_res, d.data_ptr(),
                                   hidden if d.is_contiguous() else _pitch(d), _raw_stream()))
    return d


def moe_combine_backward(dout, y, row, weight, dweight: bool = True, stream=None, out=None):
    """Gradients of ``moe_combine``: dout [tokens, hidden], y, row and weight of the
    forward call.  Returns a dict with "dy" [rows, hidden] (rows without a slot are
    not written) and, with ``dweight``, "dweight" (fp32 [tokens, k], 0 for a slot
    without a row)."""
    if stream is not None:
        with _on(stream):
            return moe_combine_backward(dout, y, row, weight, dweight=dweight, out=out)
    torch = _torch or _load_torch()
    rows, hidden = y.shape
    tokens, k = row.shape
    device = y.get_device()
    assert device >= 0 and device == _current_device()
    assert _matrix(row, tokens, k, torch.int32, device) and _matrix(weight, tokens, k, torch.float32, device)
    assert weight is not None and _like(dout, (tokens, hidden), y.dtype, device)
    o = {} if out is None else dict(out)
    if o:
        assert _like(o.get("dy"), y.shape, y.dtype, device) and _matrix(o.get("dweight"), tokens, k, torch.float32, device)
    if "dy" not in o:
        o["dy"] = torch.empty_like(y, memory_format=torch.contiguous_format)
    if dweight and "dweight" not in o:
        o["dweight"] = torch.empty_like(weight)
    dy = o["dy"]
    _check(lib().te_mx_moe_combine_backward(dout.data_ptr(), hidden if dout.is_contiguous() else _pitch(dout), y.data_ptr(),
                                            hidden if y.is_contiguous() else _pitch(y), rows, hidden, _dtype_code[y.dtype],
                                            row.data_ptr(), weight.data_ptr(), tokens, k, dy.data_ptr(),
                                            hidden if dy.is_contiguous() else _pitch(dy), _ptr(o.get("dweight")),
                                            _raw_stream()))
    return o
