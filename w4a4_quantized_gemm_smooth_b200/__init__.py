"""Python binding of the SVDQuant W4A4 linear-layer library (libsvdq.so).

Argument marshalling only: every step of the layer runs in the C-ABI
library (host pack code and sm_100a kernels).  PyTorch supplies device
memory and the current CUDA stream.  The binding never falls back to another
implementation: if the library is missing it raises.

The call names follow include/svdq.h:
    svdq_calib_absmax, svdq_pack_weights, svdq_pack_weights_host,
    svdq_weights_export, svdq_weights_save, svdq_weights_load,
    svdq_quantize_act, svdq_linear, svdq_get_device_error,
    svdq_debug_partials, svdq_linear_splitk*, svdq_pack_weights_calibrated,
    the W8A8 comparator svdq_pack_weights_w8a8, svdq_quantize_act_w8a8,
    svdq_linear_w8a8, and the NVFP4 variant svdq_pack_weights_nvfp4,
    svdq_quantize_act_nvfp4, svdq_linear_nvfp4, and the cross-layer fusion
    svdq_linear_quantize_next,
    the 16-bit operators around the quantised layers svdq_linear16,
    svdq_layer_norm, svdq_rope (with svdq_rope_create) and the gradients
    svdq_linear16_backward, svdq_layer_norm_backward, and svdq_get_op_error
and SVDQLinear / W8A8Linear / NVFP4Linear bundle one packed layer with its
two hot-path calls; SVDQMLP chains two layers (fc1, GELU, fc2) with or
without the fusion, behind a layer norm if one is given; SVDQQKV chains a
norm, a packed QKV layer and the rotary positions of its queries and keys;
Linear16 and LayerNorm bundle a 16-bit operator with its buffers and its
gradient.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

__all__ = [
    "lib", "SVDQError", "Weights", "SVDQLinear", "svdq_calib_absmax",
    "svdq_pack_weights", "svdq_pack_weights_host", "svdq_weights_load",
    "svdq_quantize_act", "svdq_linear", "svdq_get_device_error",
    "svdq_debug_partials", "EPI_NONE", "EPI_GELU", "LIB_PATH",
    "svdq_pack_weights_w8a8", "svdq_quantize_act_w8a8", "svdq_linear_w8a8", "W8A8Linear",
    "FORMAT_W4A4", "FORMAT_W8A8", "FORMAT_NVFP4", "svdq_pack_weights_nvfp4",
    "svdq_quantize_act_nvfp4", "svdq_linear_nvfp4", "svdq_nvfp4_sf_bytes", "NVFP4Linear",
    "svdq_linear_quantize_next", "svdq_linear_quantize_next_workspace", "SVDQMLP",
    "svdq_linear_host", "svdq_linear_host_workspace",
    "EPI_SILU", "svdq_linear16", "svdq_linear16_backward", "svdq_linear16_backward_workspace",
    "svdq_debug_linear16_forms", "svdq_get_op_error", "svdq_layer_norm", "svdq_layer_norm_backward",
    "svdq_layer_norm_backward_workspace", "ROPE_INTERLEAVED", "ROPE_HALVES", "RopePlan",
    "svdq_rope_create", "svdq_rope", "rope_frequencies", "Linear16", "LayerNorm", "SVDQQKV",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libsvdq.so")
EPI_NONE = 0
EPI_GELU = 1
EPI_SILU = 2        # 16-bit products only
ROPE_INTERLEAVED = 0
ROPE_HALVES = 1
FORMAT_W4A4 = 0
FORMAT_W8A8 = 1
FORMAT_NVFP4 = 2

_STATUS = {
    0: "SVDQ_OK", 1: "SVDQ_ERR_INVALID_ARG", 2: "SVDQ_ERR_SHAPE",
    3: "SVDQ_ERR_ALIGNMENT", 4: "SVDQ_ERR_UNSUPPORTED", 5: "SVDQ_ERR_NUMERIC",
    6: "SVDQ_ERR_CUDA", 7: "SVDQ_ERR_DEVICE_TIMEOUT", 8: "SVDQ_ERR_OOM",
    9: "SVDQ_ERR_IO",
}


class SVDQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)}")


_lib = None
_vp = ctypes.c_void_p
_i = ctypes.c_int


def lib() -> ctypes.CDLL:
    """Load libsvdq.so (built in-tree by `python -m
    w4a4_quantized_gemm_smooth_b200.build`).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m w4a4_quantized_gemm_smooth_b200.build` (no fallback exists)")
    L = ctypes.CDLL(LIB_PATH)
    sig = {
        "svdq_status_string": (ctypes.c_char_p, [_i]),
        "svdq_version": (_i, []),
        "svdq_calib_absmax": (_i, [_i, _i, _vp, _i, _vp]),
        "svdq_pack_weights": (_i, [_i, _i, _i, _i, _vp, _vp, ctypes.c_double, _vp, _i,
                                   _vp, _vp, ctypes.c_float, _vp, _vp]),
        "svdq_pack_weights_host": (_i, [_i, _i, _i, _i, _vp, _vp, ctypes.c_double, _vp,
                                        _i, _vp, _vp, ctypes.c_float, _vp]),
        "svdq_weights_info": (_i, [_vp, _vp, _vp, _vp, _vp, _vp]),
        "svdq_pack_weights_calibrated": (_i, [_i, _i, _i, _i, _vp, _vp, _i, _i, _i, _vp, _i,
                                              _i, _vp, _i, _vp, _vp, ctypes.c_float, _i, _vp,
                                              _vp, _vp]),
        "svdq_weights_export": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
        "svdq_weights_save": (_i, [_vp, ctypes.c_char_p]),
        "svdq_weights_load": (_i, [ctypes.c_char_p, _vp, _vp]),
        "svdq_weights_free": (None, [_vp]),
        "svdq_quantize_act": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp, _vp]),
        "svdq_linear": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _vp]),
        "svdq_get_device_error": (_i, [_vp, _vp]),
        "svdq_debug_partials": (_i, [_vp, _i, _vp, _i, _i, _i, _i, _vp, _vp]),
        "svdq_debug_linear_stall": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _i, ctypes.c_uint, _vp]),
        "svdq_linear_splitk_workspace": (ctypes.c_size_t, [_vp, _i, _i]),
        "svdq_linear_splitk": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _vp,
                                    ctypes.c_size_t, _vp]),
        "svdq_linear_splitk_noalloc": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _vp]),
        "svdq_pack_weights_w8a8": (_i, [_i, _i, _i, _vp, _vp, ctypes.c_double, _vp, _i, _vp,
                                        _vp]),
        "svdq_weights_export_w8a8": (_i, [_vp, _vp, _vp]),
        "svdq_weights_format": (_i, [_vp]),
        "svdq_quantize_act_w8a8": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp, _vp]),
        "svdq_linear_w8a8": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _vp]),
        "svdq_pack_weights_nvfp4": (_i, [_i, _i, _i, _vp, _vp, ctypes.c_double, _vp, _i, _vp,
                                         _vp]),
        "svdq_weights_export_nvfp4": (_i, [_vp, _vp, _vp, _vp]),
        "svdq_nvfp4_sf_bytes": (ctypes.c_size_t, [_i, _i]),
        "svdq_quantize_act_nvfp4": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp]),
        "svdq_linear_nvfp4": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _vp]),
        "svdq_linear_host_workspace": (ctypes.c_size_t, [_vp, _i]),
        "svdq_linear_host": (_i, [_vp, _i, _vp, _i, _vp, _i, _i, _vp, ctypes.c_size_t, _vp]),
        "svdq_linear_quantize_next_workspace": (ctypes.c_size_t, [_vp, _vp, _i]),
        "svdq_linear_quantize_next": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp,
                                           ctypes.c_size_t, _vp]),
        "svdq_linear16": (_i, [_i, _i, _i, _i, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _vp, _i, _vp,
                               _i, _vp]),
        "svdq_linear16_backward_workspace": (ctypes.c_size_t, [_i, _i, _i, _i]),
        "svdq_linear16_backward": (_i, [_i, _i, _i, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _i, _i,
                                        _vp, _i, _vp, _i, _vp, _vp, ctypes.c_size_t, _vp]),
        "svdq_debug_linear16_forms": (_i, [_i, _i, _i, _i, _vp]),
        "svdq_get_op_error": (_i, [_vp]),
        "svdq_layer_norm": (_i, [_i, _i, _i, _i, _vp, _i, _vp, _i, _vp, _i, ctypes.c_float, _i,
                                 ctypes.c_float, _vp, _i, _vp, _vp, _vp]),
        "svdq_layer_norm_backward_workspace": (ctypes.c_size_t, [_i, _i, _i]),
        "svdq_layer_norm_backward": (_i, [_i, _i, _i, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _i,
                                          ctypes.c_float, _i, _vp, _i, _vp, _i, _vp, _i, _vp,
                                          ctypes.c_size_t, _vp]),
        "svdq_rope_create": (_i, [_i, _vp, _vp, _i, _vp]),
        "svdq_rope_free": (None, [_vp]),
        "svdq_rope": (_i, [_vp, _i, _i, _i, _i, _vp, _i, _i, _vp, ctypes.c_longlong,
                           ctypes.c_longlong, _vp, ctypes.c_longlong, ctypes.c_longlong, _i, _vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(status: int, where: str):
    if status != 0:
        raise SVDQError(status, where)


def _np_ptr(a: np.ndarray | None):
    return None if a is None else a.ctypes.data_as(_vp)


def _stream_ptr(stream=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return _vp(stream.cuda_stream)


def _dev_ptr(t):
    return None if t is None else _vp(t.data_ptr())


class Weights:
    """Owns one packed layer handle (svdq_weights*)."""

    def __init__(self, handle: ctypes.c_void_p):
        self._h = handle
        K, N, r, sr, lr = (ctypes.c_int() for _ in range(5))
        _check(lib().svdq_weights_info(handle, ctypes.byref(K), ctypes.byref(N),
                                       ctypes.byref(r), ctypes.byref(sr),
                                       ctypes.byref(lr)), "svdq_weights_info")
        self.K, self.N, self.rank = K.value, N.value, r.value
        self.svd_rank, self.lora_rank = sr.value, lr.value
        self.format = int(lib().svdq_weights_format(handle))

    @property
    def handle(self):
        return self._h

    def export(self) -> dict:
        K, N, r = self.K, self.N, self.rank
        out = dict(
            inv_lambda=np.empty(K, np.float32), wq=np.empty((N, K // 2), np.uint8),
            s_w=np.empty((K // 64, N), np.float32), L1=np.empty((K, r), np.uint16),
            L2=np.empty((r, N), np.uint16), bias=np.empty(N, np.uint16),
            sigma=np.empty(self.svd_rank + 1, np.float64))
        _check(lib().svdq_weights_export(
            self._h, _np_ptr(out["inv_lambda"]), _np_ptr(out["wq"]), _np_ptr(out["s_w"]),
            _np_ptr(out["L1"]), _np_ptr(out["L2"]), _np_ptr(out["bias"]),
            _np_ptr(out["sigma"])), "svdq_weights_export")
        if self.format == FORMAT_W8A8:
            out["wq8"] = np.empty((N, K), np.int8)
            out["s_w8"] = np.empty(N, np.float32)
            _check(lib().svdq_weights_export_w8a8(self._h, _np_ptr(out["wq8"]),
                                                  _np_ptr(out["s_w8"])), "svdq_weights_export_w8a8")
        if self.format == FORMAT_NVFP4:
            out["wq4"] = np.empty((N, K // 2), np.uint8)
            out["sf4"] = np.empty((N, K // 16), np.uint8)
            out["s_w4"] = np.empty(N, np.float32)
            _check(lib().svdq_weights_export_nvfp4(self._h, _np_ptr(out["wq4"]), _np_ptr(out["sf4"]),
                                                   _np_ptr(out["s_w4"])), "svdq_weights_export_nvfp4")
        return out

    def save(self, path: str):
        _check(lib().svdq_weights_save(self._h, path.encode()), "svdq_weights_save")

    def free(self):
        if self._h:
            lib().svdq_weights_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def svdq_calib_absmax(X_bits: np.ndarray, absmax: np.ndarray | None = None) -> np.ndarray:
    """Running per-channel max|X| of a host bf16 matrix (uint16 bits [M, K])."""
    X_bits = np.ascontiguousarray(X_bits, dtype=np.uint16)
    M, K = X_bits.shape
    if absmax is None:
        absmax = np.zeros(K, np.float32)
    _check(lib().svdq_calib_absmax(M, K, _np_ptr(X_bits), K, _np_ptr(absmax)),
           "svdq_calib_absmax")
    return absmax


def _pack_args(W_bits, act_absmax, bias_bits, lora_A_bits, lora_B_bits):
    W_bits = np.ascontiguousarray(W_bits, dtype=np.uint16)
    act_absmax = np.ascontiguousarray(act_absmax, dtype=np.float32)
    bias_bits = None if bias_bits is None else np.ascontiguousarray(bias_bits, dtype=np.uint16)
    A = None if lora_A_bits is None else np.ascontiguousarray(lora_A_bits, dtype=np.uint16)
    B = None if lora_B_bits is None else np.ascontiguousarray(lora_B_bits, dtype=np.uint16)
    lr = 0 if A is None else A.shape[1]
    return W_bits, act_absmax, bias_bits, A, B, lr


def svdq_pack_weights(W_bits, act_absmax, rank, alpha=0.5, bias_bits=None,
                      lora_A_bits=None, lora_B_bits=None, lora_scale=1.0,
                      stream=None) -> Weights:
    """Offline pack onto the current CUDA device (see include/svdq.h)."""
    W_bits, act_absmax, bias_bits, A, B, lr = _pack_args(
        W_bits, act_absmax, bias_bits, lora_A_bits, lora_B_bits)
    N, K = W_bits.shape
    h = _vp()
    _check(lib().svdq_pack_weights(K, N, int(rank), 64, _np_ptr(W_bits), _np_ptr(act_absmax),
                                   float(alpha), _np_ptr(bias_bits), lr, _np_ptr(A),
                                   _np_ptr(B), float(lora_scale), _stream_ptr(stream),
                                   ctypes.byref(h)), "svdq_pack_weights")
    return Weights(h)


def svdq_pack_weights_host(W_bits, act_absmax, rank, alpha=0.5, bias_bits=None,
                           lora_A_bits=None, lora_B_bits=None, lora_scale=1.0) -> Weights:
    """Same transform without a GPU (host copies only)."""
    W_bits, act_absmax, bias_bits, A, B, lr = _pack_args(
        W_bits, act_absmax, bias_bits, lora_A_bits, lora_B_bits)
    N, K = W_bits.shape
    h = _vp()
    _check(lib().svdq_pack_weights_host(K, N, int(rank), 64, _np_ptr(W_bits),
                                        _np_ptr(act_absmax), float(alpha), _np_ptr(bias_bits),
                                        lr, _np_ptr(A), _np_ptr(B), float(lora_scale),
                                        ctypes.byref(h)), "svdq_pack_weights_host")
    return Weights(h)


def svdq_pack_weights_calibrated(W_bits, X_cal_bits, rank, alphas=(0.3, 0.4, 0.5, 0.6, 0.7),
                                 refine_iters=1, bias_bits=None, lora_A_bits=None,
                                 lora_B_bits=None, lora_scale=1.0, to_device=True, stream=None,
                                 gptq=False):
    """Pack with the calibrated alpha search, the alternating factor
    refinement and, with gptq=True, GPTQ rounding of the residual.
    X_cal_bits: host bf16 bits [M_cal, K] (calibration tokens).
    Returns (Weights, errors per alpha)."""
    X_cal_bits = np.ascontiguousarray(X_cal_bits, dtype=np.uint16)
    W_bits, _, bias_bits, A, B, lr = _pack_args(
        W_bits, np.zeros(X_cal_bits.shape[1], np.float32), bias_bits, lora_A_bits, lora_B_bits)
    N, K = W_bits.shape
    al = np.ascontiguousarray(alphas, dtype=np.float64)
    errs = np.zeros(len(al), np.float64)
    h = _vp()
    _check(lib().svdq_pack_weights_calibrated(
        K, N, int(rank), 64, _np_ptr(W_bits), _np_ptr(X_cal_bits), X_cal_bits.shape[0], K,
        len(al), _np_ptr(al), int(refine_iters), 1 if gptq else 0, _np_ptr(bias_bits), lr,
        _np_ptr(A), _np_ptr(B),
        float(lora_scale), 1 if to_device else 0, _stream_ptr(stream) if to_device else None,
        _np_ptr(errs), ctypes.byref(h)), "svdq_pack_weights_calibrated")
    return Weights(h), errs


def svdq_weights_load(path: str, stream=None) -> Weights:
    h = _vp()
    _check(lib().svdq_weights_load(path.encode(), _stream_ptr(stream), ctypes.byref(h)),
           "svdq_weights_load")
    return Weights(h)


def svdq_quantize_act(w: Weights, X, xq, s_x, Z=None, stream=None):
    """X: cuda bf16 [M, K] (row stride X.stride(0)); xq uint8 [M, K/2];
    s_x float32 [K/64, M]; Z bf16 [M, rank] or None when rank == 0."""
    M = X.shape[0]
    _check(lib().svdq_quantize_act(w.handle, M, _dev_ptr(X), X.stride(0), _dev_ptr(xq),
                                   _dev_ptr(s_x), _dev_ptr(Z), _stream_ptr(stream)),
           "svdq_quantize_act")


def svdq_linear(w: Weights, xq, s_x, Z, Y, epilogue=EPI_NONE, stream=None):
    """Y: cuda bf16 [M, N] (row stride Y.stride(0))."""
    M = Y.shape[0]
    _check(lib().svdq_linear(w.handle, M, _dev_ptr(xq), _dev_ptr(s_x), _dev_ptr(Z),
                             _dev_ptr(Y), Y.stride(0), int(epilogue), _stream_ptr(stream)),
           "svdq_linear")


def svdq_linear_host_workspace(w: Weights, M: int) -> int:
    """Device workspace bytes of svdq_linear_host (0 for invalid arguments)."""
    return int(lib().svdq_linear_host_workspace(w.handle, int(M)))


def svdq_linear_host(w: Weights, X, Y, workspace, epilogue=EPI_NONE, stream=None):
    """The layer from host memory: X CPU bf16 [M, K] (row stride X.stride(0)),
    Y CPU bf16 [M, N] (row stride Y.stride(0)), both ideally pinned;
    workspace: cuda tensor of at least svdq_linear_host_workspace(w, M)
    bytes.  Enqueues the copies and both kernels on the stream; Y is valid
    after it has been synchronised."""
    M = X.shape[0]
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().svdq_linear_host(w.handle, M, _vp(X.data_ptr()), X.stride(0), _vp(Y.data_ptr()),
                                  Y.stride(0), int(epilogue), _dev_ptr(workspace), nbytes,
                                  _stream_ptr(stream)),
           "svdq_linear_host")


def svdq_linear_quantize_next_workspace(w: Weights, w_next: Weights, M: int) -> int:
    """Workspace bytes of svdq_linear_quantize_next (the column tiles'
    partial Z_next, fp32; 0 when rank_next == 0 or for invalid arguments)."""
    return int(lib().svdq_linear_quantize_next_workspace(w.handle, w_next.handle, int(M)))


def svdq_linear_quantize_next(w: Weights, w_next: Weights, xq, s_x, Z, xq_next, s_x_next,
                              Z_next, workspace, epilogue=EPI_NONE, stream=None):
    """The layer of w with the next layer's activation pass in its epilogue:
    writes xq_next uint8 [M, N/2], s_x_next float32 [N/64, M] and Z_next bf16
    [M, rank_next] (None when rank_next == 0) instead of Y.  workspace: cuda
    tensor of at least svdq_linear_quantize_next_workspace(w, w_next, M)
    bytes (None when rank_next == 0)."""
    M = xq.shape[0]
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().svdq_linear_quantize_next(w.handle, w_next.handle, M, _dev_ptr(xq),
                                           _dev_ptr(s_x), _dev_ptr(Z), int(epilogue),
                                           _dev_ptr(xq_next), _dev_ptr(s_x_next),
                                           _dev_ptr(Z_next), _dev_ptr(workspace), nbytes,
                                           _stream_ptr(stream)),
           "svdq_linear_quantize_next")


def svdq_linear_splitk_workspace(w: Weights, M: int, splits: int = 0) -> int:
    """Workspace bytes of svdq_linear_splitk (0 for invalid arguments)."""
    return int(lib().svdq_linear_splitk_workspace(w.handle, int(M), int(splits)))


def svdq_linear_splitk(w: Weights, xq, s_x, Z, Y, workspace, splits=0, epilogue=EPI_NONE,
                       stream=None):
    """Split-K svdq_linear.  workspace: cuda tensor of at least
    svdq_linear_splitk_workspace(w, M, splits) bytes (256-byte aligned)."""
    M = Y.shape[0]
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().svdq_linear_splitk(w.handle, M, _dev_ptr(xq), _dev_ptr(s_x), _dev_ptr(Z),
                                    _dev_ptr(Y), Y.stride(0), int(epilogue), int(splits),
                                    _dev_ptr(workspace), nbytes, _stream_ptr(stream)),
           "svdq_linear_splitk")


def svdq_linear_splitk_noalloc(w: Weights, xq, s_x, Z, Y, splits=0, epilogue=EPI_NONE,
                               stream=None):
    """svdq_linear_splitk with the library's fixed device scratch (no allocation)."""
    M = Y.shape[0]
    _check(lib().svdq_linear_splitk_noalloc(w.handle, M, _dev_ptr(xq), _dev_ptr(s_x),
                                            _dev_ptr(Z), _dev_ptr(Y), Y.stride(0),
                                            int(epilogue), int(splits), _stream_ptr(stream)),
           "svdq_linear_splitk_noalloc")


def svdq_pack_weights_w8a8(W_bits, act_absmax, rank, alpha=0.5, bias_bits=None, to_device=True,
                           stream=None) -> Weights:
    """Offline pack of the W8A8 comparator (int8 residual per output channel)."""
    W_bits, act_absmax, bias_bits, _, _, _ = _pack_args(W_bits, act_absmax, bias_bits, None, None)
    N, K = W_bits.shape
    h = _vp()
    _check(lib().svdq_pack_weights_w8a8(K, N, int(rank), _np_ptr(W_bits), _np_ptr(act_absmax),
                                        float(alpha), _np_ptr(bias_bits), 1 if to_device else 0,
                                        _stream_ptr(stream) if to_device else None,
                                        ctypes.byref(h)), "svdq_pack_weights_w8a8")
    return Weights(h)


def svdq_quantize_act_w8a8(w: Weights, X, xq, s_x, Z=None, stream=None):
    """X: cuda bf16 [M, K]; xq int8 [M, K]; s_x float32 [M]; Z bf16 [M, rank]."""
    M = X.shape[0]
    _check(lib().svdq_quantize_act_w8a8(w.handle, M, _dev_ptr(X), X.stride(0), _dev_ptr(xq),
                                        _dev_ptr(s_x), _dev_ptr(Z), _stream_ptr(stream)),
           "svdq_quantize_act_w8a8")


def svdq_linear_w8a8(w: Weights, xq, s_x, Z, Y, epilogue=EPI_NONE, stream=None):
    """Y: cuda bf16 [M, N] (row stride Y.stride(0))."""
    M = Y.shape[0]
    _check(lib().svdq_linear_w8a8(w.handle, M, _dev_ptr(xq), _dev_ptr(s_x), _dev_ptr(Z),
                                  _dev_ptr(Y), Y.stride(0), int(epilogue), _stream_ptr(stream)),
           "svdq_linear_w8a8")


def svdq_pack_weights_nvfp4(W_bits, act_absmax, rank, alpha=0.5, bias_bits=None, to_device=True,
                            stream=None) -> Weights:
    """Offline pack of the NVFP4 variant (E2M1 residual, E4M3 group scales)."""
    W_bits, act_absmax, bias_bits, _, _, _ = _pack_args(W_bits, act_absmax, bias_bits, None, None)
    N, K = W_bits.shape
    h = _vp()
    _check(lib().svdq_pack_weights_nvfp4(K, N, int(rank), _np_ptr(W_bits), _np_ptr(act_absmax),
                                         float(alpha), _np_ptr(bias_bits), 1 if to_device else 0,
                                         _stream_ptr(stream) if to_device else None,
                                         ctypes.byref(h)), "svdq_pack_weights_nvfp4")
    return Weights(h)


def svdq_nvfp4_sf_bytes(rows: int, K: int) -> int:
    return int(lib().svdq_nvfp4_sf_bytes(int(rows), int(K)))


def svdq_quantize_act_nvfp4(w: Weights, X, xq, sfa, s_x, Z=None, stream=None):
    """X: cuda bf16 [M, K]; xq uint8 [M, K/2]; sfa uint8 [svdq_nvfp4_sf_bytes(M, K)];
    s_x float32 [M]; Z bf16 [M, rank] (stored divided by s_x)."""
    M = X.shape[0]
    _check(lib().svdq_quantize_act_nvfp4(w.handle, M, _dev_ptr(X), X.stride(0), _dev_ptr(xq),
                                         _dev_ptr(sfa), _dev_ptr(s_x), _dev_ptr(Z),
                                         _stream_ptr(stream)), "svdq_quantize_act_nvfp4")


def svdq_linear_nvfp4(w: Weights, xq, sfa, s_x, Z, Y, epilogue=EPI_NONE, stream=None):
    """Y: cuda bf16 [M, N] (row stride Y.stride(0))."""
    M = Y.shape[0]
    _check(lib().svdq_linear_nvfp4(w.handle, M, _dev_ptr(xq), _dev_ptr(sfa), _dev_ptr(s_x),
                                   _dev_ptr(Z), _dev_ptr(Y), Y.stride(0), int(epilogue),
                                   _stream_ptr(stream)), "svdq_linear_nvfp4")


def svdq_get_device_error(w: Weights, stream=None):
    _check(lib().svdq_get_device_error(w.handle, _stream_ptr(stream)), "device")


def svdq_debug_linear_stall(w: Weights, xq, s_x, Z, Y, limit_us=200, stream=None):
    """Test hook: svdq_linear with every device wait bounded by limit_us and
    the first CTA's first stage withheld (see include/svdq.h)."""
    M = Y.shape[0]
    _check(lib().svdq_debug_linear_stall(w.handle, M, _dev_ptr(xq), _dev_ptr(s_x), _dev_ptr(Z),
                                         _dev_ptr(Y), Y.stride(0), ctypes.c_uint(int(limit_us)),
                                         _stream_ptr(stream)), "svdq_debug_linear_stall")


def svdq_debug_partials(w: Weights, M, xq, row0, nrows, col0, ncols, P, stream=None):
    """P: cuda int32 [K/64, nrows, ncols]."""
    _check(lib().svdq_debug_partials(w.handle, int(M), _dev_ptr(xq), int(row0), int(nrows),
                                     int(col0), int(ncols), _dev_ptr(P), _stream_ptr(stream)),
           "svdq_debug_partials")


# ------------------------------------------------------------------------
# 16-bit operators around the quantised layers.  These calls take plain
# tensors, so the binding checks each one's device, type and shape before it
# passes the pointer on (ValueError); the library checks sizes, alignment and
# overlap (SVDQError).
# They go through a small CPython module, since a call through ctypes takes
# the host longer than one token's kernels take the device.

_fast = None


def _fastcall():
    """The CPython binding (_svdq_fastcall in _lib, built with the library for
    the interpreter that runs).  Raises if it is missing."""
    global _fast
    if _fast is None:
        import importlib.util
        import torch
        lib()
        from .build import FASTCALL as path
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with "
                "`python -m w4a4_quantized_gemm_smooth_b200.build` (no fallback exists)")
        spec = importlib.util.spec_from_file_location("_svdq_fastcall", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        # torch's own short cuts where it has them, else what they stand for
        device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                  or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
        mod.init((torch.bfloat16, torch.float16, torch.float32), torch.int32, device, stream)
        _fast = mod
    return _fast


def svdq_linear16(X, W, Y, bias=None, residual=None, epilogue=EPI_NONE, preact=None, stream=None):
    """Y = epi(X W^T + bias) + residual.  X [M, K], W [N, K], Y [M, N], all
    cuda bf16 or fp16 with contiguous rows; bias [N]; residual [M, N] (may be
    Y); preact [M, N] receives X W^T + bias for svdq_linear16_backward."""
    rc = (_fast or _fastcall()).linear16(X, W, Y, bias, residual, epilogue, preact,
                                         None if stream is None else stream.cuda_stream)
    if rc:
        raise SVDQError(rc, "svdq_linear16")


def svdq_linear16_backward_workspace(M: int, K: int, N: int, epilogue=EPI_NONE) -> int:
    """Workspace bytes of svdq_linear16_backward (may be 0; 0 for invalid arguments)."""
    return int(lib().svdq_linear16_backward_workspace(int(M), int(K), int(N), int(epilogue)))


def svdq_linear16_backward(dY, X, W, preact, dX, dW, dbias, workspace, epilogue=EPI_NONE,
                           stream=None):
    """Gradients of svdq_linear16: dX [M, K], dW [N, K] and dbias [N] (each may
    be None) for dY [M, N]; preact is the forward call's (None without an
    activation).  The residual's gradient is dY itself."""
    rc = (_fast or _fastcall()).linear16_backward(dY, X, W, preact, dX, dW, dbias, workspace, epilogue,
                                                  None if stream is None else stream.cuda_stream)
    if rc:
        raise SVDQError(rc, "svdq_linear16_backward")


def svdq_debug_linear16_forms(M: int, K: int, N: int, gradients: int = 0) -> list:
    """Test hook, host only: the forms (on CTA pairs, tile columns, splits of the
    reduction) of a 16-bit product's launches; gradients: 0 forward, 1 dX, 2 dW,
    3 both.  Empty for the few rows that take another way."""
    f = (ctypes.c_int * 6)()
    n = lib().svdq_debug_linear16_forms(int(M), int(K), int(N), int(gradients), f)
    return [(bool(f[3 * i]), f[3 * i + 1], f[3 * i + 2]) for i in range(n)]


def svdq_get_op_error(stream=None):
    """Synchronises the stream and raises if a bounded wait of a 16-bit
    operator expired on the current device since the last call."""
    _check(lib().svdq_get_op_error(_stream_ptr(stream)), "device")


def svdq_layer_norm(X, Y, weight=None, bias=None, eps=1e-6, weight_offset=0.0, rows_per_group=0,
                    mean=None, rstd=None, stream=None):
    """Y = (X - mean) rstd (weight + weight_offset) + bias over rows of X
    [M, K] (bf16, fp16 or fp32).  weight, bias: [K], or [groups, K] with one
    row for every rows_per_group rows of X; X's type or fp32.  mean, rstd:
    fp32 [M], the statistics for svdq_layer_norm_backward.  Y may be X."""
    rc = (_fast or _fastcall()).layer_norm(X, Y, weight, bias, eps, weight_offset, rows_per_group,
                                           mean, rstd,
                                           None if stream is None else stream.cuda_stream)
    if rc:
        raise SVDQError(rc, "svdq_layer_norm")


def svdq_layer_norm_backward_workspace(M: int, K: int, rows_per_group: int = 0) -> int:
    """Workspace bytes of svdq_layer_norm_backward (may be 0)."""
    return int(lib().svdq_layer_norm_backward_workspace(int(M), int(K), int(rows_per_group)))


def svdq_layer_norm_backward(dY, X, mean, rstd, dX, weight=None, weight_offset=0.0,
                             rows_per_group=0, dweight=None, dbias=None, workspace=None,
                             stream=None):
    """Gradients of svdq_layer_norm: dX [M, K] (may be dY or X), dweight and
    dbias [groups, K] or, with one group, [K]; each may be None."""
    rc = (_fast or _fastcall()).layer_norm_backward(dY, X, mean, rstd, dX, weight, weight_offset,
                                                    rows_per_group, dweight, dbias, workspace,
                                                    None if stream is None else stream.cuda_stream)
    if rc:
        raise SVDQError(rc, "svdq_layer_norm_backward")


class RopePlan:
    """Owns one rotary-position plan (svdq_rope_plan*): host data only."""

    def __init__(self, handle, n_axes: int, pairs: int):
        self._h = handle
        self.n_axes, self.pairs = n_axes, pairs

    @property
    def handle(self):
        return self._h

    def free(self):
        if self._h:
            lib().svdq_rope_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def rope_frequencies(pairs_per_axis, theta: float = 10000.0) -> list:
    """The usual frequencies, theta^(-i / p) for pair i of an axis of p pairs."""
    return [float(theta) ** (-i / p) for p in pairs_per_axis for i in range(p)]


def svdq_rope_create(pairs_per_axis, freq, pairing=ROPE_INTERLEAVED) -> RopePlan:
    """Plan of rotary positions: axis a turns pairs_per_axis[a] consecutive
    pairs of a head; freq holds every pair's frequency (radians per position)."""
    pp = np.ascontiguousarray(pairs_per_axis, dtype=np.int32)
    fr = np.ascontiguousarray(freq, dtype=np.float64)
    if pp.ndim != 1 or fr.ndim != 1 or fr.shape[0] != int(pp.sum()):
        raise ValueError("freq: expected one frequency per pair")
    h = _vp()
    _check(lib().svdq_rope_create(len(pp), _np_ptr(pp), _np_ptr(fr), int(pairing),
                                  ctypes.byref(h)), "svdq_rope_create")
    return RopePlan(h, len(pp), len(fr))


def svdq_rope(plan: RopePlan, positions, X, out, inverse=False, stream=None):
    """Rotates the heads of X [T, H, D] (bf16, fp16 or fp32, any token and
    head strides) into out (same shape; X itself rotates in place).
    positions: int32 [T, axes], or [R, axes] shared by tokens t with equal
    t % R.  inverse: the opposite rotation, the gradient of the first."""
    rc = (_fast or _fastcall()).rope(plan._h.value if plan._h else 0, plan.n_axes, positions, X, out, inverse,
                                     None if stream is None else stream.cuda_stream)
    if rc:
        raise SVDQError(rc, "svdq_rope")


class SVDQLinear:
    """One packed layer plus the buffers of its two hot-path calls.

    forward(X) runs svdq_quantize_act then svdq_linear on the current stream
    and returns Y (bf16 [M, N]).  Buffers are reallocated only when M grows.
    """

    def __init__(self, weights: Weights, epilogue: int = EPI_NONE):
        self.w = weights
        self.epilogue = epilogue
        self._M = -1
        self.xq = self.s_x = self.Z = self.Y = None

    def buffers(self, M: int, device="cuda"):
        import torch
        if M != self._M:
            K, N, r = self.w.K, self.w.N, self.w.rank
            self.xq = torch.empty((M, K // 2), dtype=torch.uint8, device=device)
            self.s_x = torch.empty((K // 64, M), dtype=torch.float32, device=device)
            self.Z = torch.empty((M, max(r, 1)), dtype=torch.bfloat16, device=device) if r else None
            self.Y = torch.empty((M, N), dtype=torch.bfloat16, device=device)
            self._M = M
        return self.xq, self.s_x, self.Z, self.Y

    def forward(self, X, out=None):
        M = X.shape[0]
        xq, s_x, Z, Y = self.buffers(M, X.device)
        if out is not None:
            Y = out
        svdq_quantize_act(self.w, X, xq, s_x, Z)
        svdq_linear(self.w, xq, s_x, Z, Y, self.epilogue)
        return Y

    __call__ = forward


class W8A8Linear(SVDQLinear):
    """The W8A8 comparator layer: svdq_quantize_act_w8a8 then svdq_linear_w8a8."""

    def buffers(self, M: int, device="cuda"):
        import torch
        if M != self._M:
            K, N, r = self.w.K, self.w.N, self.w.rank
            self.xq = torch.empty((M, K), dtype=torch.int8, device=device)
            self.s_x = torch.empty((M,), dtype=torch.float32, device=device)
            self.Z = torch.empty((M, max(r, 1)), dtype=torch.bfloat16, device=device) if r else None
            self.Y = torch.empty((M, N), dtype=torch.bfloat16, device=device)
            self._M = M
        return self.xq, self.s_x, self.Z, self.Y

    def forward(self, X, out=None):
        M = X.shape[0]
        xq, s_x, Z, Y = self.buffers(M, X.device)
        if out is not None:
            Y = out
        svdq_quantize_act_w8a8(self.w, X, xq, s_x, Z)
        svdq_linear_w8a8(self.w, xq, s_x, Z, Y, self.epilogue)
        return Y

    __call__ = forward


class NVFP4Linear(SVDQLinear):
    """The NVFP4 layer: svdq_quantize_act_nvfp4 then svdq_linear_nvfp4."""

    def buffers(self, M: int, device="cuda"):
        import torch
        if M != self._M:
            K, N, r = self.w.K, self.w.N, self.w.rank
            self.xq = torch.empty((M, K // 2), dtype=torch.uint8, device=device)
            self.sfa = torch.empty((svdq_nvfp4_sf_bytes(M, K),), dtype=torch.uint8, device=device)
            self.s_x = torch.empty((M,), dtype=torch.float32, device=device)
            self.Z = torch.empty((M, max(r, 1)), dtype=torch.bfloat16, device=device) if r else None
            self.Y = torch.empty((M, N), dtype=torch.bfloat16, device=device)
            self._M = M
        return self.xq, self.sfa, self.s_x, self.Z, self.Y

    def forward(self, X, out=None):
        M = X.shape[0]
        xq, sfa, s_x, Z, Y = self.buffers(M, X.device)
        if out is not None:
            Y = out
        svdq_quantize_act_nvfp4(self.w, X, xq, sfa, s_x, Z)
        svdq_linear_nvfp4(self.w, xq, sfa, s_x, Z, Y, self.epilogue)
        return Y

    __call__ = forward


class Linear16:
    """A 16-bit linear layer (the layers that are not quantised): weight
    [N, K] and bias [N], cuda bf16 or fp16, used in place.

    forward(X) returns epi(X W^T + b) + residual on the current stream; with
    save=True it keeps X and the pre-activation for backward(dY), which
    returns (dX, dW, db); X is kept by reference and has to stay as it is until
    then.  Buffers are reallocated only when M, the weight's shape, the type or
    the device changes, and the next call reuses them.
    """

    def __init__(self, weight, bias=None, epilogue: int = EPI_NONE):
        self.weight, self.bias, self.epilogue = weight, bias, epilogue
        self._key = self._keyb = None
        self.Y = self.P = self._saved = None

    @staticmethod
    def _empty(rows, cols, like):
        import torch                # rows of a multiple of 16 bytes
        return torch.empty((rows, -(-cols // 8) * 8), dtype=like.dtype, device=like.device)[:, :cols]

    def forward(self, X, residual=None, out=None, save: bool = False):
        M, N = X.shape[0], self.weight.shape[0]
        key = (M, N, X.dtype, X.device)
        if key != self._key:
            self.Y, self.P, self._key = self._empty(M, N, X), None, key
        if save and self.epilogue != EPI_NONE and self.P is None:
            self.P = self._empty(M, N, X)
        Y = self.Y if out is None else out
        keep = save and self.epilogue != EPI_NONE
        svdq_linear16(X, self.weight, Y, self.bias, residual, self.epilogue,
                      self.P if keep else None)
        self._saved = X if save else None
        return Y

    def backward(self, dY):
        import torch
        if self._saved is None:
            raise RuntimeError("backward needs a forward call with save=True")
        X, W = self._saved, self.weight
        M, (N, K) = X.shape[0], W.shape
        key = (M, N, K, X.dtype, X.device, self.bias is None, self.epilogue)
        if key != self._keyb:
            n = svdq_linear16_backward_workspace(M, K, N, self.epilogue)
            self.ws = torch.empty((n,), dtype=torch.uint8, device=X.device)
            self.dX, self.dW = self._empty(M, K, X), self._empty(N, K, X)
            self.db = None if self.bias is None else torch.empty_like(self.bias)
            self._keyb = key
        svdq_linear16_backward(dY, X, W, self.P if self.epilogue != EPI_NONE else None, self.dX,
                               self.dW, self.db, self.ws, self.epilogue)
        return self.dX, self.dW, self.db

    __call__ = forward


class LayerNorm:
    """Layer norm with optional weight and bias ([K], or [groups, K] with
    rows_per_group given to forward: the modulated norm), cuda tensors of the
    input's type or fp32, used in place; weight_offset is added to weight.

    forward(X) returns the norm on the current stream; with save=True it
    keeps X and the statistics for backward(dY), which returns
    (dX, dweight, dbias), a parameter's gradient in the parameter's shape (one
    that all groups share, [K] or [1, K], is summed over them).  X is kept by
    reference and has to stay as it is until then, so with save=True out cannot
    be X (ValueError); without it the norm may run in place.  Buffers are
    reallocated only when X's shape, type or device changes, and the next call
    reuses them.
    """

    def __init__(self, weight=None, bias=None, eps: float = 1e-6, weight_offset: float = 0.0):
        self.weight, self.bias, self.eps, self.weight_offset = weight, bias, eps, weight_offset
        self._key = self._keyb = None
        self.Y = self.mean = self.rstd = self._saved = None

    def forward(self, X, out=None, rows_per_group: int = 0, save: bool = False):
        import torch
        M, K = X.shape
        key = (M, K, X.dtype, X.device)
        if key != self._key:
            self.Y = Linear16._empty(M, K, X)
            self.mean = torch.empty((M,), dtype=torch.float32, device=X.device)
            self.rstd = torch.empty_like(self.mean)
            self._key = key
        Y = self.Y if out is None else out
        if save and X.numel() and Y.data_ptr() == X.data_ptr():
            raise ValueError("save=True keeps X for backward: out cannot be X itself")
        svdq_layer_norm(X, Y, self.weight, self.bias, self.eps, self.weight_offset, rows_per_group,
                        self.mean if save else None, self.rstd if save else None)
        self._saved = (X, rows_per_group) if save else None
        return Y

    def backward(self, dY):
        import torch
        if self._saved is None:
            raise RuntimeError("backward needs a forward call with save=True")
        X, rpg = self._saved
        M, K = X.shape
        w, b = self.weight, self.bias
        key = (M, K, X.dtype, X.device, rpg, *((p.shape, p.dtype) for p in (w, b) if p is not None))
        if key != self._keyb:
            n = max(svdq_layer_norm_backward_workspace(M, K, r) for r in (0, rpg))
            self.ws = torch.empty((n,), dtype=torch.uint8, device=X.device) if n else None
            self.dX = Linear16._empty(M, K, X)
            rows = lambda p: Linear16._empty(p.shape[0] if p.dim() == 2 else 1, K, p)
            grad = lambda p: None if p is None else rows(p) if p.dim() == 2 else rows(p)[0]
            self.dw, self.db = grad(w), grad(b)
            self._keyb = key
        # a parameter that all groups share has one gradient, over all rows: where the
        # other has a row per group, a second pass over the rows sums it
        per_group = lambda p: p is not None and p.dim() == 2 and p.shape[0] != 1
        if per_group(w) or per_group(b):
            one = [None if per_group(p) else g for p, g in ((w, self.dw), (b, self.db))]
            own = [g if per_group(p) else None for p, g in ((w, self.dw), (b, self.db))]
        else:
            rpg, one, own = 0, [None, None], [self.dw, self.db]
        svdq_layer_norm_backward(dY, X, self.mean, self.rstd, self.dX, w, self.weight_offset, rpg, *own, self.ws)
        if one != [None, None]:
            svdq_layer_norm_backward(dY, X, self.mean, self.rstd, None, None, 0.0, 0, *one, self.ws)
        return self.dX, self.dw, self.db

    __call__ = forward


class SVDQMLP:
    """Two packed layers applied in sequence, fc2(GELU(fc1(X))), as in a
    transformer block's feed-forward part.

    forward(X) runs the four plain calls, storing the bf16 hidden activation
    H in between (the faster chain on B200).  forward(X, fused=True) runs
    svdq_quantize_act(fc1), then svdq_linear_quantize_next (fc1 with GELU,
    emitting fc2's codes, scales and Z), then svdq_linear(fc2): H never
    reaches device memory, and fc2's codes and scales are the same bits.
    Buffers are reallocated only when M changes.

    norm: a LayerNorm in front of fc1 (its modulation groups are passed to
    forward as rows_per_group), or None.
    """

    def __init__(self, fc1: Weights, fc2: Weights, norm: LayerNorm | None = None):
        if fc2.K != fc1.N:
            raise ValueError("fc2's K must equal fc1's N")
        self.norm = norm
        self.fc1 = SVDQLinear(fc1, EPI_GELU)
        self.fc2 = SVDQLinear(fc2)
        self._M = -1
        self.H = self.ws = None

    def buffers(self, M: int, device="cuda"):
        import torch
        self.fc1.buffers(M, device)
        self.fc2.buffers(M, device)
        if M != self._M:
            self.H = torch.empty((M, self.fc1.w.N), dtype=torch.bfloat16, device=device)
            n = svdq_linear_quantize_next_workspace(self.fc1.w, self.fc2.w, M)
            self.ws = torch.empty((n,), dtype=torch.uint8, device=device) if n else None
            self._M = M
        return self.H, self.ws

    def forward(self, X, fused: bool = False, out=None, rows_per_group: int = 0):
        M = X.shape[0]
        H, ws = self.buffers(M, X.device)
        a, b = self.fc1, self.fc2
        if self.norm is not None:
            X = self.norm(X, rows_per_group=rows_per_group)
        Y = b.Y if out is None else out
        svdq_quantize_act(a.w, X, a.xq, a.s_x, a.Z)
        if fused:
            svdq_linear_quantize_next(a.w, b.w, a.xq, a.s_x, a.Z, b.xq, b.s_x, b.Z, ws, EPI_GELU)
        else:
            svdq_linear(a.w, a.xq, a.s_x, a.Z, H, EPI_GELU)
            svdq_quantize_act(b.w, H, b.xq, b.s_x, b.Z)
        svdq_linear(b.w, b.xq, b.s_x, b.Z, Y)
        return Y

    __call__ = forward


class SVDQQKV:
    """A packed QKV layer with the rotary positions of its queries and keys:
    norm (a LayerNorm, or None), the W4A4 product, then svdq_rope in place on
    the query and key heads of the product's rows.

    The packed layer's N is (heads + 2 kv_heads) head_dim, its columns the
    query heads, then the key heads, then the value heads; kv_heads defaults
    to heads.
    """

    def __init__(self, weights: Weights, heads: int, head_dim: int, plan: RopePlan,
                 norm: LayerNorm | None = None, kv_heads: int | None = None):
        kv = heads if kv_heads is None else kv_heads
        if weights.N != (heads + 2 * kv) * head_dim:
            raise ValueError("N must equal (heads + 2 kv_heads) head_dim")
        self.qkv = SVDQLinear(weights)
        self.norm, self.plan = norm, plan
        self.heads, self.kv_heads, self.head_dim = heads, kv, head_dim

    def forward(self, X, positions, out=None, rows_per_group: int = 0):
        """X bf16 [M, K], positions int32 [M or fewer, axes] -> bf16 [M, N]."""
        if self.norm is not None:
            X = self.norm(X, rows_per_group=rows_per_group)
        Y = self.qkv(X, out)
        qk = Y[:, :(self.heads + self.kv_heads) * self.head_dim].unflatten(1, (-1, self.head_dim))
        svdq_rope(self.plan, positions, qk, qk)
        return Y

    __call__ = forward
