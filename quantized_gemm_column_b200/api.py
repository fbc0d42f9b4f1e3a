"""ctypes binding of libaveris (include/averis.h), argument marshalling only.

Every function here has the name of the C entry point it calls.  Tensors are
torch CUDA tensors (PyTorch only provides device memory and streams); all
arithmetic happens in the library's CUDA kernels.  A missing library raises
``AverisError``: there is no CPU path.
"""

import ctypes
import os

import torch

from . import build as _build

_LIB = None

AVR_OK = 0
AVR_ERR_INVALID_ARG = 1
AVR_ERR_UNSUPPORTED_SHAPE = 2
AVR_ERR_MISALIGNED = 3
AVR_ERR_WORKSPACE_TOO_SMALL = 4
AVR_ERR_CUDA = 5
AVR_ERR_DEVICE_TIMEOUT = 6
AVR_ERR_NONFINITE = 7
AVR_ERR_NO_DEVICE = 8

AVR_F32 = 0
AVR_BF16 = 1
AVR_RNE = 0
AVR_SR = 1

_c_i64 = ctypes.c_int64
_c_u64 = ctypes.c_uint64
_c_u32 = ctypes.c_uint32
_c_size = ctypes.c_size_t
_c_int = ctypes.c_int
_c_ptr = ctypes.c_void_p


class AverisError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = int(status)
        msg = status_string(self.status) if _LIB is not None else str(status)
        super().__init__(f"{where}: {msg} (status {self.status})")


class avr_nvfp4(ctypes.Structure):
    _fields_ = [("codes", _c_ptr), ("scales", _c_ptr), ("g_dec", _c_ptr),
                ("rows", _c_i64), ("K", _c_i64)]


class avr_fp8(ctypes.Structure):
    _fields_ = [("codes", _c_ptr), ("scales", _c_ptr), ("rows", _c_i64), ("K", _c_i64)]


_SIGS = {
    "avr_nvfp4_scales_bytes": (_c_size, [_c_i64, _c_i64]),
    "averis_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "averis_workspace_init": (_c_int, [_c_ptr, _c_size, _c_ptr]),
    "averis_check_status": (_c_int, [_c_ptr, _c_ptr]),
    "averis_set_wait_limit": (_c_int, [_c_ptr, _c_size, _c_u64, _c_ptr]),
    "averis_probe_mma_rate": (_c_int, [_c_int, _c_int, _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "averis_status_string": (ctypes.c_char_p, [_c_int]),
    "averis_split_quant": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_int, _c_u64, _c_u64, _c_int,
                                    _c_ptr, ctypes.POINTER(avr_nvfp4), ctypes.POINTER(avr_nvfp4),
                                    _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "averis_moe_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int]),
    "averis_moe_quant_weights": (_c_int, [_c_ptr, _c_int, _c_int, _c_i64, _c_i64, ctypes.POINTER(avr_nvfp4),
                                          ctypes.POINTER(avr_nvfp4), _c_ptr, _c_size, _c_ptr]),
    "averis_moe_split_quant": (_c_int, [_c_ptr, _c_int, _c_i64, _c_ptr, _c_int, _c_i64, _c_int, _c_u64, _c_u64,
                                        _c_int, _c_ptr, ctypes.POINTER(avr_nvfp4), ctypes.POINTER(avr_nvfp4),
                                        _c_ptr, _c_size, _c_ptr]),
    "averis_moe_linear_fwd": (_c_int, [_c_ptr, _c_int, _c_i64, _c_ptr, _c_int, _c_i64, _c_i64,
                                       ctypes.POINTER(avr_nvfp4), _c_int, _c_u64, _c_u64, _c_ptr, _c_int, _c_ptr,
                                       _c_size, _c_ptr]),
    "averis_moe_linear_dgrad": (_c_int, [_c_ptr, _c_int, _c_i64, _c_ptr, _c_int, _c_i64, _c_i64,
                                         ctypes.POINTER(avr_nvfp4), _c_int, _c_u64, _c_u64, _c_ptr, _c_int,
                                         _c_ptr, _c_size, _c_ptr]),
    "averis_split_quant_fused": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_int, _c_u64, _c_u64, _c_int,
                                          _c_ptr, ctypes.POINTER(avr_nvfp4), ctypes.POINTER(avr_nvfp4),
                                          _c_ptr, _c_size, _c_ptr]),
    "averis_split_quant_t": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_int, _c_u64, _c_u64, _c_int,
                                      _c_ptr, ctypes.POINTER(avr_nvfp4), ctypes.POINTER(avr_nvfp4),
                                      _c_ptr, _c_size, _c_ptr]),
    "nvfp4_quant_t": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_int, _c_u64, _c_u64, _c_int,
                               ctypes.POINTER(avr_nvfp4), _c_ptr, _c_size, _c_ptr]),
    "averis_wgrad_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "averis_wgrad_gemm": (_c_int, [ctypes.POINTER(avr_nvfp4), ctypes.POINTER(avr_nvfp4),
                                   ctypes.POINTER(avr_nvfp4), ctypes.POINTER(avr_nvfp4), _c_i64,
                                   _c_ptr, _c_int, _c_ptr, _c_size, _c_ptr]),
    "averis_linear_wgrad": (_c_int, [_c_ptr, _c_int, _c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_int,
                                     _c_u64, _c_u64, _c_ptr, _c_int, _c_ptr, _c_size, _c_ptr]),
    "nvfp4_linear_wgrad": (_c_int, [_c_ptr, _c_int, _c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_int,
                                    _c_u64, _c_u64, _c_ptr, _c_int, _c_ptr, _c_size, _c_ptr]),
    "averis_mean_energy_ratio": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr,
                                          _c_size, _c_ptr]),
    "nvfp4_quant": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_int, _c_u64, _c_u64, _c_int,
                             ctypes.POINTER(avr_nvfp4), _c_ptr, _c_size, _c_ptr]),
    "averis_quant_weight": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, ctypes.POINTER(avr_nvfp4),
                                     ctypes.POINTER(avr_nvfp4), _c_ptr, _c_size, _c_ptr]),
    "averis_bias_row": (_c_int, [ctypes.POINTER(avr_nvfp4), ctypes.POINTER(avr_nvfp4), _c_ptr,
                                 _c_ptr, _c_size, _c_ptr]),
    "nvfp4_gemm": (_c_int, [ctypes.POINTER(avr_nvfp4), ctypes.POINTER(avr_nvfp4), _c_ptr, _c_ptr,
                            _c_int, _c_ptr, _c_size, _c_ptr]),
    "averis_linear_fwd": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, ctypes.POINTER(avr_nvfp4),
                                   _c_int, _c_u64, _c_u64, _c_ptr, _c_int, ctypes.POINTER(avr_nvfp4),
                                   ctypes.POINTER(avr_nvfp4), _c_ptr, _c_size, _c_ptr]),
    "averis_linear_dgrad": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, ctypes.POINTER(avr_nvfp4),
                                     _c_int, _c_u64, _c_u64, _c_ptr, _c_int, _c_ptr, _c_size, _c_ptr]),
    "nvfp4_linear_fwd": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, ctypes.POINTER(avr_nvfp4),
                                  _c_int, _c_u64, _c_u64, _c_ptr, _c_int, _c_ptr, _c_size, _c_ptr]),
    "nvfp4_linear_dgrad": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, ctypes.POINTER(avr_nvfp4),
                                    _c_int, _c_u64, _c_u64, _c_ptr, _c_int, _c_ptr, _c_size, _c_ptr]),
    "averis_probe_convert": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_i64, _c_ptr]),
    "averis_probe_philox": (_c_int, [_c_u64, _c_u64, _c_u32, _c_i64, _c_ptr, _c_ptr]),
    "averis_probe_convert_sr": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_i64, _c_ptr]),
}

_c_fp8 = ctypes.POINTER(avr_fp8)
_WS = [_c_ptr, _c_size, _c_ptr]                     # ws, ws_bytes, stream
_PERM = [_c_int, _c_i64, _c_int, _c_i64, _c_ptr]    # dtype, T, k, H, row
_SIGS.update({
    "moe_route_workspace_size": (_c_size, [_c_i64, _c_int, _c_int]),
    "moe_route": (_c_int, [_c_ptr, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_ptr, _c_ptr] + _WS),
    "moe_route_bwd": (_c_int, [_c_ptr, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_ptr]
                      + _WS),
    "moe_sort": (_c_int, [_c_ptr, _c_i64, _c_int, _c_int, _c_i64, _c_ptr, _c_ptr] + _WS),
    "moe_dispatch": (_c_int, [_c_ptr] + _PERM + [_c_i64, _c_ptr] + _WS),
    "moe_dispatch_bwd": (_c_int, [_c_ptr] + _PERM + [_c_i64, _c_ptr] + _WS),
    "moe_combine": (_c_int, [_c_ptr] + _PERM + [_c_ptr, _c_i64, _c_ptr] + _WS),
    "moe_combine_bwd": (_c_int, [_c_ptr, _c_ptr] + _PERM + [_c_ptr, _c_i64, _c_ptr, _c_ptr] + _WS),
    "moe_combine_f32": (_c_int, [_c_ptr] + _PERM + [_c_ptr, _c_i64, _c_ptr] + _WS),
    "moe_combine_f32_bwd": (_c_int, [_c_ptr, _c_ptr] + _PERM + [_c_ptr, _c_i64, _c_ptr, _c_ptr] + _WS),
    "avr_fp8_scales_bytes": (_c_size, [_c_i64, _c_i64]),
    "fp8_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "fp8_quant": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_fp8] + _WS),
    "fp8_quant_t": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_fp8] + _WS),
    "fp8_quant_weight": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_fp8, _c_fp8] + _WS),
    "fp8_gemm": (_c_int, [_c_fp8, _c_fp8, _c_ptr, _c_int] + _WS),
    "fp8_linear_fwd": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_fp8, _c_ptr, _c_int] + _WS),
    "fp8_linear_dgrad": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_fp8, _c_ptr, _c_int] + _WS),
    "fp8_linear_wgrad": (_c_int, [_c_ptr, _c_int, _c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_ptr, _c_int] + _WS),
    "fp8_moe_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int]),
    "fp8_moe_quant_weights": (_c_int, [_c_ptr, _c_int, _c_int, _c_i64, _c_i64, _c_fp8, _c_fp8] + _WS),
    "fp8_moe_dispatch": (_c_int, [_c_ptr] + _PERM + [_c_fp8] + _WS),
    "fp8_moe_gemm": (_c_int, [_c_fp8, _c_ptr, _c_int, _c_fp8, _c_ptr, _c_int] + _WS),
    "fp8_moe_linear_fwd": (_c_int, [_c_ptr, _c_int, _c_i64, _c_ptr, _c_int, _c_i64, _c_i64, _c_fp8, _c_ptr, _c_int]
                           + _WS),
    "fp8_moe_linear_dgrad": (_c_int, [_c_ptr, _c_int, _c_i64, _c_ptr, _c_int, _c_i64, _c_i64, _c_fp8, _c_ptr, _c_int]
                             + _WS),
    "fp8_moe_linear_wgrad": (_c_int, [_c_ptr, _c_int, _c_ptr, _c_int, _c_i64, _c_ptr, _c_int, _c_i64, _c_i64, _c_ptr,
                                      _c_int] + _WS),
})


def library_path():
    return _build.LIB


def load():
    """Load libaveris.so (built in-tree); raise if it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise AverisError(AVR_ERR_NO_DEVICE,
                          f"{path} is missing; build it with python -m quantized_gemm_column_b200.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def _check(st, where):
    if st != AVR_OK:
        raise AverisError(st, where)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return AVR_BF16
    if t.dtype == torch.float32:
        return AVR_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _round(rm):
    return {"rne": AVR_RNE, "sr": AVR_SR, AVR_RNE: AVR_RNE, AVR_SR: AVR_SR}[rm]


class NVFP4Tensor:
    """Device storage of an NVFP4 tensor [rows, K]: packed codes, E4M3 scales
    in the tcgen05 atom layout and the fp32 decode scale."""

    def __init__(self, rows, K, device="cuda"):
        self.rows, self.K = int(rows), int(K)
        self.codes = torch.empty((self.rows, self.K // 2), dtype=torch.uint8, device=device)
        nbytes = ((self.rows + 127) // 128 * 128) * (self.K // 16)
        self.scales = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.g_dec = torch.empty(1, dtype=torch.float32, device=device)

    def struct(self):
        return avr_nvfp4(self.codes.data_ptr(), self.scales.data_ptr(), self.g_dec.data_ptr(),
                         self.rows, self.K)


def _s(t):
    return None if t is None else ctypes.byref(t.struct())


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def avr_nvfp4_scales_bytes(rows, K):
    return int(load().avr_nvfp4_scales_bytes(rows, K))


def averis_workspace_size(l, K, N=0):
    return int(load().averis_workspace_size(l, K, N))


def status_string(st):
    return load().averis_status_string(int(st)).decode()


averis_status_string = status_string


def workspace(l, K, N=0, device="cuda", stream=None):
    """Allocate and zero-fill a workspace for the given sizes."""
    n = averis_workspace_size(l, K, N)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    averis_workspace_init(ws, stream)
    return ws


def averis_workspace_init(ws, stream=None):
    _check(load().averis_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "averis_workspace_init")


def averis_check_status(ws, stream=None):
    """Synchronize and return the latched device status (0 = ok)."""
    return int(load().averis_check_status(_ptr(ws), _stream(stream)))


def averis_probe_mma_rate(iters, ns, ws, stream=None):
    """MMA-only tcgen05 FP4 loop on ns.numel() CTAs; ns (int64, device) gets
    each CTA's elapsed nanoseconds."""
    _check(load().averis_probe_mma_rate(int(iters), ns.numel(), _ptr(ns), _ptr(ws), ws.numel(), _stream(stream)),
           "averis_probe_mma_rate")


def averis_set_wait_limit(ws, limit_ns, stream=None):
    """Bound (ns) of the waits on other CTAs; 0 restores the default 2 s."""
    _check(load().averis_set_wait_limit(_ptr(ws), ws.numel(), int(limit_ns), _stream(stream)),
           "averis_set_wait_limit")


def averis_split_quant(X, rm, seed, offset, grad, mu, mu_q, xr_q, xr_debug, ws, stream=None):
    l, K = X.shape
    _check(load().averis_split_quant(_ptr(X), _dtype(X), l, K, _round(rm), seed, offset, int(grad),
                                     _ptr(mu), _s(mu_q), _s(xr_q), _ptr(xr_debug), _ptr(ws),
                                     ws.numel(), _stream(stream)), "averis_split_quant")


def padded_tokens(l):
    """The token axis of the weight-gradient operands: l rounded up to 64."""
    return (int(l) + 63) // 64 * 64


def averis_wgrad_workspace_size(l, m, n):
    return int(load().averis_wgrad_workspace_size(l, m, n))


def wgrad_workspace(l, m, n, device="cuda"):
    """A zero-initialised workspace for the weight-gradient calls."""
    return torch.zeros(averis_wgrad_workspace_size(l, m, n), dtype=torch.uint8, device=device)


def averis_split_quant_t(X, rm, seed, offset, grad, mu, mu_q, xrt_q, ws, stream=None):
    l, K = X.shape
    _check(load().averis_split_quant_t(_ptr(X), _dtype(X), l, K, _round(rm), seed, offset, int(grad),
                                       _ptr(mu), _s(mu_q), _s(xrt_q), _ptr(ws), ws.numel(),
                                       _stream(stream)), "averis_split_quant_t")


def nvfp4_quant_t(X, rm, seed, offset, grad, out, ws, stream=None):
    l, K = X.shape
    _check(load().nvfp4_quant_t(_ptr(X), _dtype(X), l, K, _round(rm), seed, offset, int(grad),
                                _s(out), _ptr(ws), ws.numel(), _stream(stream)), "nvfp4_quant_t")


def averis_wgrad_gemm(xrt_q, drt_q, mu_x_q, mu_d_q, l, dW, ws, stream=None):
    _check(load().averis_wgrad_gemm(_s(xrt_q), _s(drt_q), _s(mu_x_q), _s(mu_d_q), l, _ptr(dW),
                                    _dtype(dW), _ptr(ws), ws.numel(), _stream(stream)),
           "averis_wgrad_gemm")


def averis_linear_wgrad(X, D, rm, seed, offset, dW, ws, stream=None):
    l, m = X.shape
    n = D.shape[1]
    _check(load().averis_linear_wgrad(_ptr(X), _dtype(X), _ptr(D), _dtype(D), l, m, n, _round(rm),
                                      seed, offset, _ptr(dW), _dtype(dW), _ptr(ws), ws.numel(),
                                      _stream(stream)), "averis_linear_wgrad")


def nvfp4_linear_wgrad(X, D, rm, seed, offset, dW, ws, stream=None):
    l, m = X.shape
    n = D.shape[1]
    _check(load().nvfp4_linear_wgrad(_ptr(X), _dtype(X), _ptr(D), _dtype(D), l, m, n, _round(rm),
                                     seed, offset, _ptr(dW), _dtype(dW), _ptr(ws), ws.numel(),
                                     _stream(stream)), "nvfp4_linear_wgrad")


def averis_mean_energy_ratio(X, mu, R, ws, stream=None):
    """R = ||mu_X|| / sqrt(E||x||^2 / m) into the 1-element fp32 device tensor R."""
    l, K = X.shape
    _check(load().averis_mean_energy_ratio(_ptr(X), _dtype(X), l, K, _ptr(mu), _ptr(R), _ptr(ws),
                                           ws.numel(), _stream(stream)), "averis_mean_energy_ratio")


class NVFP4Group(NVFP4Tensor):
    """An NVFP4 tensor [rows, K] with one decode scale per expert (MoE calls)."""

    def __init__(self, rows, K, groups, device="cuda"):
        super().__init__(rows, K, device)
        self.g_dec = torch.empty(groups, dtype=torch.float32, device=device)


def moe_padded_rows(counts):
    """Rows the permuted buffer needs: every expert's count rounded up to 128."""
    return sum((int(c) + 127) // 128 * 128 for c in counts)


def averis_moe_workspace_size(l_cap, K, N, E):
    return int(load().averis_moe_workspace_size(l_cap, K, N, E))


def moe_workspace(l_cap, K, N, E, device="cuda", stream=None):
    ws = torch.empty(averis_moe_workspace_size(l_cap, K, N, E), dtype=torch.uint8, device=device)
    averis_workspace_init(ws, stream)
    return ws


def averis_moe_quant_weights(W, w_fwd, w_dgrad, ws, stream=None):
    E, m, n = W.shape
    _check(load().averis_moe_quant_weights(_ptr(W), _dtype(W), E, m, n, _s(w_fwd), _s(w_dgrad), _ptr(ws),
                                           ws.numel(), _stream(stream)), "averis_moe_quant_weights")


def averis_moe_split_quant(X, counts, rm, seed, offset, grad, mu, mu_q, xr_q, ws, stream=None):
    l_cap, K = X.shape
    _check(load().averis_moe_split_quant(_ptr(X), _dtype(X), l_cap, _ptr(counts), counts.numel(), K, _round(rm),
                                         seed, offset, int(grad), _ptr(mu), _s(mu_q), _s(xr_q), _ptr(ws),
                                         ws.numel(), _stream(stream)), "averis_moe_split_quant")


def averis_moe_linear_fwd(X, counts, w_fwd, rm, seed, offset, Y, ws, stream=None):
    l_cap, m = X.shape
    n = Y.shape[1]
    _check(load().averis_moe_linear_fwd(_ptr(X), _dtype(X), l_cap, _ptr(counts), counts.numel(), m, n,
                                        _s(w_fwd), _round(rm), seed, offset, _ptr(Y), _dtype(Y), _ptr(ws),
                                        ws.numel(), _stream(stream)), "averis_moe_linear_fwd")


def averis_moe_linear_dgrad(D, counts, w_dgrad, rm, seed, offset, dX, ws, stream=None):
    l_cap, n = D.shape
    m = dX.shape[1]
    _check(load().averis_moe_linear_dgrad(_ptr(D), _dtype(D), l_cap, _ptr(counts), counts.numel(), m, n,
                                          _s(w_dgrad), _round(rm), seed, offset, _ptr(dX), _dtype(dX), _ptr(ws),
                                          ws.numel(), _stream(stream)), "averis_moe_linear_dgrad")


def averis_split_quant_fused(X, rm, seed, offset, grad, mu, mu_q, xr_q, ws, stream=None):
    l, K = X.shape
    _check(load().averis_split_quant_fused(_ptr(X), _dtype(X), l, K, _round(rm), seed, offset, int(grad),
                                           _ptr(mu), _s(mu_q), _s(xr_q), _ptr(ws), ws.numel(),
                                           _stream(stream)), "averis_split_quant_fused")


def nvfp4_quant(X, rm, seed, offset, grad, out, ws, stream=None):
    rows, K = X.shape
    _check(load().nvfp4_quant(_ptr(X), _dtype(X), rows, K, _round(rm), seed, offset, int(grad),
                              _s(out), _ptr(ws), ws.numel(), _stream(stream)), "nvfp4_quant")


def averis_quant_weight(W, w_fwd, w_dgrad, ws, stream=None):
    m, n = W.shape
    _check(load().averis_quant_weight(_ptr(W), _dtype(W), m, n, _s(w_fwd), _s(w_dgrad), _ptr(ws),
                                      ws.numel(), _stream(stream)), "averis_quant_weight")


def averis_bias_row(mu_q, w_q, bias, ws, stream=None):
    _check(load().averis_bias_row(_s(mu_q), _s(w_q), _ptr(bias), _ptr(ws), ws.numel(),
                                  _stream(stream)), "averis_bias_row")


def nvfp4_gemm(a, b, bias, Y, ws, stream=None):
    _check(load().nvfp4_gemm(_s(a), _s(b), _ptr(bias), _ptr(Y), _dtype(Y), _ptr(ws), ws.numel(),
                             _stream(stream)), "nvfp4_gemm")


def averis_linear_fwd(X, w_fwd, rm, seed, offset, Y, ws, save_xr=None, save_mu=None, stream=None):
    l, m = X.shape
    n = w_fwd.rows
    _check(load().averis_linear_fwd(_ptr(X), _dtype(X), l, m, n, _s(w_fwd), _round(rm), seed, offset,
                                    _ptr(Y), _dtype(Y), _s(save_xr), _s(save_mu), _ptr(ws),
                                    ws.numel(), _stream(stream)), "averis_linear_fwd")


def averis_linear_dgrad(D, w_dgrad, rm, seed, offset, dX, ws, stream=None):
    l, n = D.shape
    m = w_dgrad.rows
    _check(load().averis_linear_dgrad(_ptr(D), _dtype(D), l, m, n, _s(w_dgrad), _round(rm), seed,
                                      offset, _ptr(dX), _dtype(dX), _ptr(ws), ws.numel(),
                                      _stream(stream)), "averis_linear_dgrad")


def nvfp4_linear_fwd(X, w_fwd, rm, seed, offset, Y, ws, stream=None):
    l, m = X.shape
    n = w_fwd.rows
    _check(load().nvfp4_linear_fwd(_ptr(X), _dtype(X), l, m, n, _s(w_fwd), _round(rm), seed, offset,
                                   _ptr(Y), _dtype(Y), _ptr(ws), ws.numel(), _stream(stream)),
           "nvfp4_linear_fwd")


def nvfp4_linear_dgrad(D, w_dgrad, rm, seed, offset, dX, ws, stream=None):
    l, n = D.shape
    m = w_dgrad.rows
    _check(load().nvfp4_linear_dgrad(_ptr(D), _dtype(D), l, m, n, _s(w_dgrad), _round(rm), seed,
                                     offset, _ptr(dX), _dtype(dX), _ptr(ws), ws.numel(),
                                     _stream(stream)), "nvfp4_linear_dgrad")


def averis_probe_convert(x, e4m3, e2m1, stream=None):
    _check(load().averis_probe_convert(_ptr(x), _ptr(e4m3), _ptr(e2m1), x.numel(), _stream(stream)),
           "averis_probe_convert")


def averis_probe_convert_sr(x, rbits, out, stream=None):
    _check(load().averis_probe_convert_sr(_ptr(x), _ptr(rbits), _ptr(out), rbits.numel(), _stream(stream)),
           "averis_probe_convert_sr")


def averis_probe_philox(seed, offset, tag, n, out, stream=None):
    _check(load().averis_probe_philox(seed, offset, tag, n, _ptr(out), _stream(stream)),
           "averis_probe_philox")


# ---------------------------------------------------------------------------
# split quantization without a caller workspace
# ---------------------------------------------------------------------------
_SIGS["averis_split_quant_noalloc"] = (
    _c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_int, _c_u64, _c_u64, _c_int, _c_ptr,
             ctypes.POINTER(avr_nvfp4), ctypes.POINTER(avr_nvfp4), _c_ptr, _c_ptr, _c_ptr])


def averis_split_quant_noalloc(X, rm, seed, offset, grad, mu, mu_q, xr_q, xr_debug,
                               device_status=None, stream=None):
    """averis_split_quant without a workspace, for callers that cannot
    allocate device memory; its scratch is a fixed 4 MiB array inside the
    library (see include/averis.h for the size limit and the rules)."""
    l, K = X.shape
    _check(load().averis_split_quant_noalloc(_ptr(X), _dtype(X), l, K, _round(rm), seed, offset,
                                             int(grad), _ptr(mu), _s(mu_q), _s(xr_q), _ptr(xr_debug),
                                             _ptr(device_status), _stream(stream)),
           "averis_split_quant_noalloc")


# ---------------------------------------------------------------------------
# routing and 8-bit calls: the tensors are contiguous and on the current
# device, else AverisError (invalid argument) before any launch
# ---------------------------------------------------------------------------
# A decoding step's calls are bound by the host, so these wrappers take the
# device and the stream as plain integers (torch.cuda.current_stream() builds
# a Stream object, 3 us of a 5 us call), look at every tensor once and keep no
# generic layer between.
_device = getattr(torch._C, "_cuda_getDevice", None)               # absent from a torch without CUDA
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_DT = {torch.bfloat16: AVR_BF16, torch.float32: AVR_F32}
_I32, _F32 = torch.int32, torch.float32


def _call(name, stream, ws, tensors, args):
    """The entry point with ws, its size and the stream appended."""
    dev = _device()
    for t in tensors:
        if t.get_device() != dev or not t.is_contiguous():
            _refuse_tensor(name, dev)
    if ws.get_device() != dev or not ws.is_contiguous():
        _refuse_tensor(name, dev)
    st = getattr(_LIB or load(), name)(*args, ws.data_ptr(), ws.nbytes,
                                       _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise AverisError(st, name)


def _refuse_tensor(name, dev):
    raise AverisError(AVR_ERR_INVALID_ARG, f"{name}: every tensor must be contiguous and on device {dev}")


def _refuse_shape(name, *want):
    """want: (tensor, shape, dtype) triples, one of which does not hold."""
    for t, shape, dtype in want:
        if t.shape != shape or t.dtype is not dtype:
            raise AverisError(AVR_ERR_INVALID_ARG,
                              f"{name}: expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    raise AverisError(AVR_ERR_INVALID_ARG, name)


def _dt(t):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _route_workspace(n, device, stream):
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    averis_workspace_init(ws, stream)
    return ws


def _positive(n, where):
    if n == 0:
        raise AverisError(AVR_ERR_UNSUPPORTED_SHAPE, where)
    return n


def moe_route_workspace_size(T, k, E):
    return int(load().moe_route_workspace_size(T, k, E))


def moe_route_workspace(T, k, E, device="cuda", stream=None):
    """A workspace for the routing calls of T tokens, k slots, E experts."""
    return _route_workspace(_positive(moe_route_workspace_size(T, k, E), "moe_route_workspace"), device, stream)


def moe_max_rows(T, k, E):
    """Rows of an experts' buffer that any routing of T tokens to k of E experts fits in."""
    return (T * k + 127 * min(E, T * k)) // 128 * 128


def moe_route(logits, norm, ids, weights, ws, stream=None):
    T, E = logits.shape
    iT, k = shape = ids.shape
    if iT != T or ids.dtype is not _I32 or weights.shape != shape or weights.dtype is not _F32:
        _refuse_shape("moe_route", (ids, (T, k), _I32), (weights, (T, k), _F32))
    _call("moe_route", stream, ws, (logits, ids, weights),
          (logits.data_ptr(), _dt(logits), T, E, k, 1 if norm else 0, ids.data_ptr(), weights.data_ptr()))


def moe_route_bwd(logits, norm, ids, weights, dweights, dlogits, ws, stream=None):
    """logits may be None when norm is true."""
    T, E = full = dlogits.shape
    k = ids.shape[1]
    shape = (T, k)
    if ids.shape != shape or ids.dtype is not _I32 or weights.shape != shape or weights.dtype is not _F32 \
            or dweights.shape != shape or dweights.dtype is not _F32 \
            or (logits is not None and (logits.shape != full or logits.dtype is not dlogits.dtype)):
        _refuse_shape("moe_route_bwd", (ids, shape, _I32), (weights, shape, _F32), (dweights, shape, _F32),
                      (dlogits if logits is None else logits, full, dlogits.dtype))
    _call("moe_route_bwd", stream, ws,
          (ids, weights, dweights, dlogits) + (() if logits is None else (logits,)),
          (None if logits is None else logits.data_ptr(), _dt(dlogits), T, E, k, 1 if norm else 0, ids.data_ptr(),
           weights.data_ptr(), dweights.data_ptr(), dlogits.data_ptr()))


def moe_sort(ids, l_cap, counts, row, ws, stream=None):
    T, k = shape = ids.shape
    if ids.dtype is not _I32 or row.shape != shape or row.dtype is not _I32 or counts.dtype is not _I32 \
            or counts.dim() != 1:
        _refuse_shape("moe_sort", (ids, shape, _I32), (row, shape, _I32), (counts, (counts.numel(),), _I32))
    _call("moe_sort", stream, ws, (ids, counts, row),
          (ids.data_ptr(), T, k, counts.shape[0], l_cap, counts.data_ptr(), row.data_ptr()))


def moe_dispatch(X, row, Xp, ws, stream=None):
    T, H = X.shape
    (rT, k), (l_cap, pH) = row.shape, Xp.shape
    if rT != T or pH != H or row.dtype is not _I32 or Xp.dtype is not X.dtype:
        _refuse_shape("moe_dispatch", (row, (T, k), _I32), (Xp, (l_cap, H), X.dtype))
    _call("moe_dispatch", stream, ws, (X, row, Xp),
          (X.data_ptr(), _dt(X), T, k, H, row.data_ptr(), l_cap, Xp.data_ptr()))


def moe_dispatch_bwd(dXp, row, dX, ws, stream=None):
    T, H = dX.shape
    (rT, k), (l_cap, pH) = row.shape, dXp.shape
    if rT != T or pH != H or row.dtype is not _I32 or dXp.dtype is not dX.dtype:
        _refuse_shape("moe_dispatch_bwd", (row, (T, k), _I32), (dXp, (l_cap, H), dX.dtype))
    _call("moe_dispatch_bwd", stream, ws, (dXp, row, dX),
          (dXp.data_ptr(), _dt(dX), T, k, H, row.data_ptr(), l_cap, dX.data_ptr()))


def moe_combine(Yp, row, weights, Y, ws, stream=None):
    T, H = Y.shape
    T_k = rT, k = row.shape
    l_cap, pH = Yp.shape
    if rT != T or pH != H or row.dtype is not _I32 or weights.shape != T_k or weights.dtype is not _F32 \
            or Yp.dtype is not Y.dtype:
        _refuse_shape("moe_combine", (row, (T, k), _I32), (weights, (T, k), _F32), (Yp, (l_cap, H), Y.dtype))
    _call("moe_combine", stream, ws, (Yp, row, weights, Y),
          (Yp.data_ptr(), _dt(Y), T, k, H, row.data_ptr(), weights.data_ptr(), l_cap, Y.data_ptr()))


def moe_combine_bwd(dY, Yp, row, weights, dYp, dweights, ws, stream=None):
    T, H = dY.shape
    T_k = rT, k = row.shape
    buf = l_cap, pH = Yp.shape
    if rT != T or pH != H or row.dtype is not _I32 or weights.shape != T_k or weights.dtype is not _F32 \
            or dweights.shape != T_k or dweights.dtype is not _F32 or Yp.dtype is not dY.dtype \
            or dYp.shape != buf or dYp.dtype is not dY.dtype:
        _refuse_shape("moe_combine_bwd", (row, (T, k), _I32), (weights, (T, k), _F32), (dweights, (T, k), _F32),
                      (Yp, (l_cap, H), dY.dtype), (dYp, (l_cap, H), dY.dtype))
    _call("moe_combine_bwd", stream, ws, (dY, Yp, row, weights, dYp, dweights),
          (dY.data_ptr(), Yp.data_ptr(), _dt(dY), T, k, H, row.data_ptr(), weights.data_ptr(), l_cap,
           dYp.data_ptr(), dweights.data_ptr()))


def moe_combine_f32(Yp, row, weights, Y, ws, stream=None):
    """Yp is fp32, Y of either type."""
    T, H = Y.shape
    T_k = rT, k = row.shape
    l_cap, pH = Yp.shape
    if rT != T or pH != H or row.dtype is not _I32 or weights.shape != T_k or weights.dtype is not _F32 \
            or Yp.dtype is not _F32:
        _refuse_shape("moe_combine_f32", (row, (T, k), _I32), (weights, (T, k), _F32), (Yp, (l_cap, H), _F32))
    _call("moe_combine_f32", stream, ws, (Yp, row, weights, Y),
          (Yp.data_ptr(), _dt(Y), T, k, H, row.data_ptr(), weights.data_ptr(), l_cap, Y.data_ptr()))


def moe_combine_f32_bwd(dY, Yp, row, weights, dYp, dweights, ws, stream=None):
    """Yp is fp32, dY and dYp of one type, either."""
    T, H = dY.shape
    T_k = rT, k = row.shape
    buf = l_cap, pH = Yp.shape
    if rT != T or pH != H or row.dtype is not _I32 or weights.shape != T_k or weights.dtype is not _F32 \
            or dweights.shape != T_k or dweights.dtype is not _F32 or Yp.dtype is not _F32 \
            or dYp.shape != buf or dYp.dtype is not dY.dtype:
        _refuse_shape("moe_combine_f32_bwd", (row, (T, k), _I32), (weights, (T, k), _F32), (dweights, (T, k), _F32),
                      (Yp, (l_cap, H), _F32), (dYp, (l_cap, H), dY.dtype))
    _call("moe_combine_f32_bwd", stream, ws, (dY, Yp, row, weights, dYp, dweights),
          (dY.data_ptr(), Yp.data_ptr(), _dt(dY), T, k, H, row.data_ptr(), weights.data_ptr(), l_cap,
           dYp.data_ptr(), dweights.data_ptr()))


class FP8Tensor:
    """Device storage of an 8-bit tensor [rows, K]: E4M3 codes and one scale
    byte per row and 128 elements of K in the atom layout of averis.h."""

    def __init__(self, rows, K, device="cuda"):
        n = avr_fp8_scales_bytes(rows, K)
        if rows > 0 and K != 0:          # [K, 0]: fp8_quant_t of no tokens
            _positive(n, "FP8Tensor")
        self._hold(torch.empty((int(rows), int(K)), dtype=torch.uint8, device=device),
                   torch.empty(n, dtype=torch.uint8, device=device))

    @classmethod
    def of(cls, codes, scales):
        """The tensor held by codes [rows, K] and scales (uint8, not copied)."""
        rows, K = codes.shape
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 \
                or scales.numel() != avr_fp8_scales_bytes(rows, K):
            raise AverisError(AVR_ERR_INVALID_ARG, "FP8Tensor.of")
        t = cls.__new__(cls)
        t._hold(codes, scales)
        return t

    def _hold(self, codes, scales):
        self._parts = (codes, scales)
        self._c = avr_fp8(0, 0, codes.shape[0], codes.shape[1])
        self._ref = ctypes.byref(self._c)

    codes = property(lambda self: self._parts[0])
    scales = property(lambda self: self._parts[1])
    rows = property(lambda self: self._c.rows)
    K = property(lambda self: self._c.K)

    def struct(self):
        c, (codes, scales) = self._c, self._parts
        c.codes, c.scales = codes.data_ptr(), scales.data_ptr()
        return c


def _q(t):
    """(a reference to the descriptor, its tensors) of an FP8Tensor or None."""
    if t is None:
        return None, ()
    t.struct()
    return t._ref, t._parts


def avr_fp8_scales_bytes(rows, K):
    return int(load().avr_fp8_scales_bytes(rows, K))


def fp8_workspace_size(l, m, n):
    return int(load().fp8_workspace_size(l, m, n))


def fp8_workspace(l, m, n, device="cuda", stream=None):
    """A workspace for the 8-bit calls of l tokens, m input and n output features."""
    return _route_workspace(_positive(fp8_workspace_size(l, m, n), "fp8_workspace"), device, stream)


def fp8_quant(X, out, ws, stream=None):
    rows, K = X.shape
    q, t = _q(out)
    _call("fp8_quant", stream, ws, (X,) + t, (X.data_ptr(), _dt(X), rows, K, q))


def fp8_quant_t(X, out, ws, stream=None):
    """out: FP8Tensor(K, l rounded up to 128)."""
    l, K = X.shape
    q, t = _q(out)
    _call("fp8_quant_t", stream, ws, (X,) + t, (X.data_ptr(), _dt(X), l, K, q))


def fp8_quant_weight(W, w_fwd, w_dgrad, ws, stream=None):
    """w_dgrad may be None."""
    m, n = W.shape
    (f, tf), (d, td) = _q(w_fwd), _q(w_dgrad)
    _call("fp8_quant_weight", stream, ws, (W,) + tf + td, (W.data_ptr(), _dt(W), m, n, f, d))


def fp8_gemm(a, b, Y, ws, stream=None):
    (qa, ta), (qb, tb) = _q(a), _q(b)
    if Y.shape != (a.rows, b.rows):
        _refuse_shape("fp8_gemm", (Y, (a.rows, b.rows), Y.dtype))
    _call("fp8_gemm", stream, ws, (Y,) + ta + tb, (qa, qb, Y.data_ptr(), _dt(Y)))


def fp8_linear_fwd(X, w_fwd, Y, ws, stream=None):
    (l, m), (q, t) = X.shape, _q(w_fwd)
    n = w_fwd.rows
    if Y.shape != (l, n):
        _refuse_shape("fp8_linear_fwd", (Y, (l, n), Y.dtype))
    _call("fp8_linear_fwd", stream, ws, (X, Y) + t, (X.data_ptr(), _dt(X), l, m, n, q, Y.data_ptr(), _dt(Y)))


def fp8_linear_dgrad(D, w_dgrad, dX, ws, stream=None):
    (l, n), (q, t) = D.shape, _q(w_dgrad)
    m = w_dgrad.rows
    if dX.shape != (l, m):
        _refuse_shape("fp8_linear_dgrad", (dX, (l, m), dX.dtype))
    _call("fp8_linear_dgrad", stream, ws, (D, dX) + t, (D.data_ptr(), _dt(D), l, m, n, q, dX.data_ptr(), _dt(dX)))


def fp8_linear_wgrad(X, D, dW, ws, stream=None):
    (l, m), (dl, n) = X.shape, D.shape
    if dl != l or dW.shape != (m, n):
        _refuse_shape("fp8_linear_wgrad", (D, (l, n), D.dtype), (dW, (m, n), dW.dtype))
    _call("fp8_linear_wgrad", stream, ws, (X, D, dW),
          (X.data_ptr(), _dt(X), D.data_ptr(), _dt(D), l, m, n, dW.data_ptr(), _dt(dW)))


def fp8_moe_workspace_size(l_cap, m, n, E):
    return int(load().fp8_moe_workspace_size(l_cap, m, n, E))


def fp8_moe_workspace(l_cap, m, n, E, slots=0, device="cuda", stream=None):
    """A workspace for the experts' 8-bit calls, and for the routing calls of
    up to `slots` = T k slots."""
    need = _positive(fp8_moe_workspace_size(l_cap, m, n, E), "fp8_moe_workspace")
    return _route_workspace(max(need, moe_route_workspace_size(slots, 1, E)), device, stream)


def fp8_moe_quant_weights(W, w_fwd, w_dgrad, ws, stream=None):
    """w_dgrad may be None."""
    E, m, n = W.shape
    (f, tf), (d, td) = _q(w_fwd), _q(w_dgrad)
    _call("fp8_moe_quant_weights", stream, ws, (W,) + tf + td, (W.data_ptr(), _dt(W), E, m, n, f, d))


def fp8_moe_dispatch(X, row, xq, ws, stream=None):
    (T, K), (rT, k), (q, t) = X.shape, row.shape, _q(xq)
    if rT != T or row.dtype is not _I32:
        _refuse_shape("fp8_moe_dispatch", (row, (T, k), _I32))
    _call("fp8_moe_dispatch", stream, ws, (X, row) + t, (X.data_ptr(), _dt(X), T, k, K, row.data_ptr(), q))


def fp8_moe_gemm(xq, counts, w, Y, ws, stream=None):
    (qx, tx), (qw, tw) = _q(xq), _q(w)
    E = counts.numel()
    want = (xq.rows, w.rows // (E or 1))
    if counts.dtype is not _I32 or Y.shape != want:
        _refuse_shape("fp8_moe_gemm", (counts, counts.shape, _I32), (Y, want, Y.dtype))
    _call("fp8_moe_gemm", stream, ws, (counts, Y) + tx + tw, (qx, counts.data_ptr(), E, qw, Y.data_ptr(), _dt(Y)))


def fp8_moe_linear_fwd(X, counts, w_fwd, Y, ws, stream=None):
    (l_cap, m), E, (q, t) = X.shape, counts.numel(), _q(w_fwd)
    n = w_fwd.rows // (E or 1)
    if counts.dtype is not _I32 or Y.shape != (l_cap, n):
        _refuse_shape("fp8_moe_linear_fwd", (counts, counts.shape, _I32), (Y, (l_cap, n), Y.dtype))
    _call("fp8_moe_linear_fwd", stream, ws, (X, counts, Y) + t,
          (X.data_ptr(), _dt(X), l_cap, counts.data_ptr(), E, m, n, q, Y.data_ptr(), _dt(Y)))


def fp8_moe_linear_dgrad(D, counts, w_dgrad, dX, ws, stream=None):
    (l_cap, n), E, (q, t) = D.shape, counts.numel(), _q(w_dgrad)
    m = w_dgrad.rows // (E or 1)
    if counts.dtype is not _I32 or dX.shape != (l_cap, m):
        _refuse_shape("fp8_moe_linear_dgrad", (counts, counts.shape, _I32), (dX, (l_cap, m), dX.dtype))
    _call("fp8_moe_linear_dgrad", stream, ws, (D, counts, dX) + t,
          (D.data_ptr(), _dt(D), l_cap, counts.data_ptr(), E, m, n, q, dX.data_ptr(), _dt(dX)))


def fp8_moe_linear_wgrad(X, D, counts, dW, ws, stream=None):
    (l_cap, m), (dl, n), E = X.shape, D.shape, counts.numel()
    if dl != l_cap or counts.dtype is not _I32 or dW.shape != (E, m, n):
        _refuse_shape("fp8_moe_linear_wgrad", (D, (l_cap, n), D.dtype), (counts, counts.shape, _I32),
                      (dW, (E, m, n), dW.dtype))
    _call("fp8_moe_linear_wgrad", stream, ws, (X, D, counts, dW),
          (X.data_ptr(), _dt(X), D.data_ptr(), _dt(D), l_cap, counts.data_ptr(), E, m, n, dW.data_ptr(), _dt(dW)))
