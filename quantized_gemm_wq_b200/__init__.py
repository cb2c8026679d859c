"""Python binding of libwq.so (argument marshalling only).

Every computation happens in the CUDA kernels behind the C ABI declared in
``include/wq.h``; this module only turns torch CUDA tensors into pointers,
allocates outputs with torch (device memory is PyTorch's job here) and raises
``WQError`` on a non-OK status.  There is no fallback: if ``libwq.so`` cannot
be loaded, importing this package fails.

    codes, scales, zeros = wq_quantize_rtn(W_f16, bits, group)
    y = wq_gemm(x_bf16, codes, scales, zeros, bits, group, N, K)
    ys = wq_gemm_grouped([(x, codes, scales, zeros, N, K, group), ...], bits, workspace)

8-bit integers on both sides (one scale per token, one per output channel):

    q, qs = wq_quantize_i8(x)                       # tokens, or rows of weights
    y = wq_gemm_i8(q, qs, w, ws)
    h = wq_gated_i8(q, qs, w_gate, gate_scales, w_up, up_scales, act="silu")
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwq.so")

# Status codes of include/wq.h
WQ_OK = 0
WQ_ERR_NULL = 1
WQ_ERR_BITS = 2
WQ_ERR_GROUP = 3
WQ_ERR_SHAPE = 4
WQ_ERR_ALIGN = 5
WQ_ERR_UNSUPPORTED_DEVICE = 6
WQ_ERR_CUDA = 7
WQ_ERR_DEVICE_TIMEOUT = 8
WQ_ERR_WORKSPACE = 9
WQ_ERR_TYPE = 10
WQ_ERR_STRIDE = 11

# Functions the header declares (the tests check the library exports them).
EXPORTED = ("wq_quantize_rtn", "wq_quantize_rtn_sym", "wq_gemm", "wq_gemm_grouped", "wq_gemm_grouped_workspace_size",
            "wq_gemm_grouped_noalloc", "wq_quantize_i8", "wq_gemm_i8", "wq_gated_i8",
            "wq_codes_words", "wq_params_count", "wq_status_string", "wq_last_device_error")


class Linear(ctypes.Structure):
    """``wq_linear`` of include/wq.h: one linear of a grouped call."""
    _fields_ = [("x_bf16", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("scales_f16", ctypes.c_void_p), ("zeros_f16", ctypes.c_void_p),
                ("y_bf16", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("group", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libwq.so not built ({LIB_PATH}); run __graft_entry__.build() "
                          "or python quantized_gemm_wq_b200/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.wq_quantize_rtn.argtypes = [vp, i64, i64, ci, i64, vp, vp, vp, vp]
    lib.wq_quantize_rtn.restype = ci
    lib.wq_quantize_rtn_sym.argtypes = [vp, i64, i64, ci, i64, vp, vp, vp]
    lib.wq_quantize_rtn_sym.restype = ci
    lib.wq_gemm.argtypes = [vp, i64, i64, i64, vp, vp, vp, ci, i64, vp, vp]
    lib.wq_gemm.restype = ci
    lp = ctypes.POINTER(Linear)
    lib.wq_gemm_grouped.argtypes = [lp, ci, i64, ci, vp, ctypes.c_size_t, vp]
    lib.wq_gemm_grouped.restype = ci
    lib.wq_gemm_grouped_noalloc.argtypes = [lp, ci, i64, ci, vp]
    lib.wq_gemm_grouped_noalloc.restype = ci
    lib.wq_gemm_grouped_workspace_size.argtypes = [lp, ci, i64, ci]
    lib.wq_gemm_grouped_workspace_size.restype = ctypes.c_size_t
    lib.wq_quantize_i8.argtypes = [vp, ci, i64, i64, i64, vp, i64, vp, vp]
    lib.wq_quantize_i8.restype = ci
    lib.wq_gemm_i8.argtypes = [vp, i64, vp, i64, i64, i64, vp, i64, vp, vp, ci, i64, vp]
    lib.wq_gemm_i8.restype = ci
    lib.wq_gated_i8.argtypes = [vp, i64, vp, i64, i64, i64, vp, vp, vp, vp, i64, ci, vp, ci, i64, vp]
    lib.wq_gated_i8.restype = ci
    lib.wq_codes_words.argtypes = [i64, i64, ci]
    lib.wq_codes_words.restype = ctypes.c_size_t
    lib.wq_params_count.argtypes = [i64, i64, i64]
    lib.wq_params_count.restype = ctypes.c_size_t
    lib.wq_status_string.argtypes = [ci]
    lib.wq_status_string.restype = ctypes.c_char_p
    lib.wq_last_device_error.argtypes = []
    lib.wq_last_device_error.restype = ci
    return lib


lib = _load()


class WQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib.wq_status_string(status).decode()} (status {status})")


def _check(status: int, where: str) -> None:
    if status != WQ_OK:
        raise WQError(status, where)


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def wq_codes_words(N: int, K: int, bits: int) -> int:
    return int(lib.wq_codes_words(N, K, bits))


def wq_params_count(N: int, K: int, group: int) -> int:
    return int(lib.wq_params_count(N, K, group))


def wq_status_string(status: int) -> str:
    return lib.wq_status_string(status).decode()


def wq_last_device_error() -> int:
    return int(lib.wq_last_device_error())


def groups_per_row(K: int, group: int) -> int:
    return 1 if group in (0, K) else K // group


def wq_quantize_rtn(W: torch.Tensor, bits: int, group: int, codes=None, scales=None,
                    zeros=None, stream=None):
    """Quantise fp16 ``W`` [N, K] (CUDA) -> (codes uint32 [N, K*bits/32] as
    int32 storage, scales fp16 [N, G], zeros fp16 [N, G])."""
    if W.dtype != torch.float16 or W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous CUDA fp16 [N, K] tensor")
    N, K = W.shape
    G = groups_per_row(K, group) if group in (0, K) or (group > 0 and K % group == 0) else 1
    if codes is None:
        codes = torch.empty((N, max(1, K * bits // 32)), dtype=torch.int32, device=W.device)
    if scales is None:
        scales = torch.empty((N, G), dtype=torch.float16, device=W.device)
    if zeros is None:
        zeros = torch.empty((N, G), dtype=torch.float16, device=W.device)
    st = lib.wq_quantize_rtn(_ptr(W), N, K, bits, group, _ptr(codes), _ptr(scales), _ptr(zeros),
                             _stream_ptr(stream))
    _check(st, "wq_quantize_rtn")
    return codes, scales, zeros


def wq_quantize_rtn_sym(W: torch.Tensor, bits: int, group: int, codes=None, scales=None, stream=None):
    """Quantise fp16 ``W`` [N, K] (CUDA) on the symmetric grid (zero 2^(bits-1),
    not stored) -> (codes, scales, None); pass the None as ``zeros``."""
    if W.dtype != torch.float16 or W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous CUDA fp16 [N, K] tensor")
    N, K = W.shape
    G = groups_per_row(K, group) if group in (0, K) or (group > 0 and K % group == 0) else 1
    if codes is None:
        codes = torch.empty((N, max(1, K * bits // 32)), dtype=torch.int32, device=W.device)
    if scales is None:
        scales = torch.empty((N, G), dtype=torch.float16, device=W.device)
    st = lib.wq_quantize_rtn_sym(_ptr(W), N, K, bits, group, _ptr(codes), _ptr(scales), _stream_ptr(stream))
    _check(st, "wq_quantize_rtn_sym")
    return codes, scales, None


def wq_gemm(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, zeros,
            bits: int, group: int, N: int, K: int, y=None, stream=None) -> torch.Tensor:
    """``y = x . W'^T`` for bf16 ``x`` [M, K] (CUDA) -> bf16 ``y`` [M, N];
    ``zeros`` None for codes of the symmetric grid."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA bf16 [M, K] tensor")
    M = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("x.shape[1] must equal K")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    st = lib.wq_gemm(_ptr(x), M, N, K, _ptr(codes), _ptr(scales), _ptr(zeros), bits, group,
                     _ptr(y), _stream_ptr(stream))
    _check(st, "wq_gemm")
    return y


def _linear_array(items, M):
    """ctypes array of ``wq_linear`` from (x, codes, scales, zeros, N, K, group, y)
    tuples; allocates the missing outputs."""
    arr = (Linear * len(items))()
    ys = []
    for i, it in enumerate(items):
        x, codes, scales, zeros, N, K, group = it[:7]
        y = it[7] if len(it) > 7 and it[7] is not None else None
        if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
            raise ValueError("every x must be a contiguous CUDA bf16 [M, K] tensor")
        if x.shape[0] != M or x.shape[1] != K:
            raise ValueError("every x must be [M, K] with the call's M")
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        arr[i] = Linear(_ptr(x), _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(y), N, K, group)
        ys.append(y)
    return arr, ys


def grouped_workspace_size(items, bits: int) -> int:
    """Workspace bytes ``wq_gemm_grouped`` needs for these linears."""
    if not items:
        return 0
    M = items[0][0].shape[0]
    arr, _ = _linear_array([it[:7] for it in items], M) if items[0][0].is_cuda else (None, None)
    if arr is None:
        raise ValueError("x must be a CUDA tensor")
    return int(lib.wq_gemm_grouped_workspace_size(arr, len(items), M, bits))


def grouped_workspace(items, bits: int, device=None) -> torch.Tensor:
    """A zero-filled device workspace for ``wq_gemm_grouped`` on these linears
    (uint8, at least 16 bytes so it always has an address)."""
    n = grouped_workspace_size(items, bits)
    dev = device if device is not None else items[0][0].device
    return torch.zeros(max(16, n), dtype=torch.uint8, device=dev)


def wq_gemm_grouped(items, bits: int, workspace=None, stream=None):
    """``y_l = x_l . W'_l^T`` for every (x, codes, scales, zeros, N, K, group[, y])
    of ``items`` (common M and bits) -> list of bf16 ``y_l``.  ``workspace``: a
    zero-filled uint8 CUDA tensor from ``grouped_workspace`` (made here when
    None; reuse one across calls on the same stream)."""
    if not items:
        return []
    M = items[0][0].shape[0]
    arr, ys = _linear_array(items, M)
    if workspace is None:
        workspace = grouped_workspace(items, bits)
    st = lib.wq_gemm_grouped(arr, len(items), M, bits, _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check(st, "wq_gemm_grouped")
    return ys


def wq_gemm_grouped_noalloc(items, bits: int, stream=None):
    """``wq_gemm_grouped`` on the library's built-in 8 MiB workspace, for
    callers that cannot allocate device memory when they call.  Every item
    must carry its output ``y`` (x, codes, scales, zeros, N, K, group, y):
    nothing is allocated here either."""
    if not items:
        return []
    if any(len(it) < 8 or it[7] is None for it in items):
        raise ValueError("wq_gemm_grouped_noalloc allocates nothing: pass every y")
    M = items[0][0].shape[0]
    arr, ys = _linear_array(items, M)
    st = lib.wq_gemm_grouped_noalloc(arr, len(items), M, bits, _stream_ptr(stream))
    _check(st, "wq_gemm_grouped_noalloc")
    return ys


# ---- 8-bit integers on both sides -------------------------------------------

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}      # wq_type
_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}                        # wq_act


# The three calls below are made once per layer and token, so what they do on
# the host is kept short: one test of everything a good call has, and only where
# it fails the tests that say what is wrong; device indexes instead of device
# objects; the current stream's address without a Stream object (3 us by itself).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device
_empty_strided = torch.empty_strided
_INT8, _FP32 = torch.int8, torch.float32
_lib_quantize_i8, _lib_gemm_i8, _lib_gated_i8 = lib.wq_quantize_i8, lib.wq_gemm_i8, lib.wq_gated_i8


def _need_matrix(t: torch.Tensor, what: str, dtypes=(_INT8,), dev=None) -> None:
    if t.dtype not in dtypes:
        raise ValueError(f"{what} must be of type " + " or ".join(str(d) for d in dtypes))
    if t.dim() != 2 or not t.is_cuda or (dev is not None and t.get_device() != dev):
        raise ValueError(f"{what} must be a 2-D CUDA tensor, all operands on one device")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have adjacent columns (stride 1)")


def _need_scales(t: torch.Tensor, n: int, dev: int, what: str) -> None:
    if t.dtype is not _FP32 or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous fp32 [{n}] tensor on the codes' device")


def _pad16(n: int) -> int:
    # for the stride of a single row, which is never taken: any valid one will do
    return (n + 15) // 16 * 16


def _elsewhere(call, dev: int, stream, *args):
    """call(*args) with `dev` current and, if one is given, on `stream` (so that what
    the call allocates is the stream's too)."""
    if stream is not None and stream.device.index != dev:
        raise ValueError("stream must be one of the operands' device")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return call(*args)


def _output(y, M: int, N: int, dtype, x):
    """The given output's row stride and wq_type; or a new one on x's device, and its."""
    if y is None:
        yt = _TYPES.get(dtype)
        if yt is None:
            raise ValueError("dtype must be torch.bfloat16, torch.float16 or torch.float32")
        return _empty_strided((M, N), (N, 1), dtype=dtype, device=x.device), N, yt
    _need_matrix(y, "the output", tuple(_TYPES), x.get_device())
    if y.shape != (M, N):
        raise ValueError(f"the output must be [{M}, {N}]")
    return y, y.stride(0) if M > 1 else N, _TYPES[y.dtype]


def wq_quantize_i8(x: torch.Tensor, codes=None, scales=None, stream=None):
    """Quantise every row of bf16/fp16/fp32 ``x`` [R, K] (CUDA, any row stride from K on)
    -> (int8 codes [R, K], fp32 scales [R]), ``x ~ codes * scales[:, None]``;
    a row's scale is max|x| times fp32(1/127).
    The codes' rows start at multiples of 32 bytes, so for other K they do not
    lie side by side."""
    xt, dev = _TYPES.get(x.dtype), x.get_device()
    if xt is None or dev < 0 or x.dim() != 2:
        _need_matrix(x, "x", tuple(_TYPES))
    if stream is not None or dev != _current_device():
        return _elsewhere(wq_quantize_i8, dev, stream, x, codes, scales)
    R, K = x.shape
    ldx, step = x.stride()
    if step != 1:
        _need_matrix(x, "x", tuple(_TYPES))
    if codes is None:
        # rows on 32 bytes, L2's sectors: the tensor-core kernels take a quarter
        # longer where they are on 16 (2048 x 5120 -> 5120: 48 against 38 us)
        ldc = (K + 31) // 32 * 32
        codes = _empty_strided((R, K), (ldc, 1), dtype=_INT8, device=x.device)
    else:
        _need_matrix(codes, "codes", dev=dev)
        if codes.shape != x.shape:
            raise ValueError("codes must have x's shape")
        ldc = codes.stride(0) if R > 1 else _pad16(K)
    if scales is None:
        scales = _empty_strided((R,), (1,), dtype=_FP32, device=x.device)
    else:
        _need_scales(scales, R, dev, "scales")
    st = _lib_quantize_i8(x.data_ptr(), xt, R, K, ldx if R > 1 else K, codes.data_ptr(), ldc, scales.data_ptr(),
                          _raw_stream(dev))
    if st != WQ_OK:
        raise WQError(st, "wq_quantize_i8")
    return codes, scales


def wq_gemm_i8(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, y=None,
               dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """``y[m, n] = x_scales[m] * w_scales[n] * sum_k x[m, k] w[n, k]`` for int8
    codes ``x`` [M, K] and ``w`` [N, K] -> ``y`` [M, N] of ``dtype`` (or the
    given ``y``'s type).  Row strides of codes are multiples of 16."""
    dev = x.get_device()
    if x.dim() != 2 or w.dim() != 2 or dev < 0:
        raise ValueError("x and w must be 2-D CUDA tensors")
    if stream is not None or dev != _current_device():
        return _elsewhere(wq_gemm_i8, dev, stream, x, x_scales, w, w_scales, y, dtype)
    M, K = x.shape
    N, Kw = w.shape
    ldx, xstep = x.stride()
    ldw, wstep = w.stride()
    if not (x.dtype is _INT8 and w.dtype is _INT8 and K == Kw and xstep == 1 and wstep == 1
            and w.get_device() == dev and x_scales.dtype is _FP32 and w_scales.dtype is _FP32
            and x_scales.shape == (M,) and w_scales.shape == (N,) and x_scales.get_device() == dev
            and w_scales.get_device() == dev and x_scales.is_contiguous() and w_scales.is_contiguous()):
        _need_matrix(x, "x")
        _need_matrix(w, "w", dev=dev)
        if Kw != K:
            raise ValueError("w must be [N, K] with x's K")
        _need_scales(x_scales, M, dev, "x_scales")
        _need_scales(w_scales, N, dev, "w_scales")
    y, ldy, yt = _output(y, M, N, dtype, x)
    st = _lib_gemm_i8(x.data_ptr(), ldx if M > 1 else _pad16(K), x_scales.data_ptr(), M, N, K, w.data_ptr(),
                      ldw if N > 1 else _pad16(K), w_scales.data_ptr(), y.data_ptr(), yt, ldy, _raw_stream(dev))
    if st != WQ_OK:
        raise WQError(st, "wq_gemm_i8")
    return y


def wq_gated_i8(x: torch.Tensor, x_scales: torch.Tensor, w_gate: torch.Tensor, gate_scales: torch.Tensor,
                w_up: torch.Tensor, up_scales: torch.Tensor, act: str = "silu", h=None, dtype=torch.bfloat16,
                stream=None) -> torch.Tensor:
    """``h = act(x . w_gate^T) * (x . w_up^T)`` on int8 codes, both products
    scaled as in ``wq_gemm_i8``, in one kernel; ``act``: "silu", "gelu" (erf)
    or "gelu_tanh"."""
    at = _ACTS.get(act)
    if at is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    dev = x.get_device()
    if x.dim() != 2 or w_gate.dim() != 2 or w_up.dim() != 2 or dev < 0:
        raise ValueError("x, w_gate and w_up must be 2-D CUDA tensors")
    if stream is not None or dev != _current_device():
        return _elsewhere(wq_gated_i8, dev, stream, x, x_scales, w_gate, gate_scales, w_up, up_scales, act, h, dtype)
    M, K = x.shape
    N, Kw = w_gate.shape
    ldx, xstep = x.stride()
    strides = ldw, wstep = w_gate.stride()
    if not (x.dtype is _INT8 and w_gate.dtype is _INT8 and w_up.dtype is _INT8 and K == Kw and xstep == 1
            and wstep == 1 and w_up.shape == w_gate.shape and w_up.stride() == strides
            and w_gate.get_device() == dev and w_up.get_device() == dev and x_scales.dtype is _FP32
            and gate_scales.dtype is _FP32 and up_scales.dtype is _FP32 and x_scales.shape == (M,)
            and gate_scales.shape == (N,) and up_scales.shape == (N,) and x_scales.get_device() == dev
            and gate_scales.get_device() == dev and up_scales.get_device() == dev and x_scales.is_contiguous()
            and gate_scales.is_contiguous() and up_scales.is_contiguous()):
        _need_matrix(x, "x")
        _need_matrix(w_gate, "w_gate", dev=dev)
        _need_matrix(w_up, "w_up", dev=dev)
        if Kw != K or w_up.shape != w_gate.shape or (N > 1 and w_up.stride(0) != ldw):
            raise ValueError("w_gate and w_up must be [N, K] with x's K and one row stride")
        _need_scales(x_scales, M, dev, "x_scales")
        _need_scales(gate_scales, N, dev, "gate_scales")
        _need_scales(up_scales, N, dev, "up_scales")
    h, ldh, ht = _output(h, M, N, dtype, x)
    st = _lib_gated_i8(x.data_ptr(), ldx if M > 1 else _pad16(K), x_scales.data_ptr(), M, N, K, w_gate.data_ptr(),
                       gate_scales.data_ptr(), w_up.data_ptr(), up_scales.data_ptr(), ldw if N > 1 else _pad16(K),
                       at, h.data_ptr(), ht, ldh, _raw_stream(dev))
    if st != WQ_OK:
        raise WQError(st, "wq_gated_i8")
    return h
