"""Python binding of libw8a8 (the C ABI in include/w8a8.h).

Argument marshalling only: every step of the W8A8 linear layer runs in the library's
sm_100a kernels.  PyTorch provides device memory and streams.  Tensors must be CUDA,
contiguous, and of the dtype each entry point states; BF16 is the only activation and
weight dtype (a tensor of another dtype is rejected here, before the library is called).
There is no CPU path: without the built library every call raises.
"""
import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw8a8.so")

PATH_INT8, PATH_BF16, PATH_NONE, PATH_FP4 = 0, 1, 2, 3
DEVERR_NONE, DEVERR_TIMEOUT = 0, 1
_STATUS = {0: "ok", 1: "invalid argument", 2: "shape", 3: "not device memory",
           4: "alignment", 5: "workspace", 6: "CUDA error"}


class W8A8Error(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn}: status {code} ({_STATUS.get(code, '?')})")
        self.code = code


class _Weight(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("w_bf16", ctypes.c_void_p),
                ("wq", ctypes.c_void_p), ("ws", ctypes.c_void_p)]


class _FP4Weight(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("format", ctypes.c_int32),
                ("w_bf16", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("factor", ctypes.c_void_p)]


_lib = None
_SIGS = {
    "w8a8_quantize_weight": [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                             ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_quantize_act": [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                          ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_rmsnorm_quantize_act": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                  ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_rmsnorm_mod_quantize_act": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_float,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_linear_prequant_gated": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                   ctypes.c_int64, ctypes.POINTER(_Weight), ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                   ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_linear": [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(_Weight),
                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                    ctypes.POINTER(ctypes.c_int), ctypes.c_void_p],
    "w8a8_linear_host": [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(_Weight),
                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                         ctypes.c_int64, ctypes.POINTER(ctypes.c_int), ctypes.c_void_p],
    "w8a8_linear_noalloc": [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                            ctypes.POINTER(_Weight), ctypes.c_void_p, ctypes.c_void_p,
                            ctypes.POINTER(ctypes.c_int), ctypes.c_void_p],
    "w8a8_linear_prequant": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                             ctypes.POINTER(_Weight), ctypes.c_void_p, ctypes.c_void_p,
                             ctypes.c_void_p],
    "w8a8_bf16_linear": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                         ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p],
    "w8a8_debug_block_sums": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                              ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                              ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_debug_wait_timeout": [ctypes.c_uint64, ctypes.c_void_p],
    "w8a8_rowwise_quantize": [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                              ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_rowwise_linear": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                            ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_fp4_quantize": [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_fp4_dequantize": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                            ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_fp4_linear": [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(_FP4Weight),
                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                        ctypes.POINTER(ctypes.c_int), ctypes.c_void_p],
    "w8a8_fp4_linear_prequant": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                 ctypes.c_int64, ctypes.POINTER(_FP4Weight), ctypes.c_void_p,
                                 ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_block_norm": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                        ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int64,
                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p],
    "w8a8_block_norm_fp4": [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                            ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                            ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int64,
                            ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p],
}


def lib():
    """The loaded library (ctypes.CDLL).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.w8a8_linear_workspace_bytes.argtypes = [ctypes.c_int64] * 3
        L.w8a8_linear_workspace_bytes.restype = ctypes.c_size_t
        L.w8a8_linear_host_workspace_bytes.argtypes = [ctypes.c_int64] * 4
        L.w8a8_linear_host_workspace_bytes.restype = ctypes.c_size_t
        L.w8a8_linear_host_chunk_rows.argtypes = [ctypes.c_int64] * 2
        L.w8a8_linear_host_chunk_rows.restype = ctypes.c_int64
        L.w8a8_fp4_scale_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
        L.w8a8_fp4_scale_bytes.restype = ctypes.c_size_t
        L.w8a8_fp4_linear_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
        L.w8a8_fp4_linear_workspace_bytes.restype = ctypes.c_size_t
        L.w8a8_device_error.argtypes = []
        L.w8a8_device_error.restype = ctypes.c_int
        L.w8a8_last_cuda_error.argtypes = []
        L.w8a8_last_cuda_error.restype = ctypes.c_char_p
        L.w8a8_status_string.argtypes = [ctypes.c_int]
        L.w8a8_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(fn, code):
    if code != 0:
        err = W8A8Error(fn, code)
        if code == 6:
            err.args = (err.args[0] + ": " + lib().w8a8_last_cuda_error().decode(),)
        raise err


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    """The device's current stream as a pointer.  The raw accessor makes no Stream object,
    which costs 2 us of a small call's time."""
    if _raw_stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(torch.cuda.current_device() if device.index is None else device.index)


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t, dtype, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out(t, shape, dtype, device, name):
    """A caller-supplied output buffer: checked here, before the library writes into it,
    for type, dtype, exact shape, device and contiguity (a wrong one would be written out
    of bounds); None -> a new tensor."""
    if t is None:
        return torch.empty(tuple(shape), dtype=dtype, device=device)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != torch.device(device):
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _in(t, shape, dtype, device, name):
    """A required input buffer, checked like an output buffer."""
    if t is None:
        raise TypeError(f"{name} is required")
    return _out(t, shape, dtype, device, name)


def _block_scales(xs, M, K, device, name):
    """A block-scale table [M/128, K/128] float32 on the device."""
    return _out(xs, (M // 128, K // 128), torch.float32, device, name)


def quantize_act(x, xq=None, xs=None):
    """Block-wise 128x128 INT8 quantization of a BF16 [M, K] matrix -> (xq int8 [M, K],
    xs float32 [M/128, K/128])."""
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    xq = _out(xq, (M, K), torch.int8, x.device, "xq")
    xs = _block_scales(xs, M, K, x.device, "xs")
    _check("w8a8_quantize_act", lib().w8a8_quantize_act(_ptr(x), M, K, _ptr(xq), _ptr(xs),
                                                         _stream(x.device)))
    return xq, xs


def quantize_weight(w):
    """Block-wise 128x128 INT8 quantization of a BF16 weight [N, K] -> (wq, ws)."""
    _need(w, torch.bfloat16, "w")
    N, K = w.shape
    wq = torch.empty((N, K), dtype=torch.int8, device=w.device)
    ws = torch.empty((N // 128, K // 128), dtype=torch.float32, device=w.device)
    _check("w8a8_quantize_weight", lib().w8a8_quantize_weight(_ptr(w), N, K, _ptr(wq), _ptr(ws),
                                                               _stream(w.device)))
    return wq, ws


def rowwise_quantize(x, q=None, s=None):
    """Per-row INT8 quantization of a BF16 [rows, K] matrix (TurboT2VA's post-scale
    operator: s = max(||row||_inf, 1e-4) / 127) -> (q int8 [rows, K], s float32 [rows]).
    For a weight [N, K] this gives its per-output-channel codes and scales."""
    _need(x, torch.bfloat16, "x")
    rows, K = x.shape
    q = _out(q, (rows, K), torch.int8, x.device, "q")
    s = _out(s, (rows,), torch.float32, x.device, "s")
    _check("w8a8_rowwise_quantize", lib().w8a8_rowwise_quantize(_ptr(x), rows, K, _ptr(q), _ptr(s),
                                                                 _stream(x.device)))
    return q, s


def rowwise_linear_prequant(xq, xs, wq, ws, bias=None, out=None):
    """y = bf16(float(xq wq^T) * (xs[m] ws[n]) + bias) with INT32 accumulation over all of K."""
    _need(xq, torch.int8, "xq")
    _need(wq, torch.int8, "wq")
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError(f"wq must be [N, {K}], got {tuple(wq.shape)}")
    _in(xs, (M,), torch.float32, xq.device, "xs")
    _in(ws, (N,), torch.float32, xq.device, "ws")
    if bias is not None:
        _out(bias, (N,), torch.bfloat16, xq.device, "bias")
    y = _out(out, (M, N), torch.bfloat16, xq.device, "out")
    _check("w8a8_rowwise_linear", lib().w8a8_rowwise_linear(
        _ptr(xq), _ptr(xs), M, K, _ptr(wq), _ptr(ws), N, _ptr(bias), _ptr(y), _stream(xq.device)))
    return y


def rowwise_linear(x, wq, ws, bias=None, out=None):
    """The per-row operator on BF16 activations: per-row quantization, then the GEMM."""
    xq, xs = rowwise_quantize(x)
    return rowwise_linear_prequant(xq, xs, wq, ws, bias, out)


def rmsnorm_quantize_act(x, gamma, eps=1e-6, xq=None, xs=None, rstd=None):
    """RMSNorm (FP64 row sums, FP32 rstd, bf16((x * rstd) * gamma); gamma may be None)
    fused with the block quantizer (the normalised values are never stored) -> (xq, xs,
    rstd).  From 192 rows per SM the row sums follow the definition's column order, so rstd
    is exactly the definition's; below that a one-grid kernel splits each row over a
    cluster and rstd may differ by one FP32 ulp on rare rows (see include/w8a8.h)."""
    _need(x, torch.bfloat16, "x")
    if gamma is not None:
        _need(gamma, torch.bfloat16, "gamma")
    M, K = x.shape
    dev = x.device
    if gamma is not None:
        _out(gamma, (K,), torch.bfloat16, dev, "gamma")
    xq = _out(xq, (M, K), torch.int8, dev, "xq")
    xs = _block_scales(xs, M, K, dev, "xs")
    rstd = _out(rstd, (M,), torch.float32, dev, "rstd")
    _check("w8a8_rmsnorm_quantize_act",
           lib().w8a8_rmsnorm_quantize_act(_ptr(x), _ptr(gamma), float(eps), M, K, _ptr(xq),
                                           _ptr(xs), _ptr(rstd), _stream(dev)))
    return xq, xs, rstd


def rmsnorm_mod_quantize_act(x, gamma, scale, shift, eps=1e-6, xq=None, xs=None, rstd=None):
    """Modulated RMSNorm fused with the block quantizer: y = bf16(n * (1 + scale[b]) +
    shift[b]) with n = x * rstd (* gamma), b = m // T, T = M // scale.shape[0] rows per
    modulation row (a multiple of 128) -> (xq, xs, rstd)."""
    _need(x, torch.bfloat16, "x")
    if gamma is not None:
        _need(gamma, torch.bfloat16, "gamma")
    _need(scale, torch.bfloat16, "scale")
    _need(shift, torch.bfloat16, "shift")
    M, K = x.shape
    B = scale.shape[0]
    if scale.shape != (B, K) or shift.shape != (B, K) or B == 0 or M % B:
        raise ValueError(f"scale and shift must be [B, {K}] with B dividing M = {M}")
    dev = x.device
    if gamma is not None:
        _out(gamma, (K,), torch.bfloat16, dev, "gamma")
    xq = _out(xq, (M, K), torch.int8, dev, "xq")
    xs = _block_scales(xs, M, K, dev, "xs")
    rstd = _out(rstd, (M,), torch.float32, dev, "rstd")
    _check("w8a8_rmsnorm_mod_quantize_act",
           lib().w8a8_rmsnorm_mod_quantize_act(_ptr(x), _ptr(gamma), _ptr(scale), _ptr(shift),
                                               M // B, float(eps), M, K, _ptr(xq), _ptr(xs),
                                               _ptr(rstd), _stream(dev)))
    return xq, xs, rstd


class W8A8Weight:
    """A linear layer's weight: the retained BF16 copy plus, when N and K are multiples of
    128, its INT8 codes and block scales (quantized once, at construction)."""

    def __init__(self, w_bf16, wq=None, ws=None):
        _need(w_bf16, torch.bfloat16, "w")
        self.w = w_bf16
        self.N, self.K = w_bf16.shape
        if wq is None and self.N % 128 == 0 and self.K % 128 == 0 and self.N and self.K:
            wq, ws = quantize_weight(w_bf16)
        elif wq is not None:
            _in(wq, (self.N, self.K), torch.int8, w_bf16.device, "wq")
            _in(ws, (self.N // 128, self.K // 128), torch.float32, w_bf16.device, "ws")
        self.wq, self.ws = wq, ws
        self._rec = _Weight(self.N, self.K, w_bf16.data_ptr(),
                            0 if wq is None else wq.data_ptr(),
                            0 if ws is None else ws.data_ptr())

    def record(self):
        return ctypes.byref(self._rec)


def _weight_on(weight, K, device):
    """The weight matches the activations' K and lives on their device."""
    if not isinstance(weight, W8A8Weight):
        raise TypeError("weight must be a W8A8Weight")
    if weight.K != K:
        raise ValueError(f"weight has K = {weight.K}, the activations K = {K}")
    if weight.w.device != torch.device(device):
        raise ValueError(f"weight is on {weight.w.device}, the activations on {device}")


def linear_workspace_bytes(M, K, N):
    return int(lib().w8a8_linear_workspace_bytes(M, K, N))


def linear(x, weight, bias=None, out=None, workspace=None, return_path=False):
    """The guarded W8A8 linear: y = x W^T + bias in BF16.  x: [..., K] BF16 (leading
    dimensions flattened to M).  INT8 path when M, K, N are multiples of 128, else BF16."""
    _need(x, torch.bfloat16, "x")
    if bias is not None:
        _need(bias, torch.bfloat16, "bias")
    K = x.shape[-1]
    M = math.prod(x.shape[:-1])
    N = weight.N
    dev = x.device
    _weight_on(weight, K, dev)
    if bias is not None:
        _out(bias, (N,), torch.bfloat16, dev, "bias")
    out = _out(out, (*x.shape[:-1], N), torch.bfloat16, dev, "out")
    need = linear_workspace_bytes(M, K, N)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace is not None:
        _out(workspace, (workspace.numel(),), torch.uint8, dev, "workspace")
    path = ctypes.c_int(-1)
    _check("w8a8_linear", lib().w8a8_linear(
        _ptr(x), M, K, weight.record(), _ptr(bias), _ptr(out), _ptr(workspace),
        0 if workspace is None else workspace.numel(), ctypes.byref(path), _stream(dev)))
    return (out, path.value) if return_path else out


def linear_host_workspace_bytes(M, K, N, chunk_rows=0):
    return int(lib().w8a8_linear_host_workspace_bytes(M, K, N, chunk_rows))


def linear_host(x, weight, bias=None, out=None, workspace=None, chunk_rows=0, return_path=False):
    """w8a8_linear on host buffers: x [..., K] BF16 and the output in CPU memory (pinned
    memory lets the copies overlap with the compute).  The rows stream through the GPU in
    chunks; the result equals linear() on a device copy of x.  The work is enqueued on the
    weight device's current stream, which completes only after the output has landed in
    host memory."""
    if not isinstance(x, torch.Tensor) or x.device.type != "cpu":
        raise ValueError("x must be a CPU tensor (use linear() for device tensors)")
    if x.dtype != torch.bfloat16 or not x.is_contiguous():
        raise TypeError("x must be a contiguous torch.bfloat16 tensor")
    if bias is not None:
        _need(bias, torch.bfloat16, "bias")
    K = x.shape[-1]
    M = math.prod(x.shape[:-1])
    N = weight.N
    dev = weight.w.device
    if weight.K != K:
        raise ValueError(f"weight has K = {weight.K}, the activations K = {K}")
    if bias is not None:
        _out(bias, (N,), torch.bfloat16, dev, "bias")
    if out is None:
        out = torch.empty((*x.shape[:-1], N), dtype=torch.bfloat16, pin_memory=True)
    else:
        _out(out, (*x.shape[:-1], N), torch.bfloat16, "cpu", "out")
    need = linear_host_workspace_bytes(M, K, N, chunk_rows)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace is not None:
        _out(workspace, (workspace.numel(),), torch.uint8, dev, "workspace")
    path = ctypes.c_int(-1)
    _check("w8a8_linear_host", lib().w8a8_linear_host(
        _ptr(x), M, K, weight.record(), _ptr(bias), _ptr(out), _ptr(workspace),
        0 if workspace is None else workspace.numel(), chunk_rows, ctypes.byref(path),
        _stream(dev)))
    return (out, path.value) if return_path else out


NOALLOC_MAX_ELEMS = 16777216


def linear_noalloc(x, weight, bias=None, out=None, return_path=False):
    """w8a8_linear for callers that must not allocate device memory: the quantized
    activations live in scratch built into the library (M * K <= 16 Mi on the INT8 path).
    All calls on a device share that scratch, so calls that may overlap on the GPU must be
    ordered (e.g. issued on one stream)."""
    _need(x, torch.bfloat16, "x")
    if bias is not None:
        _need(bias, torch.bfloat16, "bias")
    K = x.shape[-1]
    M = math.prod(x.shape[:-1])
    dev = x.device
    _weight_on(weight, K, dev)
    if bias is not None:
        _out(bias, (weight.N,), torch.bfloat16, dev, "bias")
    out = _out(out, (*x.shape[:-1], weight.N), torch.bfloat16, dev, "out")
    path = ctypes.c_int(-1)
    _check("w8a8_linear_noalloc", lib().w8a8_linear_noalloc(
        _ptr(x), M, K, weight.record(), _ptr(bias), _ptr(out), ctypes.byref(path), _stream(dev)))
    return (out, path.value) if return_path else out


def linear_prequant(xq, xs, weight, bias=None, out=None):
    """The INT8 block-scaled GEMM on already-quantized activations."""
    _need(xq, torch.int8, "xq")
    M, K = xq.shape
    _in(xs, (M // 128, K // 128), torch.float32, xq.device, "xs")
    _weight_on(weight, K, xq.device)
    if bias is not None:
        _out(bias, (weight.N,), torch.bfloat16, xq.device, "bias")
    out = _out(out, (M, weight.N), torch.bfloat16, xq.device, "out")
    _check("w8a8_linear_prequant", lib().w8a8_linear_prequant(
        _ptr(xq), _ptr(xs), M, K, weight.record(), _ptr(bias), _ptr(out), _stream(xq.device)))
    return out


def linear_prequant_gated(xq, xs, weight, resid, gate, bias=None, out=None):
    """The INT8 block-scaled GEMM with the gated residual update in its epilogue:
    out = bf16(resid + gate[m // T] * (xq wq^T + bias)), T = M // gate.shape[0].  out may
    be resid itself (in-place update); by default a new tensor."""
    _need(xq, torch.int8, "xq")
    _need(resid, torch.bfloat16, "resid")
    _need(gate, torch.bfloat16, "gate")
    M, K = xq.shape
    _in(xs, (M // 128, K // 128), torch.float32, xq.device, "xs")
    _weight_on(weight, K, xq.device)
    B = gate.shape[0]
    if resid.shape != (M, weight.N) or gate.shape != (B, weight.N) or B == 0 or M % B:
        raise ValueError(f"resid must be [{M}, {weight.N}] and gate [B, {weight.N}] with B dividing M")
    if resid.device != xq.device or gate.device != xq.device:
        raise ValueError("resid and gate must be on the device of xq")
    if bias is not None:
        _out(bias, (weight.N,), torch.bfloat16, xq.device, "bias")
    out = _out(out, (M, weight.N), torch.bfloat16, xq.device, "out")
    _check("w8a8_linear_prequant_gated", lib().w8a8_linear_prequant_gated(
        _ptr(xq), _ptr(xs), M, K, weight.record(), _ptr(bias), _ptr(resid), _ptr(gate), M // B,
        _ptr(out), _stream(xq.device)))
    return out


def bf16_linear(x, w, bias=None, out=None):
    """The BF16 GEMM the guard falls back to: y = x w^T + bias, any shape."""
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w")
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K or w.device != x.device:
        raise ValueError(f"w must be [N, {K}] on {x.device}")
    if bias is not None:
        _out(bias, (N,), torch.bfloat16, x.device, "bias")
    out = _out(out, (M, N), torch.bfloat16, x.device, "out")
    _check("w8a8_bf16_linear", lib().w8a8_bf16_linear(_ptr(x), _ptr(w), _ptr(bias), _ptr(out),
                                                       M, K, N, _stream(x.device)))
    return out


# ---- the microscaled 4-bit linear and the norms around a block -----------------------------
FP4_FORMATS = {"mxfp4": 0, "nvfp4": 1}
_FP4_FEW_ROWS = 4        # up to these w8a8_fp4_linear needs no workspace
_FP4_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_FP4_MAX_K = 1 << 24     # longest row of the 4-bit operators


def _fp4_format(format):
    if format not in FP4_FORMATS:
        raise ValueError(f"format must be one of {sorted(FP4_FORMATS)}, got {format!r}")
    return FP4_FORMATS[format]


def _fp4_k(K):
    if K <= 0 or K % 32:
        raise ValueError(f"K must be a positive multiple of 32, got {K}")


def _fp4_tiles(rows, K, format):
    """Shape of a quantized matrix's scales: tiles of 128 rows x 4 blocks, 512 bytes each."""
    return (-(-rows // 128), -(-K // (4 * _FP4_BLOCK[format])), 512)


_Tensor, _BF16, _U8 = torch.Tensor, torch.bfloat16, torch.uint8


def _fits(t, shape, dtype, device):
    """Whether t is what _in accepts, in one expression: the small calls' common case."""
    return (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous())


def _need_bf16(t, name):
    """_need for BF16, in one expression where t is as it should be."""
    if not (type(t) is _Tensor and t.dtype is _BF16 and t.is_cuda and t.is_contiguous()):
        _need(t, _BF16, name)


def _bf16_out(out, like, shape, device):
    """_out for a BF16 output; a new one is made from a tensor at hand, which takes less time."""
    if out is None:
        return like.new_empty(shape, dtype=_BF16)
    return _out(out, shape, _BF16, device, "out")


def _column(t, shape, device, name):
    """An optional BF16 input: checked, as its address (None where there is none)."""
    if t is None:
        return None
    if not _fits(t, shape, _BF16, device):
        _in(t, shape, _BF16, device, name)
    return t.data_ptr()


class FP4Tensor:
    """A matrix [rows, K] in 4-bit floating point: codes uint8 [rows, K/2] (two a byte, the
    even element in the low half), scales uint8 in the tiled layout of include/w8a8.h, and
    for "nvfp4" the rows' float32 factors (None for "mxfp4").  One that the library fills
    keeps all three in one buffer and makes these tensors, views of it, when asked."""

    __slots__ = ("rows", "K", "format", "device", "_ptrs", "_buffer", "_parts")

    def __init__(self, codes, scales, factor, format):
        fmt = _fp4_format(format)
        _need(codes, _U8, "codes")
        rows, half = codes.shape
        dev, tiles = codes.device, _fp4_tiles(rows, 2 * half, format)
        _fp4_k(2 * half)
        self.rows, self.K, self.format, self.device = rows, 2 * half, format, dev
        if not _fits(scales, tiles, _U8, dev):
            _in(scales, tiles, _U8, dev, "scales")
        if fmt:
            if not _fits(factor, (rows,), torch.float32, dev):
                _in(factor, (rows,), torch.float32, dev, "factor")
        elif factor is not None:
            raise ValueError("mxfp4 has no row factors")
        self._buffer, self._parts = None, (codes, scales, factor)
        self._ptrs = (codes.data_ptr(), scales.data_ptr(), factor.data_ptr() if fmt else None)

    # Copies are made from the tensors: the addresses are of those at hand.
    def __copy__(self):
        return FP4Tensor(*self._views(), self.format)

    def __reduce__(self):
        # clones: views of one buffer with two types cannot be saved
        return FP4Tensor, (*(None if t is None else t.clone() for t in self._views()), self.format)

    def _any(self):
        return self._buffer if self._parts is None else self._parts[0]

    def _views(self):
        if self._parts is None:
            rows, half, buf = self.rows, self.K // 2, self._buffer
            base = buf.data_ptr()
            shape = _fp4_tiles(rows, self.K, self.format)
            at = self._ptrs[1] - base
            factor = None
            if self._ptrs[2] is not None:
                f = self._ptrs[2] - base
                factor = buf[f:f + 4 * rows].view(torch.float32)
            self._parts = (buf[:rows * half].view(rows, half), buf[at:at + math.prod(shape)].view(shape), factor)
        return self._parts

    @property
    def codes(self):
        return self._views()[0]

    @property
    def scales(self):
        return self._views()[1]

    @property
    def factor(self):
        return self._views()[2]


def _fp4_empty(rows, K, format, device):
    """A quantized matrix of this size, to be written: codes, scales (from a 256-byte boundary,
    where the TMA reads them fastest) and factors in one allocation."""
    _fp4_k(K)
    q = FP4Tensor.__new__(FP4Tensor)
    q.rows, q.K, q.format, q.device, q._parts = rows, K, format, device, None
    rt, ct, _ = _fp4_tiles(rows, K, format)
    at = (rows * K // 2 + 255) // 256 * 256
    end = at + rt * ct * 512
    nv = format == "nvfp4"
    q._buffer = torch.empty(end + 4 * rows if nv else end, dtype=_U8, device=device)
    base = q._buffer.data_ptr()
    q._ptrs = (base, base + at, base + end if nv else None)
    return q


def _fp4_out(out, rows, K, format, device):
    if out is None:
        return _fp4_empty(rows, K, format, device)
    if not isinstance(out, FP4Tensor):
        raise TypeError("out must be an FP4Tensor")
    if (out.rows, out.K, out.format) != (rows, K, format) or out.device != device:
        raise ValueError(f"out must be [{rows}, {K}] {format} on {device}")
    return out


def fp4_tile_scales(scales):
    """Block scales [rows, blocks] (bytes) -> the tiled layout of FP4Tensor.scales, zeros
    past the end.  For weights quantized elsewhere; plain tensor operations, once at load."""
    if scales.dim() != 2 or scales.element_size() != 1:
        raise ValueError("scales must be a matrix of bytes")
    R, C = scales.shape
    rt, ct = -(-R // 128), -(-C // 4)
    full = torch.zeros((rt * 128, ct * 4), dtype=_U8, device=scales.device)
    full[:R, :C] = scales.contiguous().view(_U8)
    return full.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).reshape(rt, ct, 512).contiguous()


def fp4_untile_scales(tiles, rows, blocks):
    """The inverse of fp4_tile_scales: bytes [rows, blocks]."""
    rt, ct = -(-rows // 128), -(-blocks // 4)
    if tuple(tiles.shape) != (rt, ct, 512):
        raise ValueError(f"tiles must have shape {(rt, ct, 512)}, got {tuple(tiles.shape)}")
    return tiles.view(rt, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)[:rows, :blocks]


def fp4_quantize(x, format="nvfp4", out=None):
    """BF16 [rows, K] -> FP4Tensor, K a multiple of 32.  "mxfp4": blocks of 32 along K with a
    power-of-two scale; "nvfp4": blocks of 16 with an E4M3 scale and a float32 factor per
    row.  A row's codes depend on that row alone."""
    fmt = _fp4_format(format)
    _need_bf16(x, "x")
    rows, K = x.shape
    dev = x.device
    q = _fp4_out(out, rows, K, format, dev)
    _check("w8a8_fp4_quantize",
           (_lib or lib()).w8a8_fp4_quantize(x.data_ptr(), rows, K, fmt, *q._ptrs, _stream(dev)))
    return q


def fp4_dequantize(q, out=None):
    """The values an FP4Tensor's codes stand for, BF16 [rows, K]."""
    if not isinstance(q, FP4Tensor):
        raise TypeError("q must be an FP4Tensor")
    y = _bf16_out(out, q._any(), (q.rows, q.K), q.device)
    _check("w8a8_fp4_dequantize", (_lib or lib()).w8a8_fp4_dequantize(
        *q._ptrs, q.rows, q.K, FP4_FORMATS[q.format], y.data_ptr(), _stream(q.device)))
    return y


class FP4Weight:
    """A linear layer's weight in 4 bits: quantized from w_bf16 at construction, or given as
    an FP4Tensor q.  w_bf16 is kept for the guard's BF16 path (K not a multiple of 32, or above
    2^24, which is not quantized; x not 16-byte aligned); without it those calls raise.
    keep_bf16=False drops it after quantizing."""

    def __init__(self, w_bf16=None, format="nvfp4", q=None, keep_bf16=True):
        if q is not None:
            if not isinstance(q, FP4Tensor):
                raise TypeError("q must be an FP4Tensor")
            self.N, self.K, self.device, format = q.rows, q.K, q.device, q.format
            if w_bf16 is not None:
                _in(w_bf16, (q.rows, q.K), _BF16, q.device, "w")
        else:
            _fp4_format(format)
            _need(w_bf16, _BF16, "w")
            (self.N, self.K), self.device = w_bf16.shape, w_bf16.device
            if self.K and self.K % 32 == 0 and self.K <= _FP4_MAX_K:
                q = fp4_quantize(w_bf16, format)
                if not keep_bf16:
                    w_bf16 = None
        self.w, self.q, self.format = w_bf16, q, format
        self._rec = _FP4Weight(self.N, self.K, FP4_FORMATS[format],
                               None if w_bf16 is None else w_bf16.data_ptr(),
                               *((None, None, None) if q is None else q._ptrs))

    def record(self):
        return ctypes.byref(self._rec)


def _fp4_weight_on(weight, K, device):
    if not isinstance(weight, FP4Weight):
        raise TypeError("weight must be an FP4Weight")
    if weight.K != K:
        raise ValueError(f"weight has K = {weight.K}, the activations K = {K}")
    if weight.device != device:
        raise ValueError(f"weight is on {weight.device}, the activations on {device}")


def fp4_linear_workspace_bytes(M, K, format="nvfp4"):
    return int(lib().w8a8_fp4_linear_workspace_bytes(M, K, _fp4_format(format)))


def fp4_linear(x, weight, bias=None, out=None, workspace=None, return_path=False):
    """y = x W^T + bias in BF16 with x quantized to the weight's 4-bit format in the call.
    x: [..., K] BF16 (leading dimensions flattened), any number of rows and outputs.  K not a
    multiple of 32, or above 2^24, takes the BF16 GEMM on the weight's BF16 copy, and so does
    an x that is not 16-byte aligned."""
    _need_bf16(x, "x")
    K = x.shape[-1]
    M = math.prod(x.shape[:-1])
    dev = x.device
    _fp4_weight_on(weight, K, dev)
    b = _column(bias, (weight.N,), dev, "bias")
    shape = (*x.shape[:-1], weight.N)
    out = _bf16_out(out, x, shape, dev)
    size = 0
    if workspace is None:
        if M > _FP4_FEW_ROWS:
            size = lib().w8a8_fp4_linear_workspace_bytes(M, K, FP4_FORMATS[weight.format])
        if size:
            workspace = torch.empty(size, dtype=_U8, device=dev)
    else:
        size = workspace.numel()
        _out(workspace, (size,), _U8, dev, "workspace")
    path = ctypes.c_int(-1) if return_path else None
    _check("w8a8_fp4_linear", (_lib or lib()).w8a8_fp4_linear(
        x.data_ptr(), M, K, weight._rec, b, out.data_ptr(), workspace.data_ptr() if size else None, size,
        path, _stream(dev)))
    return (out, path.value) if return_path else out


def fp4_linear_prequant(q, weight, bias=None, out=None):
    """The 4-bit GEMM on an FP4Tensor (e.g. from block_norm_fp4) of the weight's format."""
    if not isinstance(q, FP4Tensor):
        raise TypeError("q must be an FP4Tensor")
    _fp4_weight_on(weight, q.K, q.device)
    if weight.format != q.format:
        raise ValueError(f"weight is {weight.format}, the activations {q.format}")
    b = _column(bias, (weight.N,), q.device, "bias")
    out = _bf16_out(out, q._any(), (q.rows, weight.N), q.device)
    _check("w8a8_fp4_linear_prequant", (_lib or lib()).w8a8_fp4_linear_prequant(
        *q._ptrs, q.rows, q.K, weight._rec, b, out.data_ptr(), _stream(q.device)))
    return out


def _block_norm_args(h, y, post_gamma, gate, pre_gamma, scale, shift, post_norm, res_scale, eps, h_out):
    """Checks shared by both forms -> (h_out, the C call's arguments up to K)."""
    _need_bf16(h, "h")
    shape = h.shape
    M, K = shape
    dev = h.device
    if not _fits(y, shape, _BF16, dev):
        _in(y, shape, _BF16, dev, "y")
    if post_gamma is not None and not post_norm:
        raise ValueError("post_gamma needs post_norm")
    rows = gate if gate is not None else scale if scale is not None else shift
    B = 1 if rows is None else rows.shape[0]
    if B == 0 or M % B:
        raise ValueError(f"gate, scale and shift must be [B, {K}] with B dividing M = {M}")
    if h_out is None:
        h_out = torch.empty_like(h)
    else:
        _out(h_out, shape, _BF16, dev, "h_out")
    return h_out, (h.data_ptr(), y.data_ptr(), int(post_norm), _column(post_gamma, (K,), dev, "post_gamma"),
                   _column(gate, (B, K), dev, "gate"), res_scale, _column(pre_gamma, (K,), dev, "pre_gamma"),
                   _column(scale, (B, K), dev, "scale"), _column(shift, (B, K), dev, "shift"), max(M // B, 1),
                   eps, M, K)


def block_norm(h, y, post_gamma=None, gate=None, pre_gamma=None, scale=None, shift=None, *,
               res_scale=1.0, post_norm=True, eps=1e-6, h_out=None, n_out=None):
    """The residual update between two blocks and the next block's norm, in one pass:
    h' = bf16(res_scale * h + gate[b] * u) with u = RMSNorm(y) * post_gamma (u = y without
    post_norm), n = bf16(RMSNorm(h') * pre_gamma * (1 + scale[b]) + shift[b]).  h, y [M, K],
    K a multiple of 8; gammas [K]; gate, scale, shift [B, K] with b = m // (M // B); each may
    be None.  h_out may be h (in place) -> (h', n)."""
    h_out, args = _block_norm_args(h, y, post_gamma, gate, pre_gamma, scale, shift, post_norm, res_scale, eps,
                                   h_out)
    n = torch.empty_like(h) if n_out is None else _out(n_out, h.shape, _BF16, h.device, "n_out")
    _check("w8a8_block_norm",
           (_lib or lib()).w8a8_block_norm(*args, h_out.data_ptr(), n.data_ptr(), _stream(h.device)))
    return h_out, n


def block_norm_fp4(h, y, format="nvfp4", post_gamma=None, gate=None, pre_gamma=None, scale=None,
                   shift=None, *, res_scale=1.0, post_norm=True, eps=1e-6, h_out=None, out=None):
    """block_norm with n quantized as fp4_quantize does, without being stored (the same bits
    as the two calls); K a multiple of 32 -> (h', FP4Tensor)."""
    fmt = _fp4_format(format)
    h_out, args = _block_norm_args(h, y, post_gamma, gate, pre_gamma, scale, shift, post_norm, res_scale, eps,
                                   h_out)
    q = _fp4_out(out, *h.shape, format, h.device)
    _check("w8a8_block_norm_fp4",
           (_lib or lib()).w8a8_block_norm_fp4(*args, fmt, h_out.data_ptr(), *q._ptrs, _stream(h.device)))
    return h_out, q


def debug_block_sums(xq, wq, m0=0, rows=None, n0=0, cols=None):
    """INT32 per-K-block partial products [rows, cols, K/128] of the window rows m0 ..
    m0 + rows - 1, columns n0 .. n0 + cols - 1 (default: everything), from the tensor-core
    main loop."""
    _need(xq, torch.int8, "xq")
    _need(wq, torch.int8, "wq")
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K or wq.device != xq.device:
        raise ValueError(f"wq must be [N, {K}] on {xq.device}")
    rows = M - m0 if rows is None else rows
    cols = N - n0 if cols is None else cols
    out = torch.empty((rows, cols, K // 128), dtype=torch.int32, device=xq.device)
    _check("w8a8_debug_block_sums", lib().w8a8_debug_block_sums(
        _ptr(xq), _ptr(wq), M, K, N, m0, rows, n0, cols, _ptr(out), _stream(xq.device)))
    return out


def debug_wait_timeout(timeout_ns, device=None):
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _check("w8a8_debug_wait_timeout", lib().w8a8_debug_wait_timeout(int(timeout_ns), _stream(dev)))


def device_error():
    """Synchronize and return (and clear) the library's device error word."""
    return int(lib().w8a8_device_error())
