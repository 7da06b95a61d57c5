"""Python binding of libgq (include/gq.h): argument marshalling only.

Every function below passes device pointers, sizes and the current CUDA stream
to the C entry point of the same name and raises ``GQError`` on a non-OK
status.  All arithmetic happens in the CUDA kernels of libgq.so; there is no
Python or CPU fallback, and importing this package fails if the library has
not been built (``python bit_gemv_q4_b200/build.py``).

PyTorch is used only to allocate device memory and to name the stream.

`stream` (a torch stream or a raw handle) names the stream of one call, the
current one otherwise; what the call reads has to be ready on it.  The outputs
that a call makes on a named stream are memory of that stream: order later use
on other streams after it (Stream.wait_stream), and record such use
(Tensor.record_stream) if the tensor may be dropped before it has happened.

`workspace="auto"` of the router, the expert layer and the 8-bit product is a
buffer kept for each call, device and stream.  A call that torch.cuda.graph
captures gets one of its own from the graph's memory, and every replay clears it
before the call; with a workspace tensor given (zeroed once, one for calls that
do not overlap) nothing is cleared.  A capture made without torch.cuda.graph
needs outputs and workspaces that the program keeps.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgq.so")

GQ_OK = 0
GQ_F32, GQ_F16, GQ_BF16 = 0, 1, 2
GQ_FMT_Q4_0, GQ_FMT_KSB = 0, 1
GQ_DEV_NONFINITE, GQ_DEV_RANGE, GQ_DEV_TIMEOUT = 1, 2, 4
GQ_GEMV_PDL = 1
GQ_QUANT_REF_RULE = 1
GQ_ROUTE_NORM, GQ_ROUTE_SIGMOID = 2, 4

# every symbol include/gq.h declares
EXPORTS = (
    "gq_abi_version", "gq_status_string", "gq_status_from_dev",
    "gq_q4_0_bytes", "gq_ksb_bytes",
    "gq_quantize_q4_0", "gq_quantize_q4_0_ex", "gq_quantize_ksb",
    "gq_dequantize_q4_0", "gq_dequantize_ksb",
    "gq_gemv_workspace_bytes", "gq_gemv_q4_0", "gq_gemv_ksb",
    "gq_gemv_q4_0_grouped", "gq_gemv_ksb_grouped",
    "gq_gemm_workspace_bytes", "gq_gemm_q4_0", "gq_gemm_ksb",
    "gq_selftest_gemv_timeout", "gq_gemv_q4_0_noalloc", "gq_stream_read",
    "gq_tiled_bytes", "gq_repack_q4_0", "gq_repack_ksb", "gq_gemv_q4_0_tiled", "gq_gemv_ksb_tiled",
    "gq_gemv_q4_0_tiled_grouped", "gq_gemv_ksb_tiled_grouped",
    "gq_moe_route_workspace_bytes", "gq_moe_route",
    "gq_moe_workspace_bytes", "gq_moe_q4_0_tiled", "gq_moe_ksb_tiled", "gq_selftest_moe_timeout",
    "gq_fp8_scales", "gq_quantize_fp8", "gq_dequantize_fp8",
    "gq_gemm_fp8_workspace_bytes", "gq_gemm_fp8", "gq_selftest_gemm_fp8_timeout",
)

_DTYPE_CODE = {torch.float32: GQ_F32, torch.float16: GQ_F16, torch.bfloat16: GQ_BF16}


class GQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gq_status_string(status)} (status {status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libgq.so not found at {LIB_PATH}; build it with `python bit_gemv_q4_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    i64, vp, c_int, c_uint = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_uint
    L.gq_abi_version.restype = c_int
    L.gq_status_string.argtypes = [c_int]
    L.gq_status_string.restype = ctypes.c_char_p
    L.gq_status_from_dev.argtypes = [c_int]
    L.gq_status_from_dev.restype = c_int
    L.gq_q4_0_bytes.argtypes = [i64]
    L.gq_q4_0_bytes.restype = ctypes.c_size_t
    L.gq_ksb_bytes.argtypes = [i64]
    L.gq_ksb_bytes.restype = ctypes.c_size_t
    for name in ("gq_quantize_q4_0", "gq_quantize_ksb"):
        f = getattr(L, name)
        f.argtypes = [vp, i64, vp, vp, vp]
        f.restype = c_int
    L.gq_quantize_q4_0_ex.argtypes = [vp, i64, vp, ctypes.c_uint, vp, vp]
    L.gq_quantize_q4_0_ex.restype = c_int
    for name in ("gq_dequantize_q4_0", "gq_dequantize_ksb"):
        f = getattr(L, name)
        f.argtypes = [vp, i64, vp, vp]
        f.restype = c_int
    L.gq_gemv_workspace_bytes.argtypes = [c_int, i64, i64, i64, c_int]
    L.gq_gemv_workspace_bytes.restype = ctypes.c_size_t
    for name in ("gq_gemv_q4_0", "gq_gemv_ksb"):
        f = getattr(L, name)
        f.argtypes = [vp, i64, i64, vp, c_int, i64, vp, c_int, vp, ctypes.c_size_t, c_uint, vp,
                      vp]
        f.restype = c_int
    for name in ("gq_gemv_q4_0_grouped", "gq_gemv_ksb_grouped"):
        f = getattr(L, name)
        f.argtypes = [vp, c_int, i64, vp, c_int, i64, c_int, c_uint, vp, vp]
        f.restype = c_int
    L.gq_gemm_workspace_bytes.argtypes = [c_int, i64, i64, i64]
    L.gq_gemm_workspace_bytes.restype = ctypes.c_size_t
    for name in ("gq_gemm_q4_0", "gq_gemm_ksb"):
        f = getattr(L, name)
        f.argtypes = [vp, i64, i64, vp, c_int, i64, vp, c_int, vp, ctypes.c_size_t, vp, vp]
        f.restype = c_int
    L.gq_gemv_q4_0_noalloc.argtypes = [vp, i64, i64, vp, vp, c_int, c_uint, vp, vp]
    L.gq_gemv_q4_0_noalloc.restype = c_int
    L.gq_selftest_gemv_timeout.argtypes = [vp, i64, i64, vp, vp, vp, vp]
    L.gq_selftest_gemv_timeout.restype = c_int
    L.gq_stream_read.argtypes = [vp, ctypes.c_size_t, vp, vp]
    L.gq_stream_read.restype = c_int
    L.gq_tiled_bytes.argtypes = [c_int, i64, i64]
    L.gq_tiled_bytes.restype = ctypes.c_size_t
    for name in ("gq_repack_q4_0", "gq_repack_ksb"):
        f = getattr(L, name)
        f.argtypes = [vp, i64, i64, vp, vp]
        f.restype = c_int
    for name in ("gq_gemv_q4_0_tiled", "gq_gemv_ksb_tiled"):
        f = getattr(L, name)
        f.argtypes = [vp, i64, i64, vp, c_int, vp, c_int, c_uint, vp, vp]
        f.restype = c_int
    for name in ("gq_gemv_q4_0_tiled_grouped", "gq_gemv_ksb_tiled_grouped"):
        f = getattr(L, name)
        f.argtypes = [vp, c_int, i64, vp, c_int, c_int, c_uint, vp, vp]
        f.restype = c_int
    L.gq_moe_route_workspace_bytes.argtypes = [i64, i64]
    L.gq_moe_route_workspace_bytes.restype = ctypes.c_size_t
    L.gq_moe_route.argtypes = [vp, c_int, i64, i64, vp, c_int, i64, vp, i64, ctypes.c_float, vp, vp,
                               vp, ctypes.c_size_t, c_uint, vp, vp]
    L.gq_moe_route.restype = c_int
    L.gq_moe_workspace_bytes.argtypes = [c_int, i64, i64, i64, i64]
    L.gq_moe_workspace_bytes.restype = ctypes.c_size_t
    for name in ("gq_moe_q4_0_tiled", "gq_moe_ksb_tiled"):
        f = getattr(L, name)
        f.argtypes = [vp, vp, vp, i64, i64, i64, vp, c_int, i64, vp, vp, i64, vp, c_int, vp,
                      ctypes.c_size_t, c_uint, vp, vp]
        f.restype = c_int
    L.gq_selftest_moe_timeout.argtypes = [vp, vp, vp, i64, i64, i64, vp, i64, vp, vp, i64, vp, vp,
                                          ctypes.c_size_t, vp, vp]
    L.gq_selftest_moe_timeout.restype = c_int
    L.gq_fp8_scales.argtypes = [i64, i64, i64]
    L.gq_fp8_scales.restype = ctypes.c_size_t
    L.gq_quantize_fp8.argtypes = [vp, c_int, i64, i64, i64, vp, vp, vp, vp]
    L.gq_quantize_fp8.restype = c_int
    L.gq_dequantize_fp8.argtypes = [vp, vp, i64, i64, i64, vp, c_int, vp]
    L.gq_dequantize_fp8.restype = c_int
    L.gq_gemm_fp8_workspace_bytes.argtypes = [i64, i64, i64]
    L.gq_gemm_fp8_workspace_bytes.restype = ctypes.c_size_t
    L.gq_gemm_fp8.argtypes = [vp, vp, i64, i64, vp, vp, i64, vp, c_int, vp, ctypes.c_size_t, c_uint, vp,
                              vp]
    L.gq_gemm_fp8.restype = c_int
    L.gq_selftest_gemm_fp8_timeout.argtypes = [vp, vp, i64, i64, vp, vp, i64, vp, vp, ctypes.c_size_t, vp, vp]
    L.gq_selftest_gemm_fp8_timeout.restype = c_int
    return L


lib = _load()


def gq_abi_version() -> int:
    return int(lib.gq_abi_version())


def gq_status_string(status: int) -> str:
    return lib.gq_status_string(int(status)).decode()


def gq_status_from_dev(flags: int) -> int:
    return int(lib.gq_status_from_dev(int(flags)))


def gq_q4_0_bytes(n: int) -> int:
    return int(lib.gq_q4_0_bytes(int(n)))


def gq_ksb_bytes(n: int) -> int:
    return int(lib.gq_ksb_bytes(int(n)))


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_object(stream: int, device: torch.device):
    """A raw handle as a stream that torch allocates and launches on.  (Handles 0 and 1 are the default
    stream; ExternalStream(0) would be some stream of torch's pool.)"""
    if stream in (0, 1):
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(stream, device=device)


def _make(make, shape, dtype, device: torch.device, stream) -> torch.Tensor:
    """torch.empty or torch.zeros of a call's output or workspace, on the call's stream: what the current
    stream has freed it may still be reading, and a workspace has to be clear before the call."""
    if stream is None or device.type != "cuda":
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(_stream(stream), device)):
        return make(shape, dtype=dtype, device=device)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libgq must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libgq must be contiguous")
    return t.data_ptr() or None


def _check(status: int, where: str) -> None:
    if status != GQ_OK:
        raise GQError(status, where)


def _quantize(name: str, nbytes, x: torch.Tensor, out, dev_status, stream):
    if x.dtype != torch.float32:
        raise TypeError("quantizer input must be float32")
    n = x.numel()
    if out is None:
        out = _make(torch.empty, max(nbytes(n), 0), torch.uint8, x.device, stream)
    _check(getattr(lib, name)(_ptr(x), n, _ptr(out), _ptr(dev_status), _stream(stream)), name)
    return out


def gq_quantize_q4_0(x: torch.Tensor, out: torch.Tensor | None = None,
                     dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 values (numel % 32 == 0) -> uint8 Q4_0 blocks (18 bytes per 32)."""
    return _quantize("gq_quantize_q4_0", gq_q4_0_bytes, x, out, dev_status, stream)


def gq_quantize_q4_0_ex(x: torch.Tensor, flags: int, out: torch.Tensor | None = None,
                        dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gq_quantize_q4_0 with a rule flag (0, or GQ_QUANT_REF_RULE for the page's
    reference quantizer: d = signed max / -8, codes min(15, trunc(x/d + 8.5)))."""
    if x.dtype != torch.float32:
        raise TypeError("quantizer input must be float32")
    n = x.numel()
    if out is None:
        out = _make(torch.empty, max(gq_q4_0_bytes(n), 0), torch.uint8, x.device, stream)
    _check(lib.gq_quantize_q4_0_ex(_ptr(x), n, _ptr(out), int(flags), _ptr(dev_status),
                                   _stream(stream)), "gq_quantize_q4_0_ex")
    return out


def gq_quantize_ksb(x: torch.Tensor, out: torch.Tensor | None = None,
                    dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 values (numel % 256 == 0) -> uint8 super-blocks (138 bytes per 256)."""
    return _quantize("gq_quantize_ksb", gq_ksb_bytes, x, out, dev_status, stream)


def _dequantize(name: str, q: torch.Tensor, n: int, out, stream):
    if out is None:
        out = _make(torch.empty, n, torch.float32, q.device, stream)
    _check(getattr(lib, name)(_ptr(q), int(n), _ptr(out), _stream(stream)), name)
    return out


def gq_dequantize_q4_0(q: torch.Tensor, n: int, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    return _dequantize("gq_dequantize_q4_0", q, n, out, stream)


def gq_dequantize_ksb(q: torch.Tensor, n: int, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    return _dequantize("gq_dequantize_ksb", q, n, out, stream)


def gq_gemv_workspace_bytes(fmt: int, M: int, K: int, B: int, x_dtype) -> int:
    code = _DTYPE_CODE[x_dtype] if isinstance(x_dtype, torch.dtype) else int(x_dtype)
    return int(lib.gq_gemv_workspace_bytes(int(fmt), int(M), int(K), int(B), code))


# Zeroed GEMV workspaces, one per (device, stream): calls on one stream run in
# order, and each successful call leaves the workspace ready for the next.
_gemv_ws: dict = {}


def _gemv_workspace(need: int, device: torch.device, stream) -> torch.Tensor:
    key = (device.index, _stream(stream))
    ws = _gemv_ws.get(key)
    if ws is None or ws.numel() < need:
        ws = _make(torch.zeros, need, torch.uint8, device, stream)
        _gemv_ws[key] = ws
    return ws


def _gemv(name: str, fmt: int, W: torch.Tensor, M: int, K: int, x: torch.Tensor, y_dtype, out,
          workspace, flags: int, dev_status, stream):
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    B = x2.shape[0]
    if x2.shape[1] != K:
        raise ValueError(f"x has {x2.shape[1]} columns, expected K={K}")
    if x2.dtype not in _DTYPE_CODE or y_dtype not in _DTYPE_CODE:
        raise TypeError("activations and outputs must be float32, float16 or bfloat16")
    if out is None:
        out = _make(torch.empty, (B, M), y_dtype, x2.device, stream)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        need = gq_gemv_workspace_bytes(fmt, M, K, B, x2.dtype)
        workspace = _gemv_workspace(need, x2.device, stream) if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(getattr(lib, name)(_ptr(W), int(M), int(K), _ptr(x2), _DTYPE_CODE[x2.dtype], B,
                              _ptr(out), _DTYPE_CODE[out.dtype], _ptr(workspace), ws_bytes,
                              int(flags), _ptr(dev_status), _stream(stream)), name)
    return out


def gq_gemv_q4_0(W: torch.Tensor, M: int, K: int, x: torch.Tensor, y_dtype=torch.float16,
                 out: torch.Tensor | None = None, flags: int = 0,
                 dev_status: torch.Tensor | None = None, stream=None,
                 workspace=None) -> torch.Tensor:
    """y[B, M] = W_hat[M, K] @ x[B, K]^T for Q4_0 weights; B in 1..8.

    workspace: None (the default path), "auto" (a zeroed scratch buffer cached
    per device and stream) or a uint8 CUDA tensor of at least
    gq_gemv_workspace_bytes(...) bytes, zero before its first use; with a
    workspace, batch-1 fp16 calls take the integer tensor-core path."""
    return _gemv("gq_gemv_q4_0", GQ_FMT_Q4_0, W, M, K, x, y_dtype, out, workspace, flags,
                 dev_status, stream)


def gq_gemv_ksb(W: torch.Tensor, M: int, K: int, x: torch.Tensor, y_dtype=torch.float16,
                out: torch.Tensor | None = None, flags: int = 0,
                dev_status: torch.Tensor | None = None, stream=None,
                workspace=None) -> torch.Tensor:
    """y[B, M] = W_hat[M, K] @ x[B, K]^T for super-block weights; B in 1..8."""
    return _gemv("gq_gemv_ksb", GQ_FMT_KSB, W, M, K, x, y_dtype, out, workspace, flags,
                 dev_status, stream)


class GemvDesc(ctypes.Structure):
    """gq_gemv_desc: one matrix of a grouped GEMV."""
    _fields_ = [("W", ctypes.c_void_p), ("M", ctypes.c_int64), ("y", ctypes.c_void_p)]


def _gemv_grouped(name: str, Ws, Ms, K: int, x: torch.Tensor, y_dtype, outs, flags: int,
                  dev_status, stream):
    if len(Ws) != len(Ms):
        raise ValueError("one M per matrix")
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    B = x2.shape[0]
    if x2.shape[1] != K:
        raise ValueError(f"x has {x2.shape[1]} columns, expected K={K}")
    if x2.dtype not in _DTYPE_CODE or y_dtype not in _DTYPE_CODE:
        raise TypeError("activations and outputs must be float32, float16 or bfloat16")
    if outs is None:
        outs = [_make(torch.empty, (B, int(M)), y_dtype, x2.device, stream) for M in Ms]
    if len(outs) != len(Ws) or any(o.dtype != outs[0].dtype for o in outs):
        raise ValueError("one output per matrix, all of one dtype")
    descs = (GemvDesc * len(Ws))(*[GemvDesc(_ptr(W), int(M), _ptr(o))
                                   for W, M, o in zip(Ws, Ms, outs)])
    ytype = _DTYPE_CODE[outs[0].dtype] if outs else _DTYPE_CODE[y_dtype]
    _check(getattr(lib, name)(ctypes.cast(descs, ctypes.c_void_p), len(Ws), int(K), _ptr(x2),
                              _DTYPE_CODE[x2.dtype], B, ytype,
                              int(flags), _ptr(dev_status), _stream(stream)), name)
    return outs


def gq_gemv_q4_0_grouped(Ws, Ms, K: int, x: torch.Tensor, y_dtype=torch.float16, outs=None,
                         flags: int = 0, dev_status: torch.Tensor | None = None, stream=None):
    """[y_i = W_hat_i @ x^T for each Q4_0 matrix W_i (M_i x K)], one shared x [B, K]."""
    return _gemv_grouped("gq_gemv_q4_0_grouped", Ws, Ms, K, x, y_dtype, outs, flags,
                         dev_status, stream)


def gq_gemv_ksb_grouped(Ws, Ms, K: int, x: torch.Tensor, y_dtype=torch.float16, outs=None,
                        flags: int = 0, dev_status: torch.Tensor | None = None, stream=None):
    """[y_i = W_hat_i @ x^T for each super-block matrix W_i (M_i x K)], one shared x."""
    return _gemv_grouped("gq_gemv_ksb_grouped", Ws, Ms, K, x, y_dtype, outs, flags,
                         dev_status, stream)


def gq_gemm_workspace_bytes(fmt: int, M: int, K: int, B: int) -> int:
    return int(lib.gq_gemm_workspace_bytes(int(fmt), int(M), int(K), int(B)))


def _gemm(name: str, fmt: int, W: torch.Tensor, M: int, K: int, X: torch.Tensor, y_dtype, out,
          workspace, dev_status, stream):
    X2 = X if X.dim() == 2 else X.reshape(1, -1)
    B = X2.shape[0]
    if X2.shape[1] != K:
        raise ValueError(f"X has {X2.shape[1]} columns, expected K={K}")
    if X2.dtype not in _DTYPE_CODE or y_dtype not in _DTYPE_CODE:
        raise TypeError("X must be bfloat16; Y float32, float16 or bfloat16")
    if out is None:
        out = _make(torch.empty, (B, M), y_dtype, X2.device, stream)
    need = gq_gemm_workspace_bytes(fmt, M, K, B)
    if workspace is None and need > 0:
        workspace = _make(torch.zeros, need, torch.uint8, X2.device, stream)
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(getattr(lib, name)(_ptr(W), int(M), int(K), _ptr(X2), _DTYPE_CODE[X2.dtype], B,
                              _ptr(out), _DTYPE_CODE[out.dtype], _ptr(workspace), ws_bytes,
                              _ptr(dev_status), _stream(stream)), name)
    return out


def gq_gemm_q4_0(W: torch.Tensor, M: int, K: int, X: torch.Tensor, y_dtype=torch.float32,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y[B, M] = W_hat[M, K] @ X[B, K]^T on the tensor cores (X bfloat16, B <= 256)."""
    return _gemm("gq_gemm_q4_0", GQ_FMT_Q4_0, W, M, K, X, y_dtype, out, workspace, dev_status,
                 stream)


def gq_gemm_ksb(W: torch.Tensor, M: int, K: int, X: torch.Tensor, y_dtype=torch.float32,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y[B, M] = W_hat[M, K] @ X[B, K]^T for super-block weights on the tensor cores."""
    return _gemm("gq_gemm_ksb", GQ_FMT_KSB, W, M, K, X, y_dtype, out, workspace, dev_status,
                 stream)


def gq_gemv_q4_0_noalloc(W: torch.Tensor, M: int, K: int, x: torch.Tensor, y_dtype=torch.float16,
                         out: torch.Tensor | None = None, flags: int = 0,
                         dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Batch-1 Q4_0 GEMV (fp16 x) on the library's static scratch."""
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    if x2.shape != (1, K) or x2.dtype != torch.float16:
        raise ValueError("x must be one fp16 vector of length K")
    if out is None:
        out = _make(torch.empty, (1, M), y_dtype, x2.device, stream)
    _check(lib.gq_gemv_q4_0_noalloc(_ptr(W), int(M), int(K), _ptr(x2), _ptr(out),
                                    _DTYPE_CODE[out.dtype], int(flags), _ptr(dev_status),
                                    _stream(stream)), "gq_gemv_q4_0_noalloc")
    return out


def gq_selftest_gemv_timeout(W: torch.Tensor, M: int, K: int, x: torch.Tensor, y: torch.Tensor,
                             dev_status: torch.Tensor, stream=None) -> None:
    """Run the GEMV with a first stage that never fills; the bounded wait must
    report GQ_DEV_TIMEOUT in dev_status (see include/gq.h)."""
    _check(lib.gq_selftest_gemv_timeout(_ptr(W), int(M), int(K), _ptr(x), _ptr(y),
                                        _ptr(dev_status), _stream(stream)),
           "gq_selftest_gemv_timeout")


def gq_stream_read(buf: torch.Tensor, sink: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Read every byte of `buf` once on the GPU and XOR its 32-bit words into
    `sink` (an int32 tensor of one element, zeroed here when not given): the
    practical read ceiling of one launch of that size."""
    if sink is None:
        sink = _make(torch.zeros, 1, torch.int32, buf.device, stream)
    nbytes = buf.numel() * buf.element_size()
    _check(lib.gq_stream_read(_ptr(buf), nbytes, _ptr(sink), _stream(stream)), "gq_stream_read")
    return sink


def gq_tiled_bytes(fmt: int, M: int, K: int) -> int:
    """Bytes of the tiled storage of an M x K matrix (0 for unsupported K)."""
    return int(lib.gq_tiled_bytes(int(fmt), int(M), int(K)))


def gq_repack(fmt: int, W: torch.Tensor, M: int, K: int, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Canonical packed rows (uint8 CUDA tensor) -> tiled storage (uint8)."""
    n = gq_tiled_bytes(fmt, M, K)
    if out is None:
        out = _make(torch.empty, n, torch.uint8, W.device, stream)
    name = "gq_repack_q4_0" if fmt == GQ_FMT_Q4_0 else "gq_repack_ksb"
    _check(getattr(lib, name)(_ptr(W), int(M), int(K), _ptr(out), _stream(stream)), name)
    return out


def _gemv_tiled(name: str, T: torch.Tensor, M: int, K: int, x: torch.Tensor, y_dtype, out,
                flags: int, dev_status, stream):
    x1 = x.reshape(-1)
    if x1.numel() != K:
        raise ValueError(f"x has {x1.numel()} values, expected K={K}")
    if x1.dtype not in _DTYPE_CODE or y_dtype not in _DTYPE_CODE:
        raise TypeError("activations and outputs must be float32, float16 or bfloat16")
    if out is None:
        out = _make(torch.empty, (1, M), y_dtype, x1.device, stream)
    _check(getattr(lib, name)(_ptr(T), int(M), int(K), _ptr(x1), _DTYPE_CODE[x1.dtype],
                              _ptr(out), _DTYPE_CODE[out.dtype], int(flags), _ptr(dev_status),
                              _stream(stream)), name)
    return out


def gq_gemv_q4_0_tiled(T: torch.Tensor, M: int, K: int, x: torch.Tensor, y_dtype=torch.float16,
                       out: torch.Tensor | None = None, flags: int = 0,
                       dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[1, M] = W_hat @ x for Q4_0 weights in tiled storage (x: K fp16 values)."""
    return _gemv_tiled("gq_gemv_q4_0_tiled", T, M, K, x, y_dtype, out, flags, dev_status, stream)


def gq_gemv_ksb_tiled(T: torch.Tensor, M: int, K: int, x: torch.Tensor, y_dtype=torch.float16,
                      out: torch.Tensor | None = None, flags: int = 0,
                      dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[1, M] = W_hat @ x for super-block weights in tiled storage."""
    return _gemv_tiled("gq_gemv_ksb_tiled", T, M, K, x, y_dtype, out, flags, dev_status, stream)


def _gemv_tiled_grouped(name: str, Ts, Ms, K: int, x: torch.Tensor, y_dtype, outs, flags: int,
                        dev_status, stream):
    if len(Ts) != len(Ms):
        raise ValueError("one M per matrix")
    x1 = x.reshape(-1)
    if x1.numel() != K:
        raise ValueError(f"x has {x1.numel()} values, expected K={K}")
    if x1.dtype not in _DTYPE_CODE or y_dtype not in _DTYPE_CODE:
        raise TypeError("activations and outputs must be float32, float16 or bfloat16")
    if outs is None:
        outs = [_make(torch.empty, (1, int(M)), y_dtype, x1.device, stream) for M in Ms]
    if len(outs) != len(Ts) or any(o.dtype != outs[0].dtype for o in outs):
        raise ValueError("one output per matrix, all of one dtype")
    descs = (GemvDesc * len(Ts))(*[GemvDesc(_ptr(T), int(M), _ptr(o))
                                   for T, M, o in zip(Ts, Ms, outs)])
    ytype = _DTYPE_CODE[outs[0].dtype] if outs else _DTYPE_CODE[y_dtype]
    _check(getattr(lib, name)(ctypes.cast(descs, ctypes.c_void_p), len(Ts), int(K), _ptr(x1),
                              _DTYPE_CODE[x1.dtype], ytype, int(flags), _ptr(dev_status),
                              _stream(stream)), name)
    return outs


def gq_gemv_q4_0_tiled_grouped(Ts, Ms, K: int, x: torch.Tensor, y_dtype=torch.float16,
                               outs=None, flags: int = 0, dev_status: torch.Tensor | None = None,
                               stream=None):
    """[y_i = W_hat_i @ x for each Q4_0 matrix in tiled storage T_i (M_i x K)], one fp16 x."""
    return _gemv_tiled_grouped("gq_gemv_q4_0_tiled_grouped", Ts, Ms, K, x, y_dtype, outs, flags,
                               dev_status, stream)


def gq_gemv_ksb_tiled_grouped(Ts, Ms, K: int, x: torch.Tensor, y_dtype=torch.float16,
                              outs=None, flags: int = 0, dev_status: torch.Tensor | None = None,
                              stream=None):
    """[y_i = W_hat_i @ x for each super-block matrix in tiled storage T_i], one fp16 x."""
    return _gemv_tiled_grouped("gq_gemv_ksb_tiled_grouped", Ts, Ms, K, x, y_dtype, outs, flags,
                               dev_status, stream)


# Zeroed workspaces of the calls below, one per (call, device, stream): calls on
# one stream run in order, and each leaves its workspace ready for the next.
_call_ws: dict = {}


def _auto_workspace(name: str, need: int, device: torch.device, stream: int):
    """(tensor, address, bytes) of the call's workspace on `stream`."""
    key = (name, device.index, stream)
    ws = _call_ws.get(key)
    if (ws is not None and ws[2] >= need and stream == torch._C._cuda_getCurrentRawStream(device.index)
            and not torch._C._cuda_isCurrentStreamCapturing()):
        return ws
    # cleared on the call's own stream; a captured call keeps a workspace of its own, which its
    # graph clears
    with torch.cuda.stream(_stream_object(stream, device)):
        capturing = torch._C._cuda_isCurrentStreamCapturing()
        if ws is None or ws[2] < need or capturing:
            t = torch.zeros(need, dtype=torch.uint8, device=device)
            ws = (t, t.data_ptr() or None, need)
            if not capturing:
                _call_ws[key] = ws
    return ws


def _on_device(call):
    """Run the call with its first tensor's device as the current one."""
    name = next(iter(inspect.signature(call).parameters))

    @functools.wraps(call)
    def wrapped(*args, **kw):
        first = args[0] if args else kw.get(name)
        device = -1 if first is None else first.get_device()  # -1: no CUDA tensor, which the call refuses
        if device >= 0 and device != torch._C._cuda_getDevice():
            with torch.cuda.device(device):
                return call(*args, **kw)
        return call(*args, **kw)
    return wrapped


@functools.lru_cache(maxsize=4096)
def _size(name: str, *args) -> int:
    """A size function of the library, its answers kept (they depend on the arguments alone)."""
    return int(getattr(lib, name)(*args))


@functools.lru_cache(maxsize=4096)
def _gemm_fp8_ws(device: int, M: int, K: int, B: int) -> int:
    """gq_gemm_fp8_workspace_bytes on the GPU `device`, the current one; kept for each GPU, since how
    tiles are cut depends on its number of SMs."""
    return int(lib.gq_gemm_fp8_workspace_bytes(M, K, B))


def _where(t: torch.Tensor, stream):
    """Of a call whose tensors are on t's device: (device, raw stream, and that stream again if it is
    not the current one)."""
    d = t.get_device()
    if d < 0:
        raise ValueError("tensors passed to libgq must live on a CUDA device")
    current = torch._C._cuda_getCurrentRawStream(d)
    if stream is None:
        return d, current, None
    s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return d, s, None if s == current else s


def _at(t: torch.Tensor | None, device: int) -> int | None:
    """_ptr of a tensor that has to be on the call's device: one GPU's kernel may not read another's
    memory."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError("tensors of one call must live on one CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libgq must be contiguous")
    return t.data_ptr() or None


def _new(like: torch.Tensor, shape, dtype, named: int | None) -> torch.Tensor:
    """An output of a call, in memory of the stream that it names: what the current stream has freed it
    may still be reading.  (Use on another stream is the caller's to order, and to record before the
    tensor is dropped.)"""
    if named is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(_stream_object(named, like.device)):
        return like.new_empty(shape, dtype=dtype)


def _workspace(name: str, workspace, need: int, device: torch.device, stream: int):
    """(address, bytes, what keeps the memory until the launch)."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto' or a uint8 CUDA tensor")
        if need == 0:
            return None, 0, None
        keep, ptr, size = _auto_workspace(name, need, device, stream)
        return ptr, size, keep
    if workspace is None:
        return None, 0, None
    return _at(workspace, device.index), workspace.numel() * workspace.element_size(), workspace


def gq_moe_route_workspace_bytes(T: int, E: int) -> int:
    return int(lib.gq_moe_route_workspace_bytes(int(T), int(E)))


@_on_device
def gq_moe_route(x: torch.Tensor, Wr: torch.Tensor, k: int, bias: torch.Tensor | None = None,
                 scale: float = 1.0, flags: int = 0, ids: torch.Tensor | None = None,
                 weights: torch.Tensor | None = None, workspace="auto",
                 dev_status: torch.Tensor | None = None, stream=None):
    """(ids [T, k] int32, weights [T, k] fp32): the k experts of each token of x
    [T, H] by their scores x @ Wr^T (Wr [E, H]), and their weights.

    flags: GQ_ROUTE_NORM (weights divided by their sum), GQ_ROUTE_SIGMOID
    (sigmoid scores; `bias` [E] fp32 is added for the choice only), GQ_GEMV_PDL.
    workspace: "auto" (a zeroed buffer cached per device and stream) or a uint8
    CUDA tensor of gq_moe_route_workspace_bytes(T, E) bytes, zero before its
    first use."""
    if x.dim() != 2 or Wr.dim() != 2 or x.shape[1] != Wr.shape[1]:
        raise ValueError("x is [T, H] and Wr [E, H]")
    if x.dtype not in _DTYPE_CODE or Wr.dtype not in _DTYPE_CODE:
        raise TypeError("x and Wr must be float32, float16 or bfloat16")
    T, H = x.shape
    E = Wr.shape[0]
    if bias is not None and (bias.dtype != torch.float32 or bias.numel() != E):
        raise ValueError("bias holds E fp32 values")
    d, s, named = _where(x, stream)
    if ids is None:
        ids = _new(x, (T, k), torch.int32, named)
    elif ids.dtype != torch.int32 or ids.numel() != T * k:
        raise ValueError("ids holds T * k int32 values")
    if weights is None:
        weights = _new(x, (T, k), torch.float32, named)
    elif weights.dtype != torch.float32 or weights.numel() != T * k:
        raise ValueError("weights holds T * k fp32 values")
    ws, ws_bytes, keep = _workspace("route", workspace, _size("gq_moe_route_workspace_bytes", T, E), x.device, s)
    _check(lib.gq_moe_route(_at(x, d), _DTYPE_CODE[x.dtype], T, H, _at(Wr, d), _DTYPE_CODE[Wr.dtype], E,
                            _at(bias, d), k, scale, _at(ids, d), _at(weights, d), ws, ws_bytes, flags,
                            _at(dev_status, d), s), "gq_moe_route")
    return ids, weights


def gq_moe_workspace_bytes(fmt: int, H: int, I: int, T: int, k: int) -> int:
    return int(lib.gq_moe_workspace_bytes(int(fmt), int(H), int(I), int(T), int(k)))


def _moe(name: str, fmt: int, gate, up, down, E: int, I: int, x: torch.Tensor, ids: torch.Tensor,
         weights: torch.Tensor, y_dtype, out, workspace, flags: int, dev_status, stream):
    if x.dim() != 2 or ids.dim() != 2 or ids.shape != weights.shape or ids.shape[0] != x.shape[0]:
        raise ValueError("x is [T, H], ids and weights [T, k]")
    if x.dtype not in _DTYPE_CODE or y_dtype not in _DTYPE_CODE:
        raise TypeError("activations and outputs must be float32, float16 or bfloat16")
    if ids.dtype != torch.int32 or weights.dtype != torch.float32:
        raise TypeError("ids must be int32 and weights fp32")
    T, H = x.shape
    k = ids.shape[1]
    gu, dn = _size("gq_tiled_bytes", fmt, E * I, H), _size("gq_tiled_bytes", fmt, E * H, I)
    if gate.numel() < gu or up.numel() < gu or down.numel() < dn:
        raise ValueError("gate, up or down is smaller than the tiled storage of E experts")
    d, s, named = _where(x, stream)
    if out is None:
        out = _new(x, (T, H), y_dtype, named)
    elif out.dtype not in _DTYPE_CODE or out.numel() != T * H:
        raise ValueError("out holds T * H values")
    ws, ws_bytes, keep = _workspace(name, workspace, _size("gq_moe_workspace_bytes", fmt, H, I, T, k), x.device, s)
    _check(getattr(lib, name)(_at(gate, d), _at(up, d), _at(down, d), E, H, I, _at(x, d), _DTYPE_CODE[x.dtype],
                              T, _at(ids, d), _at(weights, d), k, _at(out, d), _DTYPE_CODE[out.dtype], ws,
                              ws_bytes, flags, _at(dev_status, d), s), name)
    return out


@_on_device
def gq_moe_q4_0_tiled(gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, E: int, I: int,
                      x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                      y_dtype=torch.float16, out: torch.Tensor | None = None, workspace="auto",
                      flags: int = 0, dev_status: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """y [T, H] of a mixture-of-experts layer on Q4_0 experts in tiled storage:
    y[t] = sum_j weights[t, j] * down_e(silu(gate_e x[t]) * (up_e x[t])), e = ids[t, j].

    gate, up: gq_repack of the E * I x H matrix of all experts' rows; down: of
    the E * H x I one.  x: [T, H], T <= 64; ids, weights: [T, k], as
    gq_moe_route returns them.  workspace: "auto" (a zeroed buffer cached per
    device and stream) or a uint8 CUDA tensor of gq_moe_workspace_bytes(...)
    bytes, zero before its first use."""
    return _moe("gq_moe_q4_0_tiled", GQ_FMT_Q4_0, gate, up, down, E, I, x, ids, weights, y_dtype, out,
                workspace, flags, dev_status, stream)


@_on_device
def gq_moe_ksb_tiled(gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, E: int, I: int,
                     x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                     y_dtype=torch.float16, out: torch.Tensor | None = None, workspace="auto",
                     flags: int = 0, dev_status: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """gq_moe_q4_0_tiled on super-block experts."""
    return _moe("gq_moe_ksb_tiled", GQ_FMT_KSB, gate, up, down, E, I, x, ids, weights, y_dtype, out,
                workspace, flags, dev_status, stream)


@_on_device
def gq_selftest_moe_timeout(gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, E: int, I: int,
                            x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, y: torch.Tensor,
                            dev_status: torch.Tensor, workspace="auto", stream=None) -> None:
    """gq_moe_q4_0_tiled on fp16 x and y with a grid barrier that is never passed; the bounded waits
    must report GQ_DEV_TIMEOUT in dev_status (see include/gq.h).  workspace: as for the layer, "auto"
    the same one that gq_moe_q4_0_tiled uses."""
    T, H = x.shape
    k = ids.shape[1]
    if x.dtype != torch.float16 or y.dtype != torch.float16 or y.numel() != T * H:
        raise ValueError("x and y are fp16 [T, H]")
    if ids.dtype != torch.int32 or weights.dtype != torch.float32 or ids.shape != (T, k) or weights.shape != (T, k):
        raise ValueError("ids and weights are [T, k], int32 and fp32")
    gu, dn = _size("gq_tiled_bytes", GQ_FMT_Q4_0, E * I, H), _size("gq_tiled_bytes", GQ_FMT_Q4_0, E * H, I)
    if gate.numel() < gu or up.numel() < gu or down.numel() < dn:
        raise ValueError("gate, up or down is smaller than the tiled storage of E experts")
    d, s, named = _where(x, stream)
    ws, ws_bytes, keep = _workspace("gq_moe_q4_0_tiled", workspace,
                                    _size("gq_moe_workspace_bytes", GQ_FMT_Q4_0, H, I, T, k), x.device, s)
    _check(lib.gq_selftest_moe_timeout(_at(gate, d), _at(up, d), _at(down, d), E, H, I, _at(x, d), T, _at(ids, d),
                                       _at(weights, d), k, _at(y, d), ws, ws_bytes, _at(dev_status, d), s),
           "gq_selftest_moe_timeout")


def gq_fp8_scales(R: int, K: int, rows: int) -> int:
    """Number of scales of an R x K matrix in blocks of rows x 128."""
    return int(lib.gq_fp8_scales(int(R), int(K), int(rows)))


def _check_codes(q: torch.Tensor, what: str) -> None:
    if q.dtype != torch.float8_e4m3fn or q.dim() != 2:
        raise TypeError(f"{what} must be a float8_e4m3fn matrix")


def _check_scales(scales: torch.Tensor, R: int, K: int, rows: int, what: str) -> None:
    # (a matrix of another shape holds scales of other blocks, or has other rows between)
    rb, kb = -(-R // rows), -(-K // 128)
    if scales.dtype != torch.float32 or (scales.shape != (rb, kb)
                                         and (scales.dim() == 2 or scales.numel() != rb * kb)):
        raise ValueError(f"{what} needs one fp32 scale for each block of {rows} x 128 values, [{rb}, {kb}]")


def _fp8_pair(q: torch.Tensor, scales: torch.Tensor, rows: int, what: str):
    _check_codes(q, what)
    R, K = q.shape
    _check_scales(scales, R, K, rows, what)
    return R, K


@_on_device
def gq_quantize_fp8(x: torch.Tensor, rows: int, out: torch.Tensor | None = None,
                    scales: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                    stream=None):
    """(codes [R, K] float8_e4m3fn, scales [ceil(R / rows), ceil(K / 128)] fp32) of x
    [R, K] (fp32, fp16 or bf16; K % 16 == 0) in blocks of rows x 128: rows = 1
    for activations, 128 for weights."""
    if x.dim() != 2:
        raise ValueError("x is [R, K]")
    if x.dtype not in _DTYPE_CODE:
        raise TypeError("x must be float32, float16 or bfloat16")
    if rows not in (1, 128):
        raise ValueError("rows is 1 or 128")
    R, K = x.shape
    if out is not None:
        _check_codes(out, "out")
        if out.shape != x.shape:
            raise ValueError("out has another shape than x")
    if scales is not None:
        _check_scales(scales, R, K, rows, "out")
    d, s, named = _where(x, stream)
    if out is None:
        out = _new(x, (R, K), torch.float8_e4m3fn, named)
    if scales is None:
        scales = _new(x, (-(-R // rows), -(-K // 128)), torch.float32, named)
    _check(lib.gq_quantize_fp8(_at(x, d), _DTYPE_CODE[x.dtype], R, K, rows, _at(out, d), _at(scales, d),
                               _at(dev_status, d), s), "gq_quantize_fp8")
    return out, scales


@_on_device
def gq_dequantize_fp8(q: torch.Tensor, scales: torch.Tensor, rows: int, dtype=torch.float32,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """scale * code of a matrix in blocks of rows x 128, in `dtype`."""
    if rows not in (1, 128):
        raise ValueError("rows is 1 or 128")
    R, K = _fp8_pair(q, scales, rows, "q")
    if dtype not in _DTYPE_CODE:
        raise TypeError("outputs must be float32, float16 or bfloat16")
    d, s, named = _where(q, stream)
    if out is None:
        out = _new(q, (R, K), dtype, named)
    elif out.dtype not in _DTYPE_CODE or out.numel() != R * K:
        raise ValueError("out holds R * K values")
    _check(lib.gq_dequantize_fp8(_at(q, d), _at(scales, d), R, K, rows, _at(out, d), _DTYPE_CODE[out.dtype],
                                 s), "gq_dequantize_fp8")
    return out


def gq_gemm_fp8_workspace_bytes(M: int, K: int, B: int) -> int:
    return int(lib.gq_gemm_fp8_workspace_bytes(int(M), int(K), int(B)))


@_on_device
def gq_gemm_fp8(W: torch.Tensor, w_scales: torch.Tensor, X: torch.Tensor, x_scales: torch.Tensor,
                y_dtype=torch.bfloat16, out: torch.Tensor | None = None, workspace="auto",
                flags: int = 0, dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [B, M] of W [M, K] in 128 x 128 blocks and X [B, K] in 1 x 128 blocks (codes and scales
    as gq_quantize_fp8 returns them).  workspace: "auto" (a buffer cached per device and stream)
    or a uint8 CUDA tensor of gq_gemm_fp8_workspace_bytes(M, K, B) bytes."""
    M, K = _fp8_pair(W, w_scales, 128, "W")
    B, K2 = _fp8_pair(X, x_scales, 1, "X")
    if K != K2:
        raise ValueError(f"X has {K2} columns, expected K={K}")
    if y_dtype not in _DTYPE_CODE:
        raise TypeError("outputs must be float32, float16 or bfloat16")
    d, s, named = _where(W, stream)
    if out is None:
        out = _new(X, (B, M), y_dtype, named)
    elif out.dtype not in _DTYPE_CODE or out.numel() != B * M:
        raise ValueError("out holds B * M values")
    ws, ws_bytes, keep = _workspace("gq_gemm_fp8", workspace, _gemm_fp8_ws(d, M, K, B), W.device, s)
    _check(lib.gq_gemm_fp8(_at(W, d), _at(w_scales, d), M, K, _at(X, d), _at(x_scales, d), B, _at(out, d),
                           _DTYPE_CODE[out.dtype], ws, ws_bytes, flags, _at(dev_status, d), s), "gq_gemm_fp8")
    return out


@_on_device
def gq_selftest_gemm_fp8_timeout(W: torch.Tensor, w_scales: torch.Tensor, X: torch.Tensor,
                                 x_scales: torch.Tensor, Y: torch.Tensor, dev_status: torch.Tensor,
                                 workspace="auto", stream=None) -> None:
    """gq_gemm_fp8 (fp32 Y [B, M]) with a first stage that never fills; the bounded waits must report
    GQ_DEV_TIMEOUT in dev_status (see include/gq.h).  More tokens than the kernel for few takes."""
    M, K = _fp8_pair(W, w_scales, 128, "W")
    B, K2 = _fp8_pair(X, x_scales, 1, "X")
    if K != K2 or Y.dtype != torch.float32 or Y.numel() != B * M:
        raise ValueError("W is [M, K], X [B, K] and Y [B, M] in fp32")
    d, s, named = _where(W, stream)
    ws, ws_bytes, keep = _workspace("gq_gemm_fp8", workspace, _gemm_fp8_ws(d, M, K, B), W.device, s)
    _check(lib.gq_selftest_gemm_fp8_timeout(_at(W, d), _at(w_scales, d), M, K, _at(X, d), _at(x_scales, d), B, _at(Y, d),
                                            ws, ws_bytes, _at(dev_status, d), s), "gq_selftest_gemm_fp8_timeout")
