"""Python binding of the w4a16 CUDA library (include/w4a16.h).

Argument marshalling only: every entry point checks tensor dtypes, shapes,
devices and contiguity, then calls the C ABI of ``_lib/libw4a16.so`` with raw
device pointers and the current CUDA stream: through ctypes, or, for the
operators of a decode step (``kv4_*``, ``w4a16_qk_norm_rope``,
``w4a16_sample``), through the small host extension ``_lib/_marshal.so``.  All
arithmetic happens in the library's CUDA kernels; there is no fallback of any
kind.  If the library (or for those operators the extension) has not been
built, importing this package succeeds but every call raises ``RuntimeError``
(build it with ``__graft_entry__.build()``).

Tensors: packed codes are ``torch.uint8``; scales and zero points
``torch.float16``; activations and outputs ``torch.bfloat16``.
"""
from __future__ import annotations

import collections
import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

__all__ = [
    "w4a16_gemv", "w4a16_gemm", "w4a16_gemm_f16", "fp4_moe_gemv", "fp4_moe_gemm", "fp4_moe_gemm_scratch_bytes",
    "w4a16_dequant", "w4a16_bf16_gemm",
    "w4a16_check_device_error", "w4a16_last_error_string", "w4a16_version",
    "w4a16_debug_inject", "INJECT_STALL_PIPELINE", "INJECT_STALL_CONSUMERS",
    "w4a16_linear", "w4a16_linear_array", "w4a16_linear_sequence", "w4a16_graph_create", "w4a16_graph_launch",
    "w4a16_linear_chain", "w4a16_linear_chain_scratch_bytes", "chain_scratch", "w4a16_linear_chain_noalloc",
    "w4a16_graph_destroy", "W4A16Graph",
    "kv4_plan", "kv4_plan_buffers", "KV4Plan", "w4a16_qk_norm_rope", "kv4_append", "kv4_gather", "kv4_cache",
    "kv4_attention", "kv4_attention_scratch", "kv4_attention_scratch_bytes",
    "kv4_prefix_attention", "kv4_prefix_attention_scratch", "kv4_prefix_attention_scratch_bytes",
    "kv4_bounds", "kv4_bounds_buffer", "kv4_select", "kv4_sparse_attention", "w4a16_sample",
    "library_path", "W4A16Error", "STATUS", "FMT_INT4", "FMT_FP4",
    "OUT_F32", "OUT_BF16",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libw4a16.so")
_MARSHAL_PATH = os.path.join(_HERE, "_lib", "_marshal.so")
_lock = threading.Lock()
_lib = None
_fast = None  # the host extension: checks a call's tensors and makes it

STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "MISALIGNED",
          4: "CUDA", 5: "TIMEOUT", 6: "DEVICE"}
FMT_INT4, FMT_FP4 = 0, 1
OUT_F32, OUT_BF16 = 0, 1

# Exported symbols and their ctypes signatures (mirrors include/w4a16.h).
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int


class w4a16_linear(ctypes.Structure):
    """One INT4 linear of a sequence (mirrors the C struct)."""
    _fields_ = [("x", ctypes.c_void_p), ("qw", ctypes.c_void_p), ("s", ctypes.c_void_p),
                ("z", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


_OPS = ctypes.POINTER(w4a16_linear)
_F = ctypes.c_float
SIGNATURES = {
    "w4a16_gemv": ([_P, _P, _P, _P, _P, _I64, _I64, _INT, _P], _INT),
    "w4a16_gemm": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _INT, _P], _INT),
    "w4a16_gemm_f16": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _INT, _P], _INT),
    "w4a16_bf16_gemm": ([_P, _P, _P, _I64, _I64, _I64, _P], _INT),
    "w4a16_copy": ([_P, _P, _I64, _P], _INT),
    "fp4_moe_gemv": ([_P, _P, _P, _P, _INT, _P, _I64, _I64, _I64, _INT, _P], _INT),
    "fp4_moe_gemm": ([_P, _P, _P, _P, _INT, _INT, _P, _I64, _I64, _I64, _INT, _P, _I64, _P], _INT),
    "fp4_moe_gemm_scratch_bytes": ([_INT, _INT, _I64, _I64], _I64),
    "w4a16_dequant": ([_INT, _P, _P, _P, _P, _INT, _I64, _I64, _INT, _P], _INT),
    "w4a16_linear_sequence": ([_OPS, _INT, _INT, _P], _INT),
    "w4a16_linear_chain": ([_OPS, _INT, _INT, _P, _I64, _P], _INT),
    "w4a16_linear_chain_scratch_bytes": ([_INT], _I64),
    "w4a16_linear_chain_noalloc": ([_OPS, _INT, _INT, _P], _INT),
    "w4a16_graph_create": ([_OPS, _INT, _INT, ctypes.POINTER(ctypes.c_void_p)], _INT),
    "w4a16_graph_launch": ([_P, _P], _INT),
    "w4a16_graph_destroy": ([_P], _INT),
    "kv4_plan": ([_P, _P, _INT, _P, _I64, _P, _I64, _INT, _I64, _P, _P, _P, _P, _P, _P], _INT),
    "w4a16_qk_norm_rope": ([_P, _I64, _P, _I64, _P, _P, _P, _I64, _INT, _P, _P, _P, _I64, _INT, _INT, _INT, _F, _F,
                            _INT, _P], _INT),
    "kv4_append": ([_P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _I64, _INT, _P, _P, _P, _P, _I64, _INT, _I64, _INT,
                    _INT, _INT, _F, _F, _INT, _P], _INT),
    "kv4_gather": ([_P, _I64, _INT, _P, _P, _P, _I64, _INT, _INT, _P], _INT),
    "kv4_attention_scratch_bytes": ([_INT, _INT, _INT], _I64),
    "kv4_attention": ([_P, _I64, _P, _I64, _INT, _P, _I64, _P, _P, _INT, _P, _I64, _INT, _INT, _INT, _F, _I64, _I64,
                       _I64, _P, _I64, _P], _INT),
    "kv4_prefix_attention_scratch_bytes": ([_I64, _INT, _INT, _INT, _INT, _INT], _I64),
    "kv4_prefix_attention": ([_P, _I64, _P, _I64, _INT, _P, _I64, _P, _P, _INT, _P, _P, _INT, _P, _I64, _INT, _INT, _INT,
                              _F, _I64, _I64, _P, _I64, _P], _INT),
    "kv4_bounds": ([_P, _I64, _INT, _P, _P, _I64, _INT, _INT, _P], _INT),
    "kv4_select": ([_P, _I64, _P, _I64, _INT, _P, _I64, _P, _P, _INT, _I64, _INT, _INT, _INT, _INT, _INT, _INT, _P, _P,
                    _P], _INT),
    "kv4_sparse_attention": ([_P, _I64, _P, _I64, _INT, _P, _I64, _P, _P, _I64, _INT, _INT, _INT, _F, _P, _I64, _P], _INT),
    "w4a16_sample": ([_P, _INT, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P], _INT),
    "w4a16_check_device_error": ([_P], _INT),
    "w4a16_debug_inject": ([ctypes.c_uint], _INT),
    "w4a16_last_error_string": ([], ctypes.c_char_p),
    "w4a16_version": ([], _INT),
}


class W4A16Error(RuntimeError):
    """A nonzero status returned by the library."""

    def __init__(self, status: int, message: str):
        super().__init__("%s (%d): %s" % (STATUS.get(status, "?"), status, message))
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    "libw4a16.so is not built (%s); run __graft_entry__.build()" % _LIB_PATH)
            handle = ctypes.CDLL(_LIB_PATH)
            for name, (argtypes, restype) in SIGNATURES.items():
                fn = getattr(handle, name)
                fn.argtypes = argtypes
                fn.restype = restype
            _lib = handle
        return _lib


def _check(status: int):
    if status != 0:
        msg = lib().w4a16_last_error_string().decode(errors="replace")
        raise W4A16Error(status, msg)


# The current stream's handle without building a Stream object (2.3 us less a
# call on the host); None where this torch has no such function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None):
    """The stream handle to pass: the given stream, else the current stream
    of `device` (of the current device when None)."""
    if stream is None:
        index = device.index if isinstance(device, torch.device) else device
        if _raw_stream is not None and type(index) is int:
            return ctypes.c_void_p(_raw_stream(index))
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _need(t: torch.Tensor, name: str, dtype, numel=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if numel is not None and t.numel() != numel:
        raise ValueError("%s has %d elements, expected %d" % (name, t.numel(), numel))
    return ctypes.c_void_p(t.data_ptr())


def w4a16_gemv(x, qw, s, z, y=None, group: int = 128, stream=None):
    """y[N] = x[K] W^T with INT4 weights qw [N, K/2], s/z [N, K/group];
    z=None: symmetric INT4 (zero point 8)."""
    N = qw.shape[0]
    K = 2 * qw.shape[-1]
    dev = qw.device
    px = _need(x, "x", torch.bfloat16, K, dev)
    pq = _need(qw, "qw", torch.uint8, N * K // 2, dev)
    ps = _need(s, "s", torch.float16, N * (K // group), dev)
    pz = _need(z, "z", torch.float16, N * (K // group), dev) if z is not None else None
    if y is None:
        y = torch.empty(N, dtype=torch.bfloat16, device=dev)
    py = _need(y, "y", torch.bfloat16, N, dev)
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().w4a16_gemv(px, pq, ps, pz, py, N, K, group, _stream(stream, dev)))
    return y


def w4a16_gemm(X, qw, s, z, Y=None, group: int = 128, stream=None):
    """Y[M, N] = X[M, K] W^T with INT4 weights qw [N, K/2], s/z [N, K/group];
    z=None: symmetric INT4 (zero point 8)."""
    return _gemm("w4a16_gemm", X, qw, s, z, Y, group, stream)


def w4a16_gemm_f16(X, qw, s, z, Y=None, group: int = 128, stream=None):
    """w4a16_gemm with binary16 operands (each weight rounded once to
    binary16; see the header for the error bound)."""
    return _gemm("w4a16_gemm_f16", X, qw, s, z, Y, group, stream)


def _gemm(name, X, qw, s, z, Y, group, stream):
    N = qw.shape[0]
    K = 2 * qw.shape[-1]
    M = X.numel() // K
    dev = qw.device
    pX = _need(X, "X", torch.bfloat16, M * K, dev)
    pq = _need(qw, "qw", torch.uint8, N * K // 2, dev)
    ps = _need(s, "s", torch.float16, N * (K // group), dev)
    pz = _need(z, "z", torch.float16, N * (K // group), dev) if z is not None else None
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    pY = _need(Y, "Y", torch.bfloat16, M * N, dev)
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(getattr(lib(), name)(pX, pq, ps, pz, pY, M, N, K, group, _stream(stream, dev)))
    return Y


def w4a16_bf16_gemm(X, W, Y=None, stream=None):
    """Y[M, N] = X[M, K] W[N, K]^T, dense BF16 (the unfused path's GEMM)."""
    N, K = W.shape[0], W.shape[-1]
    M = X.numel() // K
    dev = W.device
    pX = _need(X, "X", torch.bfloat16, M * K, dev)
    pW = _need(W, "W", torch.bfloat16, N * K, dev)
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    pY = _need(Y, "Y", torch.bfloat16, M * N, dev)
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().w4a16_bf16_gemm(pX, pW, pY, M, N, K, _stream(stream, dev)))
    return Y


def fp4_moe_gemv(x, qw, s, expert_ids, y=None, group: int = 32, stream=None):
    """y[topk, N]: row i = x W_{expert_ids[i]}^T, FP4 stack qw [E, N, K/2]."""
    E, N = qw.shape[0], qw.shape[1]
    K = 2 * qw.shape[2]
    topk = expert_ids.numel()
    dev = qw.device
    px = _need(x, "x", torch.bfloat16, K, dev)
    pq = _need(qw, "qw", torch.uint8, E * N * K // 2, dev)
    ps = _need(s, "s", torch.float16, E * N * (K // group), dev)
    pi = _need(expert_ids, "expert_ids", torch.int32, topk, dev)
    if y is None:
        y = torch.empty(topk, N, dtype=torch.bfloat16, device=dev)
    py = _need(y, "y", torch.bfloat16, topk * N, dev)
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().fp4_moe_gemv(px, pq, ps, pi, topk, py, E, N, K, group, _stream(stream, dev)))
    return y


def fp4_moe_gemm_scratch_bytes(M: int, topk: int, E: int, K: int) -> int:
    """Bytes of scratch memory fp4_moe_gemm needs for M tokens x topk."""
    return int(lib().fp4_moe_gemm_scratch_bytes(int(M), int(topk), int(E), int(K)))


def fp4_moe_gemm(X, qw, s, expert_ids, Y=None, scratch=None, group: int = 32, stream=None):
    """Y[M, topk, N]: Y[m, j] = X[m] W_{expert_ids[m, j]}^T for the FP4 stack
    qw [E, N, K/2].  `scratch`: a device tensor of at least
    fp4_moe_gemm_scratch_bytes(M, topk, E, K) bytes (allocated per call when
    None)."""
    E, N = qw.shape[0], qw.shape[1]
    K = 2 * qw.shape[2]
    M = X.numel() // K if K else 0
    topk = expert_ids.numel() // M if M else 0
    dev = qw.device
    pX = _need(X, "X", torch.bfloat16, M * K, dev)
    pq = _need(qw, "qw", torch.uint8, E * N * K // 2, dev)
    ps = _need(s, "s", torch.float16, E * N * (K // group), dev)
    pi = _need(expert_ids, "expert_ids", torch.int32, M * topk, dev)
    if Y is None:
        Y = torch.empty(M, topk, N, dtype=torch.bfloat16, device=dev)
    pY = _need(Y, "Y", torch.bfloat16, M * topk * N, dev)
    need = fp4_moe_gemm_scratch_bytes(M, topk, E, K)
    if scratch is None:
        scratch = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if not isinstance(scratch, torch.Tensor) or scratch.device != dev or not scratch.is_contiguous():
        raise ValueError("scratch must be a contiguous CUDA tensor on %s" % dev)
    nbytes = scratch.numel() * scratch.element_size()
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().fp4_moe_gemm(pX, pq, ps, pi, M, topk, pY, E, N, K, group,
                                  ctypes.c_void_p(scratch.data_ptr()), nbytes, _stream(stream, dev)))
    return Y


def w4a16_dequant(fmt: int, qw, s, z=None, out=None, out_dtype: int = OUT_F32,
                  group=None, stream=None):
    """Dequantised weights [rows, K] (float32 or bfloat16) -- debug entry."""
    K = 2 * qw.shape[-1]
    rows = qw.numel() // (K // 2)
    if group is None:
        group = 128 if fmt == FMT_INT4 else 32
    dev = qw.device
    pq = _need(qw, "qw", torch.uint8, rows * K // 2, dev)
    ps = _need(s, "s", torch.float16, rows * (K // group), dev)
    pz = _need(z, "z", torch.float16, rows * (K // group), dev) if z is not None else None
    odt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty(rows, K, dtype=odt, device=dev)
    po = _need(out, "out", odt, rows * K, dev)
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().w4a16_dequant(fmt, pq, ps, pz, po, out_dtype, rows, K, group, _stream(stream, dev)))
    return out


def w4a16_linear_array(ops, group: int = 128):
    """ctypes array of w4a16_linear from (X, qw, s, z, Y) tuples (z may be
    None), each checked as w4a16_gemm checks its tensors.  The array holds
    raw addresses only: the caller keeps the tensors alive while it is used."""
    arr = (w4a16_linear * max(1, len(ops)))()
    for i, (X, qw, s, z, Y) in enumerate(ops):
        N = qw.shape[0]
        K = 2 * qw.shape[-1]
        M = X.numel() // K
        dev = qw.device
        who = "op %d " % i
        arr[i].x = _need(X, who + "x", torch.bfloat16, M * K, dev)
        arr[i].qw = _need(qw, who + "qw", torch.uint8, N * K // 2, dev)
        arr[i].s = _need(s, who + "s", torch.float16, N * (K // group), dev)
        arr[i].z = _need(z, who + "z", torch.float16, N * (K // group), dev) if z is not None else None
        arr[i].y = _need(Y, who + "y", torch.bfloat16, M * N, dev)
        arr[i].M, arr[i].N, arr[i].K = M, N, K
    return arr


def w4a16_linear_sequence(ops, group: int = 128, stream=None, count=None):
    """Launch the INT4 linears `ops` = [(X, qw, s, z, Y), ...] in order on
    one stream (each op's X is read after the previous op has finished).
    `ops` may also be an array from w4a16_linear_array, with `count` ops."""
    if isinstance(ops, ctypes.Array):
        if ops._type_ is not w4a16_linear:
            raise TypeError("ops must be an array of w4a16_linear")
        arr, n = ops, len(ops) if count is None else int(count)
        if not 0 <= n <= len(ops):
            raise ValueError("count %d outside 0..%d (the array's length)" % (n, len(ops)))
        dev = torch.cuda.current_device()  # raw addresses: the caller's current device
    else:
        arr, n = w4a16_linear_array(ops, group), len(ops)
        dev = ops[0][1].device if ops else torch.cuda.current_device()
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().w4a16_linear_sequence(arr, n, group, _stream(stream, dev)))


def w4a16_linear_chain_scratch_bytes(count: int) -> int:
    """Bytes of scratch memory w4a16_linear_chain needs for `count` ops."""
    return int(lib().w4a16_linear_chain_scratch_bytes(int(count)))


def chain_scratch(count: int, device=None) -> torch.Tensor:
    """A zeroed scratch buffer (int32) for chains of up to `count` ops."""
    n = (w4a16_linear_chain_scratch_bytes(count) + 3) // 4
    return torch.zeros(max(n, 1), dtype=torch.int32, device=device if device is not None else "cuda")


def w4a16_linear_chain(ops, scratch, group: int = 128, stream=None, count=None):
    """The M = 1 INT4 linears `ops` = [(x, qw, s, z, y), ...] (or an array
    from w4a16_linear_array with `count` ops) in one persistent launch,
    computing what w4a16_linear_sequence computes.  `scratch`: a zeroed
    device tensor of at least w4a16_linear_chain_scratch_bytes(count)
    bytes (see chain_scratch), left zeroed by every call."""
    if isinstance(ops, ctypes.Array):
        if ops._type_ is not w4a16_linear:
            raise TypeError("ops must be an array of w4a16_linear")
        arr, n = ops, len(ops) if count is None else int(count)
        if not 0 <= n <= len(ops):
            raise ValueError("count %d outside 0..%d (the array's length)" % (n, len(ops)))
        dev = scratch.device
    else:
        arr, n = w4a16_linear_array(ops, group), len(ops)
        dev = ops[0][1].device if ops else scratch.device
    if not isinstance(scratch, torch.Tensor) or not scratch.is_cuda or scratch.device != dev:
        raise ValueError("scratch must be a CUDA tensor on %s" % dev)
    if not scratch.is_contiguous():
        raise ValueError("scratch must be contiguous")
    nbytes = scratch.numel() * scratch.element_size()
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().w4a16_linear_chain(arr, n, group, ctypes.c_void_p(scratch.data_ptr()), nbytes,
                                        _stream(stream, dev)))


def w4a16_linear_chain_noalloc(ops, group: int = 128, stream=None, count=None):
    """w4a16_linear_chain with the library's built-in counters instead of
    caller scratch: nothing is allocated (for callers that may not allocate
    device memory).  At most 4032 linears; calls that can overlap on the GPU
    race on the shared counters, so keep them on one stream."""
    if isinstance(ops, ctypes.Array):
        if ops._type_ is not w4a16_linear:
            raise TypeError("ops must be an array of w4a16_linear")
        arr, n = ops, len(ops) if count is None else int(count)
        if not 0 <= n <= len(ops):
            raise ValueError("count %d outside 0..%d (the array's length)" % (n, len(ops)))
        dev = torch.cuda.current_device()
    else:
        arr, n = w4a16_linear_array(ops, group), len(ops)
        dev = ops[0][1].device if ops else torch.cuda.current_device()
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().w4a16_linear_chain_noalloc(arr, n, group, _stream(stream, dev)))


class W4A16Graph:
    """Handle of a captured linear sequence (w4a16_graph_create).  Keeps the
    tensors of its ops alive: the graph holds their addresses."""

    def __init__(self, handle, tensors, device):
        self._h = handle
        self._tensors = tensors
        self.device = device

    def launch(self, stream=None):
        w4a16_graph_launch(self, stream)

    def destroy(self):
        if self._h is not None:
            h, self._h = self._h, None
            _check(lib().w4a16_graph_destroy(h))
            self._tensors = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def w4a16_graph_create(ops, group: int = 128) -> W4A16Graph:
    """Capture the linear sequence `ops` once into a CUDA graph on the
    current device; replay it with w4a16_graph_launch."""
    arr = w4a16_linear_array(ops, group)
    h = ctypes.c_void_p()
    dev = ops[0][1].device if ops else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):  # the graph is captured on the current device
        _check(lib().w4a16_graph_create(arr, len(ops), group, ctypes.byref(h)))
    return W4A16Graph(h, [t for op in ops for t in op if t is not None], dev)


def w4a16_graph_launch(graph: W4A16Graph, stream=None) -> None:
    """Enqueue one replay of a captured sequence on the stream."""
    if graph._h is None:
        raise ValueError("graph has been destroyed")
    with torch.cuda.device(graph.device):
        _check(lib().w4a16_graph_launch(graph._h, _stream(stream, graph.device)))


def w4a16_graph_destroy(graph: W4A16Graph) -> None:
    graph.destroy()


def w4a16_copy(dst: torch.Tensor, src: torch.Tensor, stream=None, device=None) -> torch.Tensor:
    """dst <- src (the same number of bytes, both contiguous) by one kernel on
    `device` (the CUDA tensor's device; `device` when both are host
    tensors): a CUDA tensor or a pinned host tensor on either side."""
    for name, t in (("dst", dst), ("src", src)):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        if not t.is_cuda and t.numel() > 0 and not t.is_pinned():
            raise ValueError("%s: a host tensor must be pinned" % name)
    nbytes = dst.numel() * dst.element_size()
    if src.numel() * src.element_size() != nbytes:
        raise ValueError("dst has %d bytes, src %d" % (nbytes, src.numel() * src.element_size()))
    devs = {t.device for t in (dst, src) if t.is_cuda}
    if len(devs) > 1:
        raise ValueError("dst and src are on different devices")
    dev = devs.pop() if devs else torch.device(device if device is not None else "cuda")
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().w4a16_copy(ctypes.c_void_p(dst.data_ptr()), ctypes.c_void_p(src.data_ptr()), nbytes,
                                _stream(stream, dev)))
    return dst


# --------------------------------------------- the step around the linears

def _ptr(t, name, dtype, device, numel=None):
    """Address of an optional contiguous tensor (None: a null pointer)."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device.index and t.is_contiguous() and
            (numel is None or t.numel() == numel)):
        return t.data_ptr()
    # what is wrong with it
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if numel is not None and t.numel() != numel:
        raise ValueError("%s has %d elements, expected %d" % (name, t.numel(), numel))
    return t.data_ptr()


def _rows(t, name, device):
    """Address and token stride of [T, heads, D] bfloat16 rows: heads and
    elements contiguous, tokens any stride (a slice of a fused row)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s must be torch.bfloat16, got %s" % (name, t.dtype))
    if t.get_device() != (-1 if device.index is None else device.index):
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    shape = t.shape
    if len(shape) != 3:
        raise ValueError("%s must be [tokens, heads, D]" % name)
    T, H, D = shape
    a, b, c = t.stride()
    if (c != 1 and D > 1) or (b != D and H > 1):
        raise ValueError("%s: heads and elements must be contiguous" % name)
    return t.data_ptr(), (a if T > 1 else H * D)


_TYPES = {"b": torch.uint8, "h": torch.bfloat16, "i": torch.int32, "l": torch.int64, "f": torch.float32}


# The functions below make their call through the host extension.  Where that
# finds an argument amiss (it returns None) they go through the same checks
# here, to say what it is.

def _extension():
    """The loaded host extension (raises if it has not been built, or was built
    for another torch)."""
    global _fast
    if _fast is None:
        lib()
        with _lock:
            if _fast is None:
                loader = importlib.machinery.ExtensionFileLoader("_marshal", _MARSHAL_PATH)
                spec = importlib.util.spec_from_file_location("_marshal", _MARSHAL_PATH, loader=loader)
                try:
                    module = importlib.util.module_from_spec(spec)
                    loader.exec_module(module)
                    module.bind(_LIB_PATH)
                except (ImportError, RuntimeError) as e:
                    raise RuntimeError("the host extension %s cannot be loaded (%s); run __graft_entry__.build()" %
                                       (_MARSHAL_PATH, e)) from e
                _fast = module
    return _fast


def _handle(stream):
    """The stream argument of the extension: None or a handle."""
    return stream if stream is None else stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _checked(device, spec, names, *tensors):
    """Addresses of a call's tensors, given as tensor, count, tensor, count
    ... with a letter of `spec` each (r: rows, else the type)."""
    out = []
    for c, name, t, n in zip(spec, names, tensors[0::2], tensors[1::2]):
        if c == "r":
            out += _rows(t, name, device) if t is not None else (None, 0)
        else:
            out.append(_ptr(t, name, _TYPES[c], device, n if n >= 0 else None))
    if device.type != "cuda":
        raise ValueError("expected CUDA tensors, got %s" % device)
    return out


def _launch(device, stream, fn, *args):
    """Calls the library with `device` current (which it usually is)."""
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(device.index)
    else:
        handle = _stream(stream, device)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status != 0:
        _check(status)


KV4Plan = collections.namedtuple("KV4Plan", "seq_lens cu_new positions slots taken")
_PLAN_NAMES = ("ctx_lens", "new_lens", "block_table", "free_blocks", "seq_lens", "cu_new", "positions", "slots", "taken")


def kv4_plan_buffers(requests: int, num_tokens: int, device=None) -> KV4Plan:
    """Buffers for kv4_plan: `requests` requests, room for `num_tokens` new
    tokens in a step."""
    dev = torch.device(device if device is not None else "cuda")
    i32 = dict(dtype=torch.int32, device=dev)
    return KV4Plan(torch.empty(requests, **i32), torch.empty(requests + 1, **i32), torch.empty(num_tokens, **i32),
                   torch.empty(num_tokens, dtype=torch.int64, device=dev), torch.empty(1, **i32))


def kv4_plan(ctx_lens, new_lens, block_table, free_blocks, block_size: int, num_tokens=None, out=None, stream=None):
    """Block tables and slot maps of a step: `ctx_lens` tokens held and
    `new_lens` added by each request; `block_table` [requests, max_blocks]
    gets the new blocks, from the front of `free_blocks`, written in.  Returns
    KV4Plan(seq_lens, cu_new, positions, slots, taken), in `out` if given,
    else new with room for `num_tokens` tokens."""
    dev = ctx_lens.device
    B = ctx_lens.numel()
    if out is None:
        if num_tokens is None:
            raise ValueError("kv4_plan needs num_tokens or out")
        out = kv4_plan_buffers(B, num_tokens, dev)
    seq, cu, pos, slots, taken = out
    r = _extension().kv4_plan(ctx_lens, new_lens, block_table, free_blocks, block_size, seq, cu, pos, slots, taken,
                              _handle(stream))
    if r == 0:
        return out
    if r is not None:
        _check(r)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [%d, max_blocks]" % B)
    T = pos.numel()
    a = _checked(dev, "iiiiiiili", _PLAN_NAMES, ctx_lens, B, new_lens, B, block_table, -1, free_blocks, -1, seq, B, cu,
                 B + 1, pos, T, slots, T, taken, 1)
    _launch(dev, stream, lib().kv4_plan, a[0], a[1], B, a[2], block_table.shape[1], a[3], free_blocks.numel(), block_size,
            T, a[4], a[5], a[6], a[7], a[8])
    return out


_ROPE_NAMES = ("q", "k", "q_weight", "k_weight", "cos_sin", "positions", "q_out", "k_out")


def _table(cos_sin, positions):
    """Rows and width of a cos_sin table (0, 0: no rotation)."""
    if cos_sin is None:
        return 0, 0
    if positions is None:
        raise ValueError("cos_sin needs positions")
    rows, rot = cos_sin.shape
    return rows, rot


def w4a16_qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, q_out=None, k_out=None, eps: float = 1e-6,
                       weight_offset: float = 0.0, interleaved: bool = False, stream=None):
    """RMS norm and position rotation of every head of q [T, Hq, D] and
    k [T, Hkv, D] (tokens may be strided) in one pass; weights [D] or None (no
    norm), cos_sin float32 [positions, rot] or None (no rotation).  Returns
    (q_out, k_out)."""
    dev = q.device
    T, Hq, D = q.shape
    Tk, Hk, Dk = k.shape
    if Tk != T or Dk != D:
        raise ValueError("k must be [%d, heads, %d]" % (T, D))
    rows, rot = _table(cos_sin, positions)
    if q_out is None:
        q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    if k_out is None:
        k_out = torch.empty(T, Hk, D, dtype=torch.bfloat16, device=dev)
    r = _extension().w4a16_qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out, float(eps),
                                        float(weight_offset), interleaved, _handle(stream))
    if r == 0:
        return q_out, k_out
    if r is not None:
        _check(r)
    a = _checked(dev, "rrhhfihh", _ROPE_NAMES, q, 0, k, 0, q_weight, D, k_weight, D, cos_sin, -1,
                 positions if rot else None, T, q_out, T * Hq * D, k_out, T * Hk * D)
    _launch(dev, stream, lib().w4a16_qk_norm_rope, a[0], a[1], a[2], a[3], a[4], a[5], a[6], rows, rot, a[7], a[8], a[9],
            T, Hq, Hk, D, eps, weight_offset, 1 if interleaved else 0)
    return q_out, k_out


def kv4_cache(num_blocks: int, Hkv: int, block_size: int, D: int, device=None) -> torch.Tensor:
    """An empty 4-bit cache, uint8 [num_blocks, Hkv, block_size / 16, 18 D]."""
    if block_size % 16 != 0:
        raise ValueError("block_size %d is not a multiple of 16" % block_size)
    return torch.zeros(num_blocks, Hkv, block_size // 16, 18 * D, dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def _cache_shape(cache):
    """Blocks, page size, heads and D of a cache tensor."""
    shape = cache.shape
    if len(shape) != 4 or shape[3] % 18 != 0:
        raise ValueError("cache must be [num_blocks, Hkv, block_size / 16, 18 D]")
    return shape[0], shape[2] * 16, shape[1], shape[3] // 18


_APPEND_NAMES = ("q", "k", "v", "q_weight", "k_weight", "cos_sin", "positions", "slots", "q_out", "cache")


def kv4_append(k, v, cache, slots, q=None, q_weight=None, k_weight=None, cos_sin=None, positions=None, q_out=None,
               eps: float = 1e-6, weight_offset: float = 0.0, interleaved: bool = False, stream=None):
    """k and v [T, Hkv, D] quantised to 4 bits into `slots` of the cache; with
    weights or cos_sin also norm and rotation of k, and of q [T, Hq, D] where
    given, in the same pass.  Returns q_out (None without q)."""
    dev = cache.device
    blocks, bs, Hkv, D = _cache_shape(cache)
    T = k.shape[0]
    for name, t in (("k", k), ("v", v)):
        if t.shape != (T, Hkv, D):
            raise ValueError("%s must be [%d, %d, %d]" % (name, T, Hkv, D))
    rows, rot = _table(cos_sin, positions)
    Hq = 0
    if q is not None:
        Tq, Hq, Dq = q.shape
        if Tq != T or Dq != D:
            raise ValueError("q must be [%d, heads, %d]" % (T, D))
        if q_out is None:
            q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    r = _extension().kv4_append(k, v, cache, slots, q, q_weight, k_weight, cos_sin, positions, q_out, float(eps),
                                float(weight_offset), interleaved, _handle(stream))
    if r == 0:
        return q_out if q is not None else None
    if r is not None:
        _check(r)
    a = _checked(dev, "rrrhhfilhb", _APPEND_NAMES, q, 0, k, 0, v, 0, q_weight, D, k_weight, D, cos_sin, -1,
                 positions if rot else None, T, slots, T, q_out if q is not None else None, T * Hq * D, cache, -1)
    _launch(dev, stream, lib().kv4_append, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], rows, rot, a[9], a[10],
            a[11], a[12], blocks, bs, T, Hq, Hkv, D, eps, weight_offset, 1 if interleaved else 0)
    return q_out if q is not None else None


def kv4_gather(cache, slots, k=None, v=None, stream=None):
    """The values the cache holds at `slots`: (k, v) bfloat16 [T, Hkv, D]."""
    dev = cache.device
    blocks, bs, Hkv, D = _cache_shape(cache)
    T = slots.numel()
    if k is None:
        k = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev)
    if v is None:
        v = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev)
    r = _extension().kv4_gather(cache, slots, k, v, _handle(stream))
    if r == 0:
        return k, v
    if r is not None:
        _check(r)
    n = T * Hkv * D
    a = _checked(dev, "blhh", ("cache", "slots", "k", "v"), cache, -1, slots, T, k, n, v, n)
    _launch(dev, stream, lib().kv4_gather, a[0], blocks, bs, a[1], a[2], a[3], T, Hkv, D)
    return k, v


def kv4_attention_scratch_bytes(Hq: int, Hkv: int, D: int) -> int:
    """Bytes of scratch memory kv4_attention needs."""
    return int(lib().kv4_attention_scratch_bytes(int(Hq), int(Hkv), int(D)))


def kv4_attention_scratch(Hq: int, Hkv: int, D: int, device=None) -> torch.Tensor:
    """A zeroed scratch buffer for kv4_attention, for calls on one stream."""
    return torch.zeros(max(kv4_attention_scratch_bytes(Hq, Hkv, D), 1), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


_ATTENTION_NAMES = ("q", "cache", "block_table", "seq_lens", "cu_new", "out", "scratch")


def kv4_attention(q, cache, block_table, seq_lens, cu_new, scratch, out=None, scale=None, window: int = 0,
                  sinks: int = 0, max_new=None, stream=None):
    """Attention of the new tokens q [T, Hq, D] over the 4-bit cache, causal
    by position; window > 0: the last `window` tokens and the first `sinks`.
    `max_new`: the most new tokens any request has (T when None); scale
    1 / sqrt(D) when None; `scratch` from kv4_attention_scratch.  Returns
    out bfloat16 [T, Hq, D]."""
    dev = cache.device
    T, Hq, D = q.shape
    if out is None:
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    scale = D ** -0.5 if scale is None else float(scale)
    max_new = max(T, 1) if max_new is None else max_new
    r = _extension().kv4_attention(q, cache, block_table, seq_lens, cu_new, scratch, out, scale, window, sinks, max_new,
                                   _handle(stream))
    if r == 0:
        return out
    if r is not None:
        _check(r)
    blocks, bs, Hkv, Dc = _cache_shape(cache)
    if Dc != D:
        raise ValueError("q has heads of %d, the cache of %d" % (D, Dc))
    B = seq_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [%d, max_blocks]" % B)
    a = _checked(dev, "rbiiihb", _ATTENTION_NAMES, q, 0, cache, -1, block_table, -1, seq_lens, B, cu_new, B + 1, out,
                 T * Hq * D, scratch, -1)
    _launch(dev, stream, lib().kv4_attention, a[0], a[1], a[2], blocks, bs, a[3], block_table.shape[1], a[4], a[5], B,
            a[6], T, Hq, Hkv, D, scale, window, sinks, max_new, a[7], scratch.numel())
    return out


def kv4_prefix_attention_scratch_bytes(T: int, requests: int, groups: int, Hq: int, Hkv: int, D: int) -> int:
    """Bytes of scratch memory kv4_prefix_attention needs for up to T new
    tokens, `requests` requests and `groups` groups."""
    return int(lib().kv4_prefix_attention_scratch_bytes(int(T), int(requests), int(groups), int(Hq), int(Hkv), int(D)))


def kv4_prefix_attention_scratch(T: int, requests: int, groups: int, Hq: int, Hkv: int, D: int, device=None) -> torch.Tensor:
    """A zeroed scratch buffer for kv4_prefix_attention, for calls on one stream."""
    return torch.zeros(max(kv4_prefix_attention_scratch_bytes(T, requests, groups, Hq, Hkv, D), 1), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


_PREFIX_NAMES = ("q", "cache", "block_table", "seq_lens", "cu_new", "prefix_lens", "cu_groups", "out", "scratch")


def kv4_prefix_attention(q, cache, block_table, seq_lens, cu_new, prefix_lens, cu_groups, scratch, out=None, scale=None,
                         max_new=None, max_group=None, stream=None):
    """kv4_attention for requests that share the first tokens of their
    contexts: those from cu_groups[g] to cu_groups[g + 1] the first
    prefix_lens[g], in the same pages.  What they share is attended to once for
    a whole group.  `max_new` and `max_group`: the most new tokens any request,
    any group has (T when None); `scratch` from kv4_prefix_attention_scratch.
    Returns out bfloat16 [T, Hq, D]."""
    dev = cache.device
    T, Hq, D = q.shape
    if out is None:
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    scale = D ** -0.5 if scale is None else float(scale)
    max_new = max(T, 1) if max_new is None else max_new
    max_group = max(T, 1) if max_group is None else max_group
    r = _extension().kv4_prefix_attention(q, cache, block_table, seq_lens, cu_new, prefix_lens, cu_groups, scratch, out,
                                          scale, max_new, max_group, _handle(stream))
    if r == 0:
        return out
    if r is not None:
        _check(r)
    blocks, bs, Hkv, Dc = _cache_shape(cache)
    if Dc != D:
        raise ValueError("q has heads of %d, the cache of %d" % (D, Dc))
    B, N = seq_lens.numel(), prefix_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [%d, max_blocks]" % B)
    a = _checked(dev, "rbiiiiihb", _PREFIX_NAMES, q, 0, cache, -1, block_table, -1, seq_lens, B, cu_new, B + 1,
                 prefix_lens, N, cu_groups, N + 1, out, T * Hq * D, scratch, -1)
    _launch(dev, stream, lib().kv4_prefix_attention, a[0], a[1], a[2], blocks, bs, a[3], block_table.shape[1], a[4], a[5], B,
            a[6], a[7], N, a[8], T, Hq, Hkv, D, scale, max_new, max_group, a[9], scratch.numel())
    return out


def kv4_bounds_buffer(num_blocks: int, Hkv: int, D: int, device=None) -> torch.Tensor:
    """Bounds of the pages of a cache, uint8 [num_blocks, Hkv, 2 D + 16], all zero."""
    return torch.zeros(num_blocks, Hkv, 2 * D + 16, dtype=torch.uint8, device=device if device is not None else "cuda")


def kv4_bounds(cache, slots, bounds, stream=None):
    """The bounds of every page whose last slot is among `slots` (int64), from
    the keys that the cache holds; call it after kv4_append with the same
    slots.  Returns `bounds`."""
    dev = cache.device
    blocks, bs, Hkv, D = _cache_shape(cache)
    r = _extension().kv4_bounds(cache, slots, bounds, _handle(stream))
    if r == 0:
        return bounds
    if r is not None:
        _check(r)
    T = slots.numel()
    a = _checked(dev, "blb", ("cache", "slots", "bounds"), cache, -1, slots, T, bounds, blocks * Hkv * (2 * D + 16))
    _launch(dev, stream, lib().kv4_bounds, a[0], blocks, bs, a[1], a[2], T, Hkv, D)
    return bounds


_SELECT_NAMES = ("q", "bounds", "block_table", "seq_lens", "cu_new", "tables", "lens")


def kv4_select(q, bounds, block_table, seq_lens, cu_new, block_size: int, top: int, first: int = 1, recent: int = 1,
               tables=None, lens=None, stream=None):
    """For every new token and key head a table of `top` pages at most: the
    `first` first and the `recent` last ones that the token sees, and of those
    between the ones with the highest scores by their bounds.  Returns
    (tables int32 [T, Hkv, top], lens int32 [T]) for kv4_sparse_attention."""
    dev = bounds.device
    T, Hq, D = q.shape
    blocks, Hkv, width = bounds.shape
    if width != 2 * D + 16:
        raise ValueError("bounds must be [num_blocks, Hkv, %d]" % (2 * D + 16))
    if top < 1:
        raise ValueError("top must be at least 1, got %d" % top)
    if tables is None:
        tables = torch.empty(T, Hkv, top, dtype=torch.int32, device=dev)
    if lens is None:
        lens = torch.empty(T, dtype=torch.int32, device=dev)
    r = _extension().kv4_select(q, bounds, block_table, seq_lens, cu_new, block_size, top, first, recent, tables, lens,
                                _handle(stream))
    if r == 0:
        return tables, lens
    if r is not None:
        _check(r)
    B = seq_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [%d, max_blocks]" % B)
    a = _checked(dev, "rbiiiii", _SELECT_NAMES, q, 0, bounds, -1, block_table, -1, seq_lens, B, cu_new, B + 1, tables,
                 T * Hkv * top, lens, T)
    _launch(dev, stream, lib().kv4_select, a[0], a[1], a[2], blocks, block_size, a[3], block_table.shape[1], a[4], a[5], B,
            T, Hq, Hkv, D, top, first, recent, a[6], a[7])
    return tables, lens


_SPARSE_NAMES = ("q", "cache", "tables", "lens", "out", "scratch")


def kv4_sparse_attention(q, cache, tables, lens, scratch, out=None, scale=None, stream=None):
    """Attention of every new token q [T, Hq, D] over pages of its own: those
    in its row of `tables` [T, Hkv, top] for the key head, of which it sees the
    first lens[t] tokens (kv4_select writes both).  `scratch` from
    kv4_attention_scratch.  Returns out bfloat16 [T, Hq, D]."""
    dev = cache.device
    T, Hq, D = q.shape
    if out is None:
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    scale = D ** -0.5 if scale is None else float(scale)
    r = _extension().kv4_sparse_attention(q, cache, tables, lens, scratch, out, scale, _handle(stream))
    if r == 0:
        return out
    if r is not None:
        _check(r)
    blocks, bs, Hkv, Dc = _cache_shape(cache)
    if Dc != D:
        raise ValueError("q has heads of %d, the cache of %d" % (D, Dc))
    if tables.dim() != 3 or tables.shape[0] != T or tables.shape[1] != Hkv:
        raise ValueError("tables must be [%d, %d, top]" % (T, Hkv))
    a = _checked(dev, "rbiihb", _SPARSE_NAMES, q, 0, cache, -1, tables, -1, lens, T, out, T * Hq * D, scratch, -1)
    _launch(dev, stream, lib().kv4_sparse_attention, a[0], a[1], a[2], blocks, bs, a[3], tables.shape[2], a[4], a[5], T, Hq,
            Hkv, D, scale, a[6], scratch.numel())
    return out


_SAMPLE_NAMES = ("u", "temperature", "top_k", "top_p", "min_p", "out")


def w4a16_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None, stream=None):
    """One token (int32) for each row of logits [rows, vocab] (float32 or
    bfloat16, rows may be strided) from the uniform numbers u [rows]; the
    settings are per-row tensors or None (off)."""
    dev = logits.device
    R, V = logits.shape
    if logits.stride(1) != 1 and V > 1:
        raise ValueError("logits must be [rows, vocab] with contiguous rows")
    dt = logits.dtype
    if dt is not torch.float32 and dt is not torch.bfloat16:
        raise TypeError("logits must be torch.float32 or torch.bfloat16, got %s" % dt)
    if out is None:
        out = torch.empty(R, dtype=torch.int32, device=dev)
    r = _extension().w4a16_sample(logits, u, temperature, top_k, top_p, min_p, out, _handle(stream))
    if r == 0:
        return out
    if r is not None:
        _check(r)
    a = _checked(dev, "ffiffi", _SAMPLE_NAMES, u, R, temperature, R, top_k, R, top_p, R, min_p, R, out, R)
    _launch(dev, stream, lib().w4a16_sample, logits.data_ptr(), OUT_F32 if dt is torch.float32 else OUT_BF16,
            logits.stride(0) if R > 1 else V, R, V, *a)
    return out


def w4a16_check_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status."""
    return int(lib().w4a16_check_device_error(_stream(stream)))


INJECT_STALL_PIPELINE = 1
INJECT_STALL_CONSUMERS = 2


def w4a16_debug_inject(flags: int = 0) -> None:
    """Test-only: make every later GEMV/MoE/GEMM launch on the current device
    issue no stage of its pipeline (flags=1), or take no stage that its
    producers issue (flags=2), so that its bounded waits run out (after about
    2 s) and the device status reports a timeout; flags=0 restores normal
    operation."""
    _check(lib().w4a16_debug_inject(int(flags)))


def w4a16_last_error_string() -> str:
    return lib().w4a16_last_error_string().decode(errors="replace")


def w4a16_version() -> int:
    return int(lib().w4a16_version())
