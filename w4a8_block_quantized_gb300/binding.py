"""ctypes binding of ``libw4a8.so`` (the C ABI in ``include/w4a8.h``).

Argument marshalling only: every step of the computation runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no CPU
fallback: if the library is missing or the GPU is not an sm_103 part, calls raise.

A call that names a `stream` runs there: the caller orders it behind what its inputs wait for, and keeps the
inputs until it is done.  What the call allocates is allocated for that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libw4a8.so")

W4A8_OK = 0
W4A8_ERR_ARG = -1
W4A8_ERR_ALIGN = -2
W4A8_ERR_SHAPE = -3
W4A8_ERR_CUDA = -4
W4A8_ERR_TIMEOUT = -5
W4A8_ERR_WORKSPACE = -6
W4A8_ERR_DEVICE = -7
W4A8_ERR_SCRATCH_LIMIT = -8
W4A8_ERR_INDEX = -9
NOALLOC_SCRATCH_BYTES = 16 << 20
OUT_F32 = 0
OUT_BF16 = 1
_OUT_DTYPES = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}
_IN_DTYPES = {torch.float32: 0, torch.bfloat16: 1}   # W4A8_IN_F32, W4A8_IN_BF16
_E8, _F32, _I8, _I32, _I64T = torch.float8_e4m3fn, torch.float32, torch.int8, torch.int32, torch.int64

# name -> (restype, argtypes); every symbol include/w4a8.h declares
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
SIGNATURES = {
    "w4a8_quant_pack": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P, _P]),
    "w4a8_linear": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]),
    "w4a8_prefill_linear": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]),
    "w4a8_prefill_linear_noalloc": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "w4a8_prefill_linear_batch": (ctypes.c_int, [_P, _I64, _I64, _P]),
    "w4a8_prepare_activations": (ctypes.c_int, [_P, _I64, _I64, _P, _SZ, _P]),
    "w4a8_prepare_weights": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _P, _SZ, _P]),
    "w4a8_linear_prepared": (ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "w4a8_linear_act": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]),
    "w4a8_linear_act_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "w4a8_prefill_linear_ex": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                                              _I64, _I64, _I64, _P, _SZ, _P]),
    "w4a8_linear_ex": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                                      _I64, _I64, _I64, _P, _SZ, _P]),
    "w4a8_linear_prepared_ex": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                                               _I64, _I64, _I64, _P]),
    "w4a8_prefill_linear_host": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]),
    "w4a8_prefill_host_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "w4a8_prepared_activations_bytes": (_SZ, [_I64, _I64]),
    "w4a8_prepared_weights_bytes": (_SZ, [_I64, _I64]),
    "w4a8_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "w4a8_prefill_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "w4a8_debug_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "w4a8_debug_block_acc": (ctypes.c_int, [_P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "w4a8_rmsnorm_quant": (ctypes.c_int, [_P, _P, _P, ctypes.c_float, ctypes.c_int, _P, _P, _P, _P, _I64, _I64, _P]),
    "w4a8_rmsnorm_prepare": (ctypes.c_int, [_P, _P, _P, ctypes.c_float, ctypes.c_int, _P, _P, _SZ, _I64, _I64, _P]),
    "w4a8_rmsnorm_quant_fp8": (ctypes.c_int, [_P, _P, _P, ctypes.c_float, ctypes.c_int, _P, _P, _P, _I64, _I64, _P]),
    "w4a8_swiglu_quant": (ctypes.c_int, [_P, _P, _I64, ctypes.c_int, _P, _P, _P, _I64, _I64, _P]),
    "w4a8_swiglu_prepare": (ctypes.c_int, [_P, _P, _I64, ctypes.c_int, _P, _SZ, _I64, _I64, _P]),
    "w4a8_swiglu_quant_fp8": (ctypes.c_int, [_P, _P, _I64, ctypes.c_int, _P, _P, _I64, _I64, _P]),
    "w4a8_quant_fp8": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _I64, _I64, _P]),
    "w4a8_fp8_linear": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _P]),
    "w4a8_rope_turns": (ctypes.c_int, [_I64, ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double,
                                       ctypes.c_double, ctypes.c_double, _P]),
    "w4a8_rope": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _I64, ctypes.c_int, _P, _P, _I64, ctypes.c_int,
                                 ctypes.c_float, _I64, _I64, _I64, _P]),
    "w4a8_kv_write": (ctypes.c_int, [_P, _P, _P]),
    "w4a8_kv_read": (ctypes.c_int, [_P, _P, _I64, _P, _P, ctypes.c_int, _P]),
    "w4a8_attention_workspace_bytes": (_SZ, [_P, _P]),
    "w4a8_attention_workspace_bound": (_SZ, [_P, _P]),
    "w4a8_attention": (ctypes.c_int, [_P, _P, _P, _SZ, _P]),
    "w4a8_tape_begin": (ctypes.c_int, [_P]),
    "w4a8_tape_end": (ctypes.c_int, [_P, ctypes.POINTER(_P)]),
    "w4a8_tape_replay": (ctypes.c_int, [_P, _P]),
    "w4a8_tape_free": (None, [_P]),
    "w4a8_tape_kernels": (ctypes.c_int64, [_P]),
    "w4a8_sync_status": (ctypes.c_int, [_P]),
    "w4a8_selftest_wait_timeout": (ctypes.c_int, [_I64, _P]),
    "w4a8_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "w4a8_abi_version": (ctypes.c_int, []),
}

_lib = None


class W4A8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libw4a8.so not found at {path}: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().w4a8_status_string(int(status)).decode()


def _check(rc: int, where: str) -> None:
    if rc != W4A8_OK:
        raise W4A8Error(rc, where)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _arg(t, dtype, shape, name: str, device=None, min_bytes=None):
    """Check one tensor argument before its address reaches the library, which cannot: a CUDA
    tensor on the call's device, contiguous, of the dtype and shape the C layout fixes (or, for
    an opaque buffer, at least ``min_bytes`` long).  ``None`` passes (optional arguments)."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (the library has no CPU path), got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if min_bytes is not None and _nbytes(t) < min_bytes:
        raise ValueError(f"{name} holds {_nbytes(t)} bytes, the call needs {min_bytes}")


def _want(t: torch.Tensor, dtype, name: str):
    _arg(t, dtype, None, name)
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device} but the current CUDA device is "
                         f"{torch.cuda.current_device()} (the library runs on the current device)")


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _weights(wq, w_scale, w_zero, N: int, K: int, device):
    _arg(wq, torch.uint8, (N, K // 2), "wq", device)
    _arg(w_scale, torch.float16, (N, K // 64), "w_scale", device)
    _arg(w_zero, torch.float16, (N, K // 64), "w_zero", device)


def _on(stream, device):
    """A context in which tensors are allocated for work on `stream` (None: the current one).  The caching allocator
    hands out a block freed on a stream at once, because what that stream does next comes behind the work that still
    uses it; another stream's work does not, so that its tensors come from memory of its own."""
    return contextlib.nullcontext() if stream is None or stream == torch.cuda.current_stream(device) else torch.cuda.stream(stream)


def _new(shape, dtype, device, stream):
    """An output allocated here, for a call on `stream`.  The caller's stream is recorded too: a block that is dropped while
    work queued there uses it goes to no other work before that is done."""
    with _on(stream, device):
        t = torch.empty(tuple(shape), dtype=dtype, device=device)
    return _returned(_taped(t, stream), stream)


_recording = []  # the tapes that are being recorded


def _taped(t, stream):
    """`t`, held by the tape that records `stream`, if one does: what a recorded call allocates is written by every replay."""
    if _recording:
        handle = (torch.cuda.current_stream(t.device) if stream is None else stream).cuda_stream
        for tape in _recording:
            if tape.recorded == handle:
                tape.keep.append(t)
    return t


def _returned(t, stream):
    if stream is not None and stream != torch.cuda.current_stream(t.device):
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _ws(ws, need: int, device, stream=None):
    """The caller's workspace (any dtype: its size in bytes is what the library is told), or
    a temporary one, allocated for `stream` and dropped when the call returns."""
    if ws is None:
        with _on(stream, device):
            return _taped(workspace(need, device), stream)
    _arg(ws, None, None, "ws", device)
    return ws


def _buffer(buf, need: int, device, stream, name: str):
    """An opaque buffer that the call returns: the caller's, or one allocated for `stream`."""
    buf = _returned(_ws(None, need, device, stream), stream) if buf is None else buf
    _arg(buf, None, None, name, device)
    return buf


def linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().w4a8_linear_workspace_bytes(M, N, K))


def prefill_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().w4a8_prefill_workspace_bytes(M, N, K))


def debug_workspace_bytes(m_cnt: int, n_cnt: int, K: int) -> int:
    return int(load().w4a8_debug_workspace_bytes(m_cnt, n_cnt, K))


_SIZE_REJECTED = (1 << 64) - 1   # what a size query returns for a shape the library rejects


def workspace(nbytes: int, device) -> torch.Tensor:
    """A caller-owned workspace buffer (uint8, at least 16-byte aligned).  For a rejected
    shape (size query = SIZE_MAX) a minimal buffer stands in: every call checks the shape
    before the workspace, so it then returns W4A8_ERR_SHAPE."""
    n = 16 if int(nbytes) == _SIZE_REJECTED else max(int(nbytes), 16)
    return torch.empty(n, dtype=torch.uint8, device=device)


def quant_pack(x: torch.Tensor, a_q=None, a_scale=None, rowsum=None, stream=None):
    """w4a8_quant_pack: x fp32 [M,K] -> (a_q int8 [M,K], s_a fp32 [M], rowsum int32 [M,K/64])."""
    _want(x, torch.float32, "x")
    M, K = x.shape
    dev = x.device
    a_q, a_scale, rowsum = _int8_out(M, K, dev, a_q, a_scale, rowsum, stream)
    rc = load().w4a8_quant_pack(_ptr(x), M, K, _ptr(a_q), _ptr(a_scale), _ptr(rowsum), _stream(stream))
    _check(rc, "w4a8_quant_pack")
    return a_q, a_scale, rowsum


def _quantized(a_q, a_scale, rowsum):
    """Shape (M, K) of a pre-quantized activation triple, after checking all three."""
    _want(a_q, torch.int8, "a_q")
    M, K = a_q.shape
    _arg(a_scale, torch.float32, (M,), "a_scale", a_q.device)
    _arg(rowsum, torch.int32, (M, K // 64), "rowsum", a_q.device)
    return M, K


def linear(a_q, a_scale, rowsum, wq, w_scale, w_zero, bias=None, y=None, ws=None, stream=None):
    """w4a8_linear: pre-quantized activations -> y fp32 [M,N]."""
    M, K = _quantized(a_q, a_scale, rowsum)
    dev = a_q.device
    N = _rows(wq)
    _weights(wq, w_scale, w_zero, N, K, dev)
    _arg(bias, torch.float32, (N,), "bias", dev)
    y = _new((M, N), torch.float32, dev, stream) if y is None else y
    _arg(y, torch.float32, (M, N), "y", dev)
    ws = _ws(ws, linear_workspace_bytes(M, N, K), dev, stream)
    rc = load().w4a8_linear(_ptr(a_q), _ptr(a_scale), _ptr(rowsum), _ptr(wq), _ptr(w_scale), _ptr(w_zero),
                            _ptr(bias), _ptr(y), M, N, K, _ptr(ws), _nbytes(ws), _stream(stream))
    _check(rc, "w4a8_linear")
    return y


def _rows(wq) -> int:
    _want(wq, torch.uint8, "wq")
    if wq.dim() != 2:
        raise ValueError(f"wq must be 2-D [N, K/2], got shape {tuple(wq.shape)}")
    return wq.shape[0]


def _prefill_args(x, wq, w_scale, w_zero, bias):
    """Shape (M, N, K) of a fused call, after checking x, the weights and the bias."""
    _want(x, torch.float32, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [M, K], got shape {tuple(x.shape)}")
    M, K = x.shape
    N = _rows(wq)
    _weights(wq, w_scale, w_zero, N, K, x.device)
    _arg(bias, torch.float32, (N,), "bias", x.device)
    return M, N, K


def prefill_linear(x, wq, w_scale, w_zero, bias=None, y=None, ws=None, stream=None):
    """w4a8_prefill_linear: fp32 x [M,K] -> y fp32 [M,N] (pre-pass + linear)."""
    M, N, K = _prefill_args(x, wq, w_scale, w_zero, bias)
    y = _new((M, N), torch.float32, x.device, stream) if y is None else y
    _arg(y, torch.float32, (M, N), "y", x.device)
    ws = _ws(ws, prefill_workspace_bytes(M, N, K), x.device, stream)
    rc = load().w4a8_prefill_linear(_ptr(x), _ptr(wq), _ptr(w_scale), _ptr(w_zero), _ptr(bias), _ptr(y),
                                    M, N, K, _ptr(ws), _nbytes(ws), _stream(stream))
    _check(rc, "w4a8_prefill_linear")
    return y


class LinearRef(ctypes.Structure):
    """w4a8_linear_ref: one entry of w4a8_prefill_linear_batch."""
    _fields_ = [("x", _P), ("wq", _P), ("w_scale", _P), ("w_zero", _P), ("bias", _P), ("y", _P),
                ("N", _I64), ("K", _I64), ("workspace", _P), ("workspace_bytes", _SZ)]


class Batch:
    """The entries of a w4a8_prefill_linear_batch call, checked and marshalled once: a sequence
    of dicts with x, wq, s_w, z_w, optional bias, y and ws (y and ws allocated when absent),
    one M for all.  `run(stream)` makes the call; `ys` are the outputs.  The tensors are held
    for the life of the object.  What is allocated here is allocated for `stream` (None: the current one); a
    run on another stream comes behind the work that was queued there by then."""

    def __init__(self, entries, stream=None):
        entries = list(entries)
        self.count = len(entries)
        self.refs = (LinearRef * max(1, self.count))()
        self.keep, self.ys, self.own, self.stream = [], [], [], stream
        self.M = 0
        for i, e in enumerate(entries):
            x, wq, sw, zw, bias = e["x"], e["wq"], e["s_w"], e["z_w"], e.get("bias")
            m, N, K = _prefill_args(x, wq, sw, zw, bias)
            if i == 0:
                self.M = m
            elif m != self.M:
                raise ValueError(f"entry {i}: x has {m} rows, the batch {self.M}")
            y = e.get("y")
            y = _new((m, N), torch.float32, x.device, stream) if y is None else y
            _arg(y, torch.float32, (m, N), "y", x.device)
            ws = _ws(e.get("ws"), prefill_workspace_bytes(m, N, K), x.device, stream)
            self.refs[i] = LinearRef(x.data_ptr(), wq.data_ptr(), sw.data_ptr(), zw.data_ptr(),
                                     None if bias is None else bias.data_ptr(), y.data_ptr(), N, K, ws.data_ptr(),
                                     _nbytes(ws))
            self.keep += [x, wq, sw, zw, bias, ws]
            self.ys.append(y)
            self.own += [t for t, given in ((y, e.get("y")), (ws, e.get("ws"))) if given is None]
        if stream is None and self.own:
            self.stream = torch.cuda.current_stream(self.own[0].device)

    def run(self, stream=None):
        if self.own:
            used = torch.cuda.current_stream(self.own[0].device) if stream is None else stream
            if used != self.stream:
                for t in self.own:
                    t.record_stream(used)
        rc = load().w4a8_prefill_linear_batch(ctypes.cast(self.refs, _P), self.count, self.M, _stream(stream))
        _check(rc, "w4a8_prefill_linear_batch")
        return self.ys


def prefill_linear_batch(entries, stream=None):
    """w4a8_prefill_linear_batch: the fused call on each entry in order (see Batch).  Returns
    the list of y."""
    return Batch(entries, stream).run(stream)


def prefill_linear_noalloc(x, wq, w_scale, w_zero, bias=None, y=None, stream=None):
    """w4a8_prefill_linear_noalloc: the fused call on the library's static scratch buffer,
    for callers that cannot allocate device memory.  Serialize calls that could overlap."""
    M, N, K = _prefill_args(x, wq, w_scale, w_zero, bias)
    y = _new((M, N), torch.float32, x.device, stream) if y is None else y
    _arg(y, torch.float32, (M, N), "y", x.device)
    rc = load().w4a8_prefill_linear_noalloc(_ptr(x), _ptr(wq), _ptr(w_scale), _ptr(w_zero), _ptr(bias), _ptr(y),
                                            M, N, K, _stream(stream))
    _check(rc, "w4a8_prefill_linear_noalloc")
    return y


def prefill_host_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().w4a8_prefill_host_workspace_bytes(M, N, K))


def _host(t, dtype, shape, name: str):
    """A host-buffer argument: a page-locked, contiguous CPU tensor of the C layout."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    # an empty tensor has no storage to pin; the library reads no pointer of an empty problem
    if t.device.type != "cpu" or (t.numel() and not t.is_pinned()):
        raise TypeError(f"{name} must be a page-locked host tensor (tensor.pin_memory())")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def prefill_linear_host(x, wq, w_scale, w_zero, bias=None, y=None, ws=None, stream=None):
    """w4a8_prefill_linear_host: page-locked host x fp32 [M,K] -> page-locked host y fp32
    [M,N]; the copies overlap the computation.  Asynchronous like every call: synchronize
    the stream before reading y."""
    _host(x, torch.float32, None, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [M, K], got shape {tuple(x.shape)}")
    M, K = x.shape
    N = _rows(wq)
    dev = wq.device
    _weights(wq, w_scale, w_zero, N, K, dev)
    _arg(bias, torch.float32, (N,), "bias", dev)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32)
        y = y.pin_memory() if y.numel() else y
    _host(y, torch.float32, (M, N), "y")
    ws = _ws(ws, prefill_host_workspace_bytes(M, N, K), dev, stream)
    rc = load().w4a8_prefill_linear_host(_ptr(x), _ptr(wq), _ptr(w_scale), _ptr(w_zero), _ptr(bias), _ptr(y),
                                         M, N, K, _ptr(ws), _nbytes(ws), _stream(stream))
    _check(rc, "w4a8_prefill_linear_host")
    return y


def prepared_activations_bytes(M: int, K: int) -> int:
    return int(load().w4a8_prepared_activations_bytes(M, K))


def prepared_weights_bytes(N: int, K: int) -> int:
    return int(load().w4a8_prepared_weights_bytes(N, K))


def prepare_activations(x, act=None, stream=None):
    """w4a8_prepare_activations: the pre-pass into an opaque buffer (returned)."""
    _want(x, torch.float32, "x")
    M, K = x.shape
    act = _buffer(act, prepared_activations_bytes(M, K), x.device, stream, "act")
    rc = load().w4a8_prepare_activations(_ptr(x), M, K, _ptr(act), _nbytes(act), _stream(stream))
    _check(rc, "w4a8_prepare_activations")
    return act


def prepare_weights(wq, w_scale, w_zero, pw=None, stream=None):
    """w4a8_prepare_weights: the tensor-core weight operand and the scale / zero layout
    (an opaque buffer, returned)."""
    N = _rows(wq)
    K = 2 * wq.shape[1]
    _weights(wq, w_scale, w_zero, N, K, wq.device)
    pw = _buffer(pw, prepared_weights_bytes(N, K), wq.device, stream, "pw")
    rc = load().w4a8_prepare_weights(_ptr(wq), _ptr(w_scale), _ptr(w_zero), N, K, _ptr(pw), _nbytes(pw),
                                     _stream(stream))
    _check(rc, "w4a8_prepare_weights")
    return pw


def _out(y, shape, device, out_dtype, stream):
    dt = torch.float32 if out_dtype is None else out_dtype
    if dt not in _OUT_DTYPES:
        raise TypeError(f"y: unsupported output dtype {dt}")
    y = _new(shape, dt, device, stream) if y is None else y
    _arg(y, dt, shape, "y", device)
    return y, _OUT_DTYPES[dt]


def prefill_linear_ex(x, wq, w_scale, w_zero, bias=None, y=None, out_dtype=None, clamp=(-math.inf, math.inf),
                      ws=None, stream=None):
    """w4a8_prefill_linear_ex: the fused call with the epilogue clamp and an fp32 or bf16 y."""
    M, N, K = _prefill_args(x, wq, w_scale, w_zero, bias)
    y, code = _out(y, (M, N), x.device, out_dtype if y is None else y.dtype, stream)
    ws = _ws(ws, prefill_workspace_bytes(M, N, K), x.device, stream)
    rc = load().w4a8_prefill_linear_ex(_ptr(x), _ptr(wq), _ptr(w_scale), _ptr(w_zero), _ptr(bias), _ptr(y), code,
                                       float(clamp[0]), float(clamp[1]), M, N, K, _ptr(ws), _nbytes(ws),
                                       _stream(stream))
    _check(rc, "w4a8_prefill_linear_ex")
    return y


def linear_ex(a_q, a_scale, rowsum, wq, w_scale, w_zero, bias=None, y=None, out_dtype=None,
              clamp=(-math.inf, math.inf), ws=None, stream=None):
    """w4a8_linear_ex: pre-quantized activations, epilogue clamp, fp32 or bf16 y."""
    M, K = _quantized(a_q, a_scale, rowsum)
    dev = a_q.device
    N = _rows(wq)
    _weights(wq, w_scale, w_zero, N, K, dev)
    _arg(bias, torch.float32, (N,), "bias", dev)
    y, code = _out(y, (M, N), dev, out_dtype if y is None else y.dtype, stream)
    ws = _ws(ws, linear_workspace_bytes(M, N, K), dev, stream)
    rc = load().w4a8_linear_ex(_ptr(a_q), _ptr(a_scale), _ptr(rowsum), _ptr(wq), _ptr(w_scale), _ptr(w_zero),
                               _ptr(bias), _ptr(y), code, float(clamp[0]), float(clamp[1]), M, N, K, _ptr(ws),
                               _nbytes(ws), _stream(stream))
    _check(rc, "w4a8_linear_ex")
    return y


def _prepared(act, pw, bias, M: int, N: int, K: int):
    """Check the opaque operands of a prepared call against the sizes the library derives
    from (M, N, K): the C call takes no buffer lengths, so this is the only check."""
    _want(act, None, "act")
    dev = act.device
    if min(M, N, K) < 0:
        raise ValueError(f"negative size in (M, N, K) = {(M, N, K)}")
    if M and N and K > 0 and K % 64 == 0:
        _arg(act, None, None, "act", dev, min_bytes=prepared_activations_bytes(M, K))
        _arg(pw, None, None, "pw", dev, min_bytes=prepared_weights_bytes(N, K))
    else:
        _arg(pw, None, None, "pw", dev)
    _arg(bias, torch.float32, (N,), "bias", dev)
    return dev


def linear_prepared_ex(act, pw, M: int, N: int, K: int, bias=None, y=None, out_dtype=None,
                       clamp=(-math.inf, math.inf), stream=None):
    """w4a8_linear_prepared_ex: prepared operands, epilogue clamp, fp32 or bf16 y."""
    dev = _prepared(act, pw, bias, M, N, K)
    y, code = _out(y, (M, N), dev, out_dtype if y is None else y.dtype, stream)
    rc = load().w4a8_linear_prepared_ex(_ptr(act), _ptr(pw), _ptr(bias), _ptr(y), code, float(clamp[0]),
                                        float(clamp[1]), M, N, K, _stream(stream))
    _check(rc, "w4a8_linear_prepared_ex")
    return y


def linear_prepared(act, pw, M: int, N: int, K: int, bias=None, y=None, stream=None):
    """w4a8_linear_prepared: contraction + epilogue from prepared operands -> y fp32 [M,N]."""
    dev = _prepared(act, pw, bias, M, N, K)
    y = _new((M, N), torch.float32, dev, stream) if y is None else y
    _arg(y, torch.float32, (M, N), "y", dev)
    rc = load().w4a8_linear_prepared(_ptr(act), _ptr(pw), _ptr(bias), _ptr(y), M, N, K, _stream(stream))
    _check(rc, "w4a8_linear_prepared")
    return y


def linear_act_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().w4a8_linear_act_workspace_bytes(M, N, K))


def linear_act(act, wq, w_scale, w_zero, M: int, N: int, K: int, bias=None, y=None, ws=None, stream=None):
    """w4a8_linear_act: contraction + epilogue from prepared activations and the packed
    weights as given -> y fp32 [M,N]."""
    _want(act, None, "act")
    dev = act.device
    if min(M, N, K) < 0:
        raise ValueError(f"negative size in (M, N, K) = {(M, N, K)}")
    if M and N and K > 0 and K % 64 == 0:
        _arg(act, None, None, "act", dev, min_bytes=prepared_activations_bytes(M, K))
    _weights(wq, w_scale, w_zero, N, K, dev)
    _arg(bias, torch.float32, (N,), "bias", dev)
    y = _new((M, N), torch.float32, dev, stream) if y is None else y
    _arg(y, torch.float32, (M, N), "y", dev)
    ws = _ws(ws, linear_act_workspace_bytes(M, N, K), dev, stream)
    rc = load().w4a8_linear_act(_ptr(act), _ptr(wq), _ptr(w_scale), _ptr(w_zero), _ptr(bias), _ptr(y), M, N, K,
                                _ptr(ws), _nbytes(ws), _stream(stream))
    _check(rc, "w4a8_linear_act")
    return y


# ---------------------------------------------------------------- operators around the linears
# These calls are short on the GPU (a few microseconds for a token), so what Python does around
# the library call counts.  Where every output is given, a call checks its tensors in one
# expression over cheap attributes; where that fails (or outputs are to be allocated) it goes
# through the checks that name the offending argument.  Addresses are passed as plain integers,
# and the current stream is taken as a raw handle.  Measured on the GPU's host, one token through
# rmsnorm_quant: 13.7 -> 5.8 us a call (the library call itself 2.6; a stream object alone costs 2.8,
# the raw handle 0.08).
# (They are not public torch names, and a torch without CUDA lacks them: the public calls stand in.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _handle(index: int, stream) -> int:
    return _raw_stream(index) if stream is None else stream.cuda_stream


def _adr(t):
    return None if t is None else t.data_ptr()


def _rows_in(x, name: str):
    """Shape (M, K), input type code and device of a row operator's 2-D contiguous input."""
    _want(x, None, name)
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D [M, K], got shape {tuple(x.shape)}")
    if x.dtype not in _IN_DTYPES:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {x.dtype}")
    return x.shape[0], x.shape[1], _IN_DTYPES[x.dtype], x.device


def _norm_in(x, weight, residual, residual_out, stream):
    M, K, code, dev = _rows_in(x, "x")
    _arg(weight, torch.float32, (K,), "weight", dev)
    if weight is None:
        raise TypeError("weight must be a torch.Tensor, got None")
    _arg(residual, x.dtype, (M, K), "residual", dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without a residual")
    elif residual_out is None:
        residual_out = _new((M, K), x.dtype, dev, stream)
    else:
        _arg(residual_out, x.dtype, (M, K), "residual_out", dev)
    return M, K, code, dev, residual_out


def _gate_up(gate, up):
    """(M, K, row stride, input type code, device) of two [M, K] tensors with unit column stride and
    one row stride, e.g. the halves of one projection's output."""
    for t, name in ((gate, "gate"), (up, "up")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor (the library has no CPU path), got {t.device}")
    if gate.dtype not in _IN_DTYPES:
        raise TypeError(f"gate must be torch.float32 or torch.bfloat16, got {gate.dtype}")
    if up.dtype is not gate.dtype:
        raise TypeError(f"up must be {gate.dtype}, got {up.dtype}")
    if gate.dim() != 2 or up.shape != gate.shape:
        raise ValueError(f"gate and up must be 2-D of one shape, got {tuple(gate.shape)} and {tuple(up.shape)}")
    M, K = gate.shape
    (ld, one), (ldu, oneu) = gate.stride(), up.stride()
    if M and K and (one != 1 or oneu != 1 or (M > 1 and (ldu != ld or ld < K))):
        raise ValueError(f"gate and up must have unit column stride and one row stride, got strides "
                         f"{gate.stride()} and {up.stride()}")
    dev = gate.get_device()
    if up.get_device() != dev:
        raise ValueError(f"up is on {up.device}, the call's other tensors on {gate.device}")
    if dev != torch.cuda.current_device():
        raise ValueError(f"gate is on {gate.device} but the current CUDA device is "
                         f"{torch.cuda.current_device()} (the library runs on the current device)")
    return M, K, (ld if M > 1 else K), _IN_DTYPES[gate.dtype], gate.device


def _int8_out(M, K, dev, a_q, a_scale, rowsum, stream):
    a_q = _new((M, K), _I8, dev, stream) if a_q is None else a_q
    a_scale = _new((M,), _F32, dev, stream) if a_scale is None else a_scale
    rowsum = _new((M, K // 64), _I32, dev, stream) if rowsum is None else rowsum
    _arg(a_q, _I8, (M, K), "a_q", dev)
    _arg(a_scale, _F32, (M,), "a_scale", dev)
    _arg(rowsum, _I32, (M, K // 64), "rowsum", dev)
    return a_q, a_scale, rowsum


def _e4m3_out(M, K, dev, a_q, a_scale, stream):
    nb = (K + 127) // 128
    a_q = _new((M, K), _E8, dev, stream) if a_q is None else a_q
    a_scale = _new((nb, M), _F32, dev, stream) if a_scale is None else a_scale
    _arg(a_q, _E8, (M, K), "a_q", dev)
    _arg(a_scale, _F32, (nb, M), "a_scale", dev)
    return a_q, a_scale


# what a missing or foreign argument raises in those expressions: the naming checks follow
_NOT_FITTING = (AttributeError, KeyError, TypeError, ValueError)


def rmsnorm_quant(x, weight, eps, residual=None, residual_out=None, a_q=None, a_scale=None, rowsum=None, stream=None):
    """w4a8_rmsnorm_quant: rms_norm(x + residual) * weight as INT8 codes for `linear`.  Returns
    (a_q int8 [M,K], a_scale fp32 [M], rowsum int32 [M,K/64], x + residual or None)."""
    try:
        M, K = shape = x.shape
        index, dt = x.get_device(), x.dtype
        code = _IN_DTYPES[dt]
        fits = weight.dtype is _F32 and residual.dtype is dt and residual_out.dtype is dt and a_q.dtype is _I8 and \
            a_scale.dtype is _F32 and rowsum.dtype is _I32 and weight.shape == (K,) and residual.shape == shape and \
            residual_out.shape == shape and a_q.shape == shape and a_scale.shape == (M,) and \
            rowsum.shape == (M, K // 64) and weight.get_device() == index and residual.get_device() == index and \
            residual_out.get_device() == index and a_q.get_device() == index and a_scale.get_device() == index and \
            rowsum.get_device() == index and x.is_contiguous() and weight.is_contiguous() and \
            residual.is_contiguous() and residual_out.is_contiguous() and a_q.is_contiguous() and \
            a_scale.is_contiguous() and rowsum.is_contiguous() and index == _current_device()
    except _NOT_FITTING:
        fits = False
    if not fits:
        M, K, code, dev, residual_out = _norm_in(x, weight, residual, residual_out, stream)
        a_q, a_scale, rowsum = _int8_out(M, K, dev, a_q, a_scale, rowsum, stream)
        index = dev.index
    rc = (_lib or load()).w4a8_rmsnorm_quant(
        x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(), eps, code,
        None if residual_out is None else residual_out.data_ptr(), a_q.data_ptr(), a_scale.data_ptr(),
        rowsum.data_ptr(), M, K, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "w4a8_rmsnorm_quant")
    return a_q, a_scale, rowsum, residual_out


def rmsnorm_prepare(x, weight, eps, residual=None, residual_out=None, act=None, stream=None):
    """w4a8_rmsnorm_prepare: rms_norm(x + residual) * weight as the opaque operand of
    `linear_prepared` and `linear_act`.  Returns (act, x + residual or None)."""
    M, K, code, dev, residual_out = _norm_in(x, weight, residual, residual_out, stream)
    act = _buffer(act, prepared_activations_bytes(M, K), dev, stream, "act")
    rc = load().w4a8_rmsnorm_prepare(x.data_ptr(), _adr(residual), weight.data_ptr(), eps, code, _adr(residual_out),
                                     act.data_ptr(), _nbytes(act), M, K, _handle(dev.index, stream))
    _check(rc, "w4a8_rmsnorm_prepare")
    return act, residual_out


def rmsnorm_quant_fp8(x, weight, eps, residual=None, residual_out=None, a_q=None, a_scale=None, stream=None):
    """w4a8_rmsnorm_quant_fp8: rms_norm(x + residual) * weight as e4m3 codes for `fp8_linear`.
    Returns (a_q e4m3 [M,K], a_scale fp32 [ceil(K/128),M], x + residual or None)."""
    try:
        M, K = shape = x.shape
        index, dt = x.get_device(), x.dtype
        code = _IN_DTYPES[dt]
        fits = weight.dtype is _F32 and residual.dtype is dt and residual_out.dtype is dt and a_q.dtype is _E8 and \
            a_scale.dtype is _F32 and weight.shape == (K,) and residual.shape == shape and \
            residual_out.shape == shape and a_q.shape == shape and a_scale.shape == ((K + 127) // 128, M) and \
            weight.get_device() == index and residual.get_device() == index and \
            residual_out.get_device() == index and a_q.get_device() == index and a_scale.get_device() == index and \
            x.is_contiguous() and weight.is_contiguous() and residual.is_contiguous() and \
            residual_out.is_contiguous() and a_q.is_contiguous() and a_scale.is_contiguous() and \
            index == _current_device()
    except _NOT_FITTING:
        fits = False
    if not fits:
        M, K, code, dev, residual_out = _norm_in(x, weight, residual, residual_out, stream)
        a_q, a_scale = _e4m3_out(M, K, dev, a_q, a_scale, stream)
        index = dev.index
    rc = (_lib or load()).w4a8_rmsnorm_quant_fp8(
        x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(), eps, code,
        None if residual_out is None else residual_out.data_ptr(), a_q.data_ptr(), a_scale.data_ptr(), M, K,
        _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "w4a8_rmsnorm_quant_fp8")
    return a_q, a_scale, residual_out


def swiglu_quant(gate, up, a_q=None, a_scale=None, rowsum=None, stream=None):
    """w4a8_swiglu_quant: silu(gate) * up as INT8 codes for `linear`.  Returns (a_q, a_scale, rowsum)."""
    M, K, ld, code, dev = _gate_up(gate, up)
    a_q, a_scale, rowsum = _int8_out(M, K, dev, a_q, a_scale, rowsum, stream)
    rc = load().w4a8_swiglu_quant(gate.data_ptr(), up.data_ptr(), ld, code, a_q.data_ptr(), a_scale.data_ptr(),
                                  rowsum.data_ptr(), M, K, _handle(dev.index, stream))
    _check(rc, "w4a8_swiglu_quant")
    return a_q, a_scale, rowsum


def swiglu_prepare(gate, up, act=None, stream=None):
    """w4a8_swiglu_prepare: silu(gate) * up as the opaque operand of `linear_prepared` and
    `linear_act` (returned)."""
    M, K, ld, code, dev = _gate_up(gate, up)
    act = _buffer(act, prepared_activations_bytes(M, K), dev, stream, "act")
    rc = load().w4a8_swiglu_prepare(gate.data_ptr(), up.data_ptr(), ld, code, act.data_ptr(), _nbytes(act), M, K,
                                    _handle(dev.index, stream))
    _check(rc, "w4a8_swiglu_prepare")
    return act


def swiglu_quant_fp8(gate, up, a_q=None, a_scale=None, stream=None):
    """w4a8_swiglu_quant_fp8: silu(gate) * up as e4m3 codes for `fp8_linear`.  Returns
    (a_q e4m3 [M,K], a_scale fp32 [ceil(K/128),M])."""
    try:
        M, K = shape = gate.shape
        index, dt, strides = gate.get_device(), gate.dtype, gate.stride()
        code, ld = _IN_DTYPES[dt], strides[0] if M > 1 else K  # the stride of a single row says nothing
        fits = up.shape == shape and up.dtype is dt and up.get_device() == index and up.stride() == strides and \
            strides[1] == 1 and ld >= K and a_q.dtype is _E8 and a_scale.dtype is _F32 and a_q.shape == shape and \
            a_scale.shape == ((K + 127) // 128, M) and a_q.get_device() == index and \
            a_scale.get_device() == index and a_q.is_contiguous() and a_scale.is_contiguous() and \
            index == _current_device()
    except _NOT_FITTING:
        fits = False
    if not fits:
        M, K, ld, code, dev = _gate_up(gate, up)
        a_q, a_scale = _e4m3_out(M, K, dev, a_q, a_scale, stream)
        index = dev.index
    rc = (_lib or load()).w4a8_swiglu_quant_fp8(
        gate.data_ptr(), up.data_ptr(), ld, code, a_q.data_ptr(), a_scale.data_ptr(), M, K,
        _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "w4a8_swiglu_quant_fp8")
    return a_q, a_scale


def quant_fp8(x, a_q=None, a_scale=None, stream=None):
    """w4a8_quant_fp8: x as e4m3 codes for `fp8_linear`.  Returns (a_q, a_scale)."""
    M, K, code, dev = _rows_in(x, "x")
    a_q, a_scale = _e4m3_out(M, K, dev, a_q, a_scale, stream)
    rc = load().w4a8_quant_fp8(x.data_ptr(), code, a_q.data_ptr(), a_scale.data_ptr(), M, K,
                               _handle(dev.index, stream))
    _check(rc, "w4a8_quant_fp8")
    return a_q, a_scale


def _fp8_in(a_q, a_scale, w_q, w_scale, bias, y, out_dtype, stream):
    """The checks of fp8_linear that name the offending argument; y allocated when absent."""
    _want(a_q, torch.float8_e4m3fn, "a_q")
    _want(w_q, torch.float8_e4m3fn, "w_q")
    if a_q.dim() != 2 or w_q.dim() != 2:
        raise ValueError(f"a_q and w_q must be 2-D, got shapes {tuple(a_q.shape)} and {tuple(w_q.shape)}")
    M, K = a_q.shape
    N = w_q.shape[0]
    dev, nb = a_q.device, (K + 127) // 128
    _arg(w_q, torch.float8_e4m3fn, (N, K), "w_q", dev)
    _arg(a_scale, torch.float32, (nb, M), "a_scale", dev)
    _arg(w_scale, torch.float32, ((N + 127) // 128, nb), "w_scale", dev)
    if a_scale is None or w_scale is None:
        raise TypeError("a_scale and w_scale must be torch.Tensors")
    _arg(bias, torch.float32, (N,), "bias", dev)
    y, _ = _out(y, (M, N), dev, out_dtype if y is None else y.dtype, stream)
    return M, N, K, y


def fp8_linear(a_q, a_scale, w_q, w_scale, bias=None, y=None, out_dtype=None, stream=None):
    """w4a8_fp8_linear: e4m3 activations [M,K] with a_scale fp32 [ceil(K/128),M], e4m3 weights
    [N,K] with w_scale fp32 [ceil(N/128),ceil(K/128)] -> y fp32 or bf16 [M,N]."""
    try:
        (M, K), (N, _) = a_q.shape, w_q.shape
        nb, index = (K + 127) // 128, a_q.get_device()
        code = _OUT_DTYPES[y.dtype]
        fits = a_q.dtype is _E8 and w_q.dtype is _E8 and a_scale.dtype is _F32 and w_scale.dtype is _F32 and \
            a_scale.shape == (nb, M) and w_scale.shape == ((N + 127) // 128, nb) and w_q.shape == (N, K) and \
            y.shape == (M, N) and w_q.get_device() == index and a_scale.get_device() == index and \
            w_scale.get_device() == index and y.get_device() == index and a_q.is_contiguous() and \
            w_q.is_contiguous() and a_scale.is_contiguous() and w_scale.is_contiguous() and y.is_contiguous() and \
            (bias is None or (bias.dtype is _F32 and bias.shape == (N,) and bias.get_device() == index and
                              bias.is_contiguous())) and index == _current_device()
    except _NOT_FITTING:
        fits = False
    if not fits:
        M, N, K, y = _fp8_in(a_q, a_scale, w_q, w_scale, bias, y, out_dtype, stream)
        index, code = y.get_device(), _OUT_DTYPES[y.dtype]
    rc = (_lib or load()).w4a8_fp8_linear(
        a_q.data_ptr(), a_scale.data_ptr(), w_q.data_ptr(), w_scale.data_ptr(),
        None if bias is None else bias.data_ptr(), y.data_ptr(), code,
        M, N, K, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "w4a8_fp8_linear")
    return y


# ---------------------------------------------------------------- rotary positions, cache, attention
_ROPE_SCALINGS = {None: 0, "linear": 1, "base": 2, "bands": 3}
_KV_FORMATS = {_I8: 0, _E8: 1}   # W4A8_KV_INT8, W4A8_KV_E4M3


def rope_table(rot, base=10000.0, scaling=None, factor=1.0, original_len=0.0, low=1.0, high=4.0, device="cuda"):
    """w4a8_rope_turns: the frequencies of a rotary embedding over `rot` values, base^(-2i/rot), as the
    int64 [rot/2] table (64-bit fractions of a turn a position) that `rope` and `kv_write` take.
    scaling, for contexts `factor` times longer than the model's: "linear" (all frequencies / factor),
    "base" (a larger base) or "bands" (frequencies of fewer than `low` turns over original_len
    positions / factor, of more than `high` kept, a blend between)."""
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {tuple(_ROPE_SCALINGS)}, got {scaling!r}")
    rot = int(rot)
    turns = torch.empty((max(rot, 0) // 2,), dtype=torch.int64)
    _check(load().w4a8_rope_turns(rot, base, _ROPE_SCALINGS[scaling], factor, original_len, low, high,
                                  turns.data_ptr()), "w4a8_rope_turns")
    return turns.to(device)


class _KvCache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("pages", _I64), ("heads", _I64),
                ("page", _I64), ("head_dim", _I64), ("format", ctypes.c_int)]


class _KvRows(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("q", _P), ("q_out", _P), ("k_token", _I64), ("k_head", _I64),
                ("v_token", _I64), ("v_head", _I64), ("q_token", _I64), ("q_head", _I64), ("q_out_token", _I64),
                ("q_out_head", _I64), ("slots", _P), ("positions", _P), ("turns", _P), ("tokens", _I64),
                ("q_heads", _I64), ("rot", _I64), ("dtype", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("magnitude", ctypes.c_float)]


class _AttentionArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("out", _P), ("q_token", _I64), ("q_head", _I64), ("out_token", _I64), ("out_head", _I64),
                ("page_table", _P), ("kv_len", _P), ("q_start", _P), ("table_stride", _I64), ("batch", _I64),
                ("total", _I64), ("q_heads", _I64), ("max_q", _I64), ("max_kv", _I64), ("window", _I64),
                ("sinks", _I64), ("q_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("scale", ctypes.c_float)]


# the two argument blocks as bytes, field by field as in the structures: packed in 1 us, for 3 that a structure takes
_pack_rows = struct.Struct("@4Q8q3Q3q2if").pack
_pack_attention = struct.Struct("@2Q4q3Q8q2if").pack


class KVCache:
    """w4a8_kv_cache: a layer's keys and values in 8 bits, in pages.  Codes k and v int8 or float8_e4m3fn
    [pages, heads, page, head_dim], scales k_scale and v_scale fp32 [pages, heads, page], checked once;
    `slot` page_number * page + offset names a token's place.  The tensors are held for the life of
    the object."""

    def __init__(self, k, v, k_scale, v_scale):
        _arg(k, None, None, "k")
        if k is None or k.dtype not in _KV_FORMATS:
            raise TypeError(f"k must be torch.int8 or torch.float8_e4m3fn, got {None if k is None else k.dtype}")
        if k.dim() != 4:
            raise ValueError(f"k must be 4-D [pages, heads, page, head_dim], got shape {tuple(k.shape)}")
        for t, name in ((v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None:
                raise TypeError(f"{name} must be a torch.Tensor, got None")
        _arg(v, k.dtype, k.shape, "v", k.device)
        _arg(k_scale, _F32, k.shape[:3], "k_scale", k.device)
        _arg(v_scale, _F32, k.shape[:3], "v_scale", k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page, self.head_dim = k.shape
        self.index = k.get_device()
        self.c = _KvCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *k.shape,
                          _KV_FORMATS[k.dtype])
        self.ref = ctypes.addressof(self.c)
        self.inner = (self.heads, self.head_dim)

    def __setattr__(self, name, value):
        """Set once: the library holds the arrays' addresses."""
        if name in self.__dict__:
            raise AttributeError(f"a KVCache's {name} cannot be replaced (fill its arrays in place, or make another)")
        super().__setattr__(name, value)

    @classmethod
    def empty(cls, pages, heads, page, head_dim, dtype=torch.int8, device="cuda"):
        """A cache of zeros."""
        k, v = (torch.zeros((pages, heads, page, head_dim), dtype=torch.uint8, device=device).view(dtype) for _ in "kv")
        return cls(k, v, *(torch.zeros((pages, heads, page), dtype=_F32, device=device) for _ in "kv"))


def _cache_arg(cache):
    if not isinstance(cache, KVCache):
        raise TypeError(f"cache must be a KVCache, got {type(cache).__name__}")
    if cache.index != _current_device():
        raise ValueError(f"cache is on {cache.k.device} but the current CUDA device is {_current_device()} "
                         "(the library runs on the current device)")


def _heads_arg(t, name, device, dtype=None, shape=None):
    """Token and head stride of a [tokens, heads, head_dim] tensor with unit stride inside a head."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (the library has no CPU path), got {t.device}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{device}")
    if t.dtype not in _IN_DTYPES:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {'[tokens, heads, head_dim]' if shape is None else tuple(shape)}, "
                         f"got {tuple(t.shape)}")
    a, b, one = t.stride()
    if one != 1 and t.shape[2] > 1 and t.numel():
        raise ValueError(f"{name} must have unit stride inside a head, got strides {t.stride()}")
    return a, b


def _rotary_arg(positions, table, tokens, head_dim, index):
    _arg(positions, _I32, (tokens,), "positions")
    _arg(table, torch.int64, None, "table")
    if positions is None or table is None:
        raise TypeError("positions and table must be torch.Tensors")
    for t, name in ((positions, "positions"), (table, "table")):
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{index}")
    if table.dim() != 1 or not 0 < 2 * table.numel() <= head_dim:
        raise ValueError(f"table must be 1-D with at most head_dim / 2 entries, got shape {tuple(table.shape)}")
    return 2 * table.numel()


def _slots_arg(slots, index):
    _arg(slots, torch.int64, None, "slots")
    if slots is None:
        raise TypeError("slots must be a torch.Tensor, got None")
    if slots.dim() != 1 or slots.get_device() != index:
        raise ValueError(f"slots must be 1-D on cuda:{index}, got shape {tuple(slots.shape)} on {slots.device}")
    return slots.shape[0]


def _apart(a, b, name, in_place=True):
    """Output a and input b of one launch: no common memory, or (in_place) the very same rows."""
    if in_place and a.data_ptr() == b.data_ptr() and a.stride() == b.stride() and a.shape == b.shape:
        return
    ends = [t.data_ptr() + t.element_size() * (1 + sum((n - 1) * st for n, st in zip(t.shape, t.stride())))
            for t in (a, b)]
    if a.numel() and b.numel() and a.data_ptr() < ends[1] and b.data_ptr() < ends[0] and not _interleaved(a, b):
        raise ValueError(f"{name} overlaps an input of the call")


def _interleaved(a, b):
    """Two slices of one [tokens, width] array, each inside columns of its own; all in bytes: their types may differ."""
    st = a.stride(0) * a.element_size()
    if st != b.stride(0) * b.element_size() or a.shape[0] < 2 or st == 0:
        return False
    width = [t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape[1:], t.stride()[1:]))) for t in (a, b)]
    gap = (b.data_ptr() - a.data_ptr()) % st
    return width[0] <= gap and gap + width[1] <= st


def rope(x, positions, table, interleaved=False, magnitude=1.0, out=None, stream=None):
    """w4a8_rope: the rotary embedding of x fp32 or bf16 [tokens, heads, head_dim] (any token and head
    strides) at positions int32 [tokens]; pairs (i, i + rot/2) of the first rot = 2 * len(table)
    values, or neighbours where `interleaved`; times `magnitude`.  Returns out (allocated when
    absent; x itself: in place)."""
    try:
        T, H, D = shape = x.shape
        dt, index, (n,) = x.dtype, x.get_device(), table.shape
        (xt, xh, one), (ot, oh, other), rot = x.stride(), out.stride(), 2 * n
        px, po, code = x.data_ptr(), out.data_ptr(), _IN_DTYPES[dt]
        el = 4 - 2 * code  # bytes; apart, or the very same rows
        fits = one == 1 and other == 1 and out.dtype is dt and out.shape == shape and 0 < rot <= D and \
            positions.dtype is _I32 and positions.shape == (T,) and table.dtype is _I64T and \
            positions.is_contiguous() and table.is_contiguous() and out.get_device() == index and \
            positions.get_device() == index and table.get_device() == index and index == _current_device() and \
            (po >= px + el * ((T - 1) * xt + (H - 1) * xh + D) or px >= po + el * ((T - 1) * ot + (H - 1) * oh + D) or
             (px == po and xt == ot and xh == oh))
    except _NOT_FITTING:
        fits = False
    if not fits:
        index = _current_device()
        xt, xh = _heads_arg(x, "x", index)
        T, H, D = x.shape
        rot = _rotary_arg(positions, table, T, D, index)
        if out is None:
            out = _new((T, H, D), x.dtype, x.device, stream)
        ot, oh = _heads_arg(out, "out", index, x.dtype, x.shape)
        if out is not x:
            _apart(out, x, "out")
        px, po, code = x.data_ptr(), out.data_ptr(), _IN_DTYPES[x.dtype]
    rc = (_lib or load()).w4a8_rope(px, xt, xh, po, ot, oh, code, positions.data_ptr(), table.data_ptr(), rot,
                                    interleaved, magnitude, T, H, D,
                                    _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "w4a8_rope")
    return out


def kv_write(cache, k, v, slots, positions=None, table=None, interleaved=False, magnitude=1.0, q=None, q_out=None,
             stream=None):
    """w4a8_kv_write: a step's k and v [tokens, cache.heads, head_dim] into the cache's slots (int64 [tokens],
    negative: left out).  With `table` k is rotated on the way, and q [tokens, heads, head_dim], if
    given, into q_out (allocated when absent; q itself: in place).  Returns q_out, or None."""
    try:
        T, heads, D = q.shape
        dt, index, (n,) = k.dtype, cache.index, table.shape
        shape, rot, code = (T, *cache.inner), 2 * n, _IN_DTYPES[dt]
        (kt, kh, k1), (vt, vh, v1), (qt, qh, q1), (ot, oh, o1) = k.stride(), v.stride(), q.stride(), q_out.stride()
        pk, pv, pq, po = k.data_ptr(), v.data_ptr(), q.data_ptr(), q_out.data_ptr()
        el, t1, h1, m1 = 4 - 2 * code, T - 1, heads - 1, shape[1] - 1
        inputs_end = max(pk + el * (t1 * kt + m1 * kh + D), pv + el * (t1 * vt + m1 * vh + D), pq + el * (t1 * qt + h1 * qh + D))
        fits = k1 == v1 == q1 == o1 == 1 and v.dtype is dt and q.dtype is dt and q_out.dtype is dt and \
            k.shape == shape and v.shape == shape and D == shape[2] and q_out.shape == (T, heads, D) and \
            slots.dtype is _I64T and slots.shape == (T,) and positions.dtype is _I32 and positions.shape == (T,) and \
            table.dtype is _I64T and 0 < rot <= D and slots.is_contiguous() and \
            positions.is_contiguous() and table.is_contiguous() and k.get_device() == index and \
            v.get_device() == index and q.get_device() == index and q_out.get_device() == index and \
            slots.get_device() == index and positions.get_device() == index and table.get_device() == index and \
            index == _current_device() and (po >= inputs_end or min(pk, pv, pq) >= po + el * (t1 * ot + h1 * oh + D))
        ps, pp, pt = slots.data_ptr(), positions.data_ptr(), table.data_ptr()
    except _NOT_FITTING:
        fits = False
    if not fits:
        _cache_arg(cache)
        index = cache.index
        T = _slots_arg(slots, index)
        shape = (T, cache.heads, cache.head_dim)
        kt, kh = _heads_arg(k, "k", index, None, shape)
        vt, vh = _heads_arg(v, "v", index, k.dtype, shape)
        rot = pp = pt = 0
        if table is not None:
            rot = _rotary_arg(positions, table, T, cache.head_dim, index)
            pp, pt = positions.data_ptr(), table.data_ptr()
        qt = qh = ot = oh = heads = pq = po = 0
        if q is not None:
            if table is None:
                raise ValueError("q is only rotated: it needs positions and table")
            qt, qh = _heads_arg(q, "q", index, k.dtype)
            if q.shape[0] != T or q.shape[2] != cache.head_dim:
                raise ValueError(f"q must have shape [{T}, heads, {cache.head_dim}], got {tuple(q.shape)}")
            heads = q.shape[1]
            if q_out is None:
                q_out = _new(q.shape, q.dtype, q.device, stream)
            ot, oh = _heads_arg(q_out, "q_out", index, q.dtype, q.shape)
            if q_out is not q:
                _apart(q_out, q, "q_out")
            _apart(q_out, k, "q_out", in_place=False)
            _apart(q_out, v, "q_out", in_place=False)
            pq, po = q.data_ptr(), q_out.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out without a q")
        pk, pv, ps, code = k.data_ptr(), v.data_ptr(), slots.data_ptr(), _IN_DTYPES[k.dtype]
    rc = (_lib or load()).w4a8_kv_write(
        cache.ref, _pack_rows(pk, pv, pq, po, kt, kh, vt, vh, qt, qh, ot, oh, ps, pp, pt, T, heads, rot, code,
                              interleaved, magnitude), _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "w4a8_kv_write")
    return q_out


def kv_read(cache, slots, dtype=None, k=None, v=None, stream=None):
    """w4a8_kv_read: the stored keys and values of the slots (int64 [tokens]) as (k, v), each
    [tokens, cache.heads, head_dim] of `dtype` (bf16 where absent) or the type of the k and v given;
    zeros for a negative slot."""
    try:
        (T,), index, want = slots.shape, cache.index, k.dtype
        shape, code = (T, *cache.inner), _IN_DTYPES[want]
        fits = dtype is None and slots.dtype is _I64T and v.dtype is want and k.shape == shape and v.shape == shape and \
            slots.is_contiguous() and k.is_contiguous() and v.is_contiguous() and slots.get_device() == index and \
            k.get_device() == index and v.get_device() == index and index == _current_device() and \
            abs(k.data_ptr() - v.data_ptr()) >= (4 - 2 * code) * k.numel()
    except _NOT_FITTING:
        fits = False
    if not fits:
        _cache_arg(cache)
        index = cache.index
        T = _slots_arg(slots, index)
        shape = (T, cache.heads, cache.head_dim)
        want = dtype if dtype is not None else torch.bfloat16 if k is None and v is None else (v if k is None else k).dtype
        if want not in _IN_DTYPES:
            raise TypeError(f"dtype must be torch.float32 or torch.bfloat16, got {want}")
        code = _IN_DTYPES[want]
        k = _new(shape, want, slots.device, stream) if k is None else k
        v = _new(shape, want, slots.device, stream) if v is None else v
        _arg(k, want, shape, "k", slots.device)
        _arg(v, want, shape, "v", slots.device)
        _apart(v, k, "v", in_place=False)
    rc = (_lib or load()).w4a8_kv_read(cache.ref, slots.data_ptr(), T, k.data_ptr(), v.data_ptr(), code,
                                       _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "w4a8_kv_read")
    return k, v


def attention_workspace_bytes(q, cache, batch, max_q=1, max_kv=None, window=0, sinks=0, page_table=None):
    """w4a8_attention_workspace_bytes for an `attention` call with q [total, heads, head_dim] over `cache`; max_kv absent: what
    `page_table` holds, as in the call.  A smaller call may need more than a larger one: see attention_workspace_bound."""
    if max_kv is None:
        if page_table is None:
            raise ValueError("max_kv or the call's page_table is needed: the size goes by the bound on the keys")
        max_kv = page_table.shape[1] * cache.page
    a = _AttentionArgs(total=q.shape[0], batch=batch, q_heads=q.shape[1], max_q=max_q, max_kv=max_kv, window=window,
                       sinks=sinks)
    return int(load().w4a8_attention_workspace_bytes(cache.ref, ctypes.addressof(a)))


def attention_workspace_bound(cache, q_heads, batch, total, max_q=1, *, max_kv, window=0, sinks=0):
    """w4a8_attention_workspace_bound: bytes that suffice for every `attention` call over `cache` with q_heads heads, at most
    `batch` sequences, `total` rows of q, max_q queries a sequence and max_kv keys, and this window and sinks."""
    a = _AttentionArgs(total=total, batch=batch, q_heads=q_heads, max_q=max_q, max_kv=max_kv, window=window, sinks=sinks)
    return int(load().w4a8_attention_workspace_bound(cache.ref, ctypes.addressof(a)))


def attention(q, cache, page_table, kv_len, q_start=None, max_q=1, max_kv=None, window=0, sinks=0, scale=None, out=None,
              out_dtype=None, ws=None, stream=None):
    """w4a8_attention: softmax(scale q k^T) v of each sequence's newest tokens over the cache, causal, with a
    sliding `window` (0: none) beside which the first `sinks` keys stay visible.  q fp32 or bf16
    [total, heads, head_dim]; page_table int32 [batch, pages of a sequence], kv_len int32 [batch] (the
    queries' own keys included), q_start int32 [batch + 1] with at most max_q queries each, or None: row b
    is sequence b's one query.  max_kv bounds the lengths (absent: what the page table holds; where that is much more than
    the lengths, a bound saves workspace, which for prompts grows with it); scale
    head_dim^-0.5 when absent.  Returns out fp32 or bf16 [total, heads, head_dim] (bf16 when allocated here
    without an out_dtype); its rows that belong to no sequence are left as they are."""
    try:
        T, H, D = shape = q.shape
        B, width = page_table.shape
        index, (qt, qh, one), (ot, oh, other) = cache.index, q.stride(), out.stride()
        pq, po, q_code, out_code = q.data_ptr(), out.data_ptr(), _IN_DTYPES[q.dtype], _OUT_DTYPES[out.dtype]
        size = ws.numel() * ws.element_size()
        fits = one == 1 and other == 1 and D == cache.head_dim and H % cache.heads == 0 and out.shape == shape and \
            out_dtype is None and kv_len.dtype is _I32 and kv_len.shape == (B,) and page_table.dtype is _I32 and \
            page_table.is_contiguous() and kv_len.is_contiguous() and ws.is_contiguous() and \
            q.get_device() == index and out.get_device() == index and page_table.get_device() == index and \
            kv_len.get_device() == index and ws.get_device() == index and index == _current_device() and \
            (po >= pq + (4 - 2 * q_code) * ((T - 1) * qt + (H - 1) * qh + D) or
             pq >= po + (4 - 2 * out_code) * ((T - 1) * ot + (H - 1) * oh + D)) and \
            (max_q == 1 and B <= T if q_start is None else
             q_start.dtype is _I32 and q_start.shape == (B + 1,) and q_start.is_contiguous() and q_start.get_device() == index)
        pw = ws.data_ptr()
    except _NOT_FITTING:
        fits = False
    if not fits:
        _cache_arg(cache)
        index = cache.index
        qt, qh = _heads_arg(q, "q", index)
        T, H, D = q.shape
        if D != cache.head_dim or H % cache.heads:
            raise ValueError(f"q must have shape [total, a multiple of {cache.heads}, {cache.head_dim}], got {tuple(q.shape)}")
        for t, name in ((page_table, "page_table"), (kv_len, "kv_len")):
            if t is None:
                raise TypeError(f"{name} must be a torch.Tensor, got None")
        _arg(kv_len, _I32, None, "kv_len", q.device)
        B = kv_len.shape[0] if kv_len.dim() == 1 else -1
        if B < 0 or page_table.dim() != 2 or page_table.shape[0] != B:
            raise ValueError(f"kv_len must be 1-D and page_table 2-D with a row for each sequence, got shapes "
                             f"{tuple(kv_len.shape)} and {tuple(page_table.shape)}")
        _arg(page_table, _I32, None, "page_table", q.device)
        _arg(q_start, _I32, (B + 1,), "q_start", q.device)
        if q_start is None and max_q != 1:
            raise ValueError("several queries a sequence need q_start")
        if q_start is None and B > T:
            raise ValueError(f"{B} sequences of one query each, but q has {T} rows")
        if out is None:
            out = _new((T, H, D), torch.bfloat16 if out_dtype is None else out_dtype, q.device, stream)
        ot, oh = _heads_arg(out, "out", index, out_dtype, q.shape)
        _apart(out, q, "out", in_place=False)
        width = page_table.shape[1]
        if ws is None:
            need = attention_workspace_bytes(q, cache, B, max_q, width * cache.page if max_kv is None else max_kv, window, sinks)
            ws = _ws(None, need, q.device, stream)
        else:
            _arg(ws, None, None, "ws", q.device)
        pq, po, q_code, out_code = q.data_ptr(), out.data_ptr(), _IN_DTYPES[q.dtype], _OUT_DTYPES[out.dtype]
        pw, size = ws.data_ptr(), _nbytes(ws)
    a = _pack_attention(pq, po, qt, qh, ot, oh, page_table.data_ptr(), kv_len.data_ptr(),
                        0 if q_start is None else q_start.data_ptr(), width, B, T, H, max_q,
                        width * cache.page if max_kv is None else max_kv, window, sinks, q_code, out_code,
                        D ** -0.5 if scale is None else scale)
    rc = (_lib or load()).w4a8_attention(cache.ref, a, pw, size, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "w4a8_attention")
    return out


def debug_block_acc(a_q, wq, N, m0=0, m_cnt=None, n0=0, n_cnt=None, ws=None, stream=None):
    """w4a8_debug_block_acc: exact per-block int32 accumulators [m_cnt, n_cnt, K/64]."""
    _want(a_q, torch.int8, "a_q")
    M, K = a_q.shape
    _arg(wq, torch.uint8, (N, K // 2), "wq", a_q.device)
    m_cnt = M - m0 if m_cnt is None else m_cnt
    n_cnt = N - n0 if n_cnt is None else n_cnt
    if not (0 <= m0 and 0 <= m_cnt and m0 + m_cnt <= M and 0 <= n0 and 0 <= n_cnt and n0 + n_cnt <= N):
        raise ValueError(f"window rows [{m0}, {m0}+{m_cnt}) x cols [{n0}, {n0}+{n_cnt}) outside [{M}] x [{N}]")
    acc = _new((m_cnt, n_cnt, K // 64), torch.int32, a_q.device, stream)
    ws = _ws(ws, debug_workspace_bytes(m_cnt, n_cnt, K), a_q.device, stream)
    rc = load().w4a8_debug_block_acc(_ptr(a_q), _ptr(wq), M, N, K, m0, m_cnt, n0, n_cnt, _ptr(acc),
                                     _ptr(ws), _nbytes(ws), _stream(stream))
    _check(rc, "w4a8_debug_block_acc")
    return acc


def sync_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device status word."""
    return int(load().w4a8_sync_status(_stream(stream)))


def selftest_wait_timeout(limit_us: int, stream=None) -> None:
    _check(load().w4a8_selftest_wait_timeout(int(limit_us), _stream(stream)), "w4a8_selftest_wait_timeout")


class Tape:
    """A recorded call sequence (w4a8_tape_*): `with Tape(stream) as t:` records the library
    calls made on `stream` inside the block; `t.replay(stream)` runs them again with one
    launch.  The tensors given to the recorded calls must stay alive while the tape is; outputs and
    workspaces that the calls allocated for themselves the tape holds.  (Device memory cannot be
    requested while a stream is recorded: such calls are made once before, so that the allocator has
    their blocks at hand.)"""

    def __init__(self, stream):
        self.stream = stream
        self.handle = None
        self.recorded, self.keep = None, []

    def __enter__(self):
        _check(load().w4a8_tape_begin(_stream(self.stream)), "w4a8_tape_begin")
        self.recorded = _stream(self.stream).value
        _recording.append(self)
        return self

    def __exit__(self, exc_type, exc, tb):
        _recording.remove(self)
        h = _P()
        rc = load().w4a8_tape_end(_stream(self.stream), ctypes.byref(h))
        if exc_type is None:
            _check(rc, "w4a8_tape_end")
            self.handle = h
        elif rc == 0 and h:
            load().w4a8_tape_free(h)
        return False

    def replay(self, stream=None):
        if self.handle is None:
            raise RuntimeError("tape not recorded")
        if self.keep:
            used = torch.cuda.current_stream() if stream is None else stream
            for t in self.keep:
                t.record_stream(used)
        _check(load().w4a8_tape_replay(self.handle, _stream(stream)), "w4a8_tape_replay")

    def kernels(self) -> int:
        """Kernel launches per replay (w4a8_tape_kernels)."""
        if self.handle is None:
            raise RuntimeError("tape not recorded")
        return int(load().w4a8_tape_kernels(self.handle))

    def free(self):
        if self.handle is not None:
            load().w4a8_tape_free(self.handle)
            self.handle = None
        self.keep.clear()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

