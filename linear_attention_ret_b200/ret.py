"""Thin Python binding of libret.so, the C ABI declared in include/ret.h.

Argument marshalling only: shape and dtype checks, output allocation with
torch (device memory is plumbing), and the call through ctypes. Every step of
retention runs in the library's CUDA kernels; there is no fallback. If the
library is missing, load() raises.

Names match the C ABI: ret_parallel, ret_chunkwise, ret_recurrent_step,
gated_ret_chunkwise. Tensors are CUDA, contiguous, heads leading:
q, k [B, H, N, dk]; v [B, H, N, dv]; gamma [H] fp32; g [B, H, N] fp32;
state [B, H, dk, dv] fp32. q, k, v share one dtype (float32 or bfloat16).
A call on device tensors is made on their device, whichever is current.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libret.so")

RET_F32, RET_BF16 = 0, 1
STATUS = {0: "RET_OK", 1: "RET_ERR_NULL", 2: "RET_ERR_SHAPE", 3: "RET_ERR_DTYPE", 4: "RET_ERR_UNSUPPORTED",
          5: "RET_ERR_CUDA", 6: "RET_ERR_TIMEOUT", 7: "RET_ERR_ALIGN", 8: "RET_ERR_SCRATCH"}
# every symbol include/ret.h declares
SYMBOLS = ("ret_parallel", "ret_chunkwise", "ret_recurrent_step", "gated_ret_chunkwise", "ret_status_str",
           "ret_last_device_error", "ret_chunkwise_path", "ret_chunkwise_launches", "ret_version",
           "ret_chunkwise_noalloc", "ret_selftest_wait_timeout", "gated_ret_recurrent_step",
           "ret_chunkwise_state", "gated_ret_chunkwise_state", "ret_state_prefix", "ret_chunkwise_state_launches",
           "ret_chunkwise_backward", "gated_ret_chunkwise_backward", "ret_chunkwise_backward_launches",
           "ret_msr_norm_gate", "ret_chunkwise_noalloc_scratch_bytes", "ret_chunkwise_host",
           "gated_ret_chunkwise_host", "ret_chunkwise_backward_host", "gated_ret_chunkwise_backward_host",
           "ret_msr_norm_gate_backward", "ret_rotary", "ret_layer_norm", "ret_layer_norm_backward")

_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_ll = ctypes.c_longlong
_f = ctypes.c_float


class RetError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn}: {STATUS.get(code, code)} ({msg})")
        self.code = code


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libret.so (built in-tree by linear_attention_ret_b200.build)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libret.so not found at {p}: build it with "
                               "`python -m linear_attention_ret_b200.build`")
        lib = ctypes.CDLL(p)
        lib.ret_parallel.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]
        lib.ret_chunkwise.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]
        lib.gated_ret_chunkwise.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]
        lib.ret_chunkwise_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]
        lib.ret_recurrent_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]
        lib.gated_ret_recurrent_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]
        lib.ret_chunkwise_state.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]
        lib.gated_ret_chunkwise_state.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]
        lib.ret_state_prefix.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]
        lib.ret_chunkwise_state_launches.argtypes = [_i, _i, _i, _i, _i, _i, _i]
        lib.ret_chunkwise_backward_launches.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i, _i]
        for fn in ("ret_chunkwise_host", "gated_ret_chunkwise_host"):
            getattr(lib, fn).argtypes = [_vp] * 5 + [_i] * 7 + [_vp]
            getattr(lib, fn).restype = _i
        lib.ret_msr_norm_gate.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, ctypes.c_float, _i, _vp]
        lib.ret_msr_norm_gate.restype = _i
        lib.ret_msr_norm_gate_backward.argtypes = [_vp] * 5 + [_i] * 4 + [_f, _i, _vp]
        lib.ret_rotary.argtypes = [_vp] * 11 + [_ll] + [_i] * 8 + [_f] * 3 + [_i, _vp]
        lib.ret_layer_norm.argtypes = [_vp] * 8 + [_ll, _i, _f, _i, _i, _vp]
        lib.ret_layer_norm_backward.argtypes = [_vp] * 9 + [_ll, _i, _i, _i, _vp]
        for fn in ("ret_msr_norm_gate_backward", "ret_rotary", "ret_layer_norm", "ret_layer_norm_backward"):
            getattr(lib, fn).restype = _i
        for fn in ("ret_chunkwise_backward", "gated_ret_chunkwise_backward", "ret_chunkwise_backward_host",
                   "gated_ret_chunkwise_backward_host"):
            getattr(lib, fn).argtypes = [_vp] * 9 + [_i] * 7 + [_vp]
            getattr(lib, fn).restype = _i
        lib.ret_chunkwise_state_launches.restype = _i
        for fn in ("ret_parallel", "ret_chunkwise", "gated_ret_chunkwise", "ret_recurrent_step",
                   "ret_chunkwise_noalloc", "gated_ret_recurrent_step", "ret_chunkwise_state",
                   "gated_ret_chunkwise_state", "ret_state_prefix"):
            getattr(lib, fn).restype = _i
        lib.ret_status_str.argtypes = [_i]
        lib.ret_status_str.restype = ctypes.c_char_p
        lib.ret_last_device_error.argtypes = [_vp]
        lib.ret_last_device_error.restype = _i
        lib.ret_selftest_wait_timeout.argtypes = [ctypes.c_uint, _vp]
        lib.ret_selftest_wait_timeout.restype = _i
        lib.ret_chunkwise_path.argtypes = [_i, _i, _i, _i]
        lib.ret_chunkwise_path.restype = _i
        lib.ret_chunkwise_launches.argtypes = [_i, _i, _i, _i, _i, _i, _i]
        lib.ret_chunkwise_launches.restype = _i
        lib.ret_chunkwise_noalloc_scratch_bytes.argtypes = [_i] * 8
        lib.ret_chunkwise_noalloc_scratch_bytes.restype = ctypes.c_longlong
        lib.ret_version.argtypes = []
        lib.ret_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(fn: str, code: int):
    if code != 0:
        raise RetError(fn, code, load().ret_status_str(code).decode())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return RET_F32
    if t.dtype == torch.bfloat16:
        return RET_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _cuda(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors must be on one device, got {dev} and {t.device}")


def _on_device_of_tensors(fn):
    """A call whose first argument is a device tensor, made with that tensor's device current: the library launches
    on the current device, where another device's addresses are not valid."""
    @functools.wraps(fn)
    def call(*args, **kwargs):
        t = args[0] if args else next(iter(kwargs.values()), None)
        index = t.get_device() if hasattr(t, "get_device") else -1
        if index >= 0 and index != torch.cuda.current_device():
            with torch.cuda.device(index):
                return fn(*args, **kwargs)
        return fn(*args, **kwargs)
    return call


def _host(*ts):
    for t in ts:
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous host (CPU) tensors")


def _expect(name, t, shape, dtype=None):
    """Shape (and dtype) every tensor must have given the leading one, checked before any
    pointer reaches the library: a wrong size there would read past an allocation."""
    if t is None:
        return
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _rank(name, t, n):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(t.shape)}")


def _seq_args(q, k, v, decay, gated, o=None, state_in=None, state_out=None):
    """q, k [B, H, N, dk]; v, o [B, H, N, dv] (q's dtype); gamma [H] or g [B, H, N] fp32;
    states [B, H, dk, dv] fp32. Returns (B, H, N, dk, dv)."""
    _rank("q", q, 4)
    _rank("v", v, 4)
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    _expect("k", k, (B, H, N, dk), q.dtype)
    _expect("v", v, (B, H, N, dv), q.dtype)
    _expect("g" if gated else "gamma", decay, (B, H, N) if gated else (H,), torch.float32)
    _expect("o", o, (B, H, N, dv), q.dtype)
    _expect("state_in", state_in, (B, H, dk, dv), torch.float32)
    _expect("state_out", state_out, (B, H, dk, dv), torch.float32)
    return B, H, N, dk, dv


def _step_args(q, k, v, decay, state, o, gated):
    """q, k [B, H, dk]; v, o [B, H, dv]; gamma [H] or g [B, H] fp32; state [B, H, dk, dv] fp32."""
    _rank("q", q, 3)
    _rank("v", v, 3)
    B, H, dk = q.shape
    dv = v.shape[-1]
    _expect("k", k, (B, H, dk), q.dtype)
    _expect("v", v, (B, H, dv), q.dtype)
    _expect("g" if gated else "gamma", decay, (B, H) if gated else (H,), torch.float32)
    _expect("state", state, (B, H, dk, dv), torch.float32)
    _expect("o", o, (B, H, dv), q.dtype)
    return B, H, dk, dv


@_on_device_of_tensors
def ret_parallel(q, k, v, gamma, o=None, stream=None):
    """O = (Q K^T (.) D) V. Returns o [B, H, N, dv] (dtype of q)."""
    B, H, N, dk, dv = _seq_args(q, k, v, gamma, False, o)
    o = torch.empty(B, H, N, dv, dtype=q.dtype, device=q.device) if o is None else o
    _cuda(q, k, v, gamma, o)
    _check("ret_parallel", load().ret_parallel(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(o),
                                               B, H, N, dk, dv, _dt(q), _stream(stream)))
    return o


@_on_device_of_tensors
def ret_chunkwise(q, k, v, gamma, chunk, state_in=None, state_out=None, o=None, stream=None):
    """Chunkwise retention. Returns o; writes the final state into state_out if given."""
    B, H, N, dk, dv = _seq_args(q, k, v, gamma, False, o, state_in, state_out)
    o = torch.empty(B, H, N, dv, dtype=q.dtype, device=q.device) if o is None else o
    _cuda(q, k, v, gamma, o, state_in, state_out)
    _check("ret_chunkwise", load().ret_chunkwise(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(o),
                                                 _ptr(state_in), _ptr(state_out), B, H, N, dk, dv, int(chunk),
                                                 _dt(q), _stream(stream)))
    return o


@_on_device_of_tensors
def ret_chunkwise_noalloc(q, k, v, gamma, chunk, state_in=None, state_out=None, o=None, stream=None):
    """ret_chunkwise without device allocation by the library: scratch comes from a
    fixed 16 MiB buffer inside libret.so (see include/ret.h). Returns o."""
    B, H, N, dk, dv = _seq_args(q, k, v, gamma, False, o, state_in, state_out)
    o = torch.empty(B, H, N, dv, dtype=q.dtype, device=q.device) if o is None else o
    _cuda(q, k, v, gamma, o, state_in, state_out)
    _check("ret_chunkwise_noalloc", load().ret_chunkwise_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(o),
                                                                 _ptr(state_in), _ptr(state_out), B, H, N, dk, dv,
                                                                 int(chunk), _dt(q), _stream(stream)))
    return o


@_on_device_of_tensors
def gated_ret_chunkwise(q, k, v, g, chunk, state_in=None, state_out=None, o=None, stream=None):
    """Gated chunkwise retention (per-token log-decay g). Returns o."""
    B, H, N, dk, dv = _seq_args(q, k, v, g, True, o, state_in, state_out)
    o = torch.empty(B, H, N, dv, dtype=q.dtype, device=q.device) if o is None else o
    _cuda(q, k, v, g, o, state_in, state_out)
    _check("gated_ret_chunkwise", load().gated_ret_chunkwise(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o),
                                                             _ptr(state_in), _ptr(state_out), B, H, N, dk, dv,
                                                             int(chunk), _dt(q), _stream(stream)))
    return o


def _chunkwise_host(name, q, k, v, decay, chunk, o, gated, stream, sync):
    B, H, N, dk, dv = _seq_args(q, k, v, decay, gated, o)
    if o is None:
        o = torch.empty(B, H, N, dv, dtype=q.dtype, pin_memory=q.is_pinned())
    _host(q, k, v, decay, o)
    s = torch.cuda.current_stream() if stream is None else stream
    _check(name, getattr(load(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(o), B, H, N, dk, dv,
                                       int(chunk), _dt(q), ctypes.c_void_p(s.cuda_stream)))
    if sync:
        s.synchronize()
    return o


def ret_chunkwise_host(q, k, v, gamma, chunk, o=None, stream=None, sync=True):
    """ret_chunkwise on host (CPU) tensors, pinned for copy/compute overlap: the library copies
    the inputs in, computes and copies o back, pipelined over groups of heads, on the current
    CUDA device. Returns o once the stream has completed (sync=False: once enqueued)."""
    return _chunkwise_host("ret_chunkwise_host", q, k, v, gamma, chunk, o, False, stream, sync)


def gated_ret_chunkwise_host(q, k, v, g, chunk, o=None, stream=None, sync=True):
    """gated_ret_chunkwise on host (CPU) tensors; as ret_chunkwise_host."""
    return _chunkwise_host("gated_ret_chunkwise_host", q, k, v, g, chunk, o, True, stream, sync)


@_on_device_of_tensors
def ret_recurrent_step(q, k, v, gamma, state, o=None, stream=None):
    """One decode step; updates state [B, H, dk, dv] in place and returns o [B, H, dv]."""
    B, H, dk, dv = _step_args(q, k, v, gamma, state, o, False)
    o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device) if o is None else o
    _cuda(q, k, v, gamma, state, o)
    _check("ret_recurrent_step", load().ret_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(state),
                                                           _ptr(o), B, H, dk, dv, _dt(q), _stream(stream)))
    return o


@_on_device_of_tensors
def gated_ret_recurrent_step(q, k, v, g, state, o=None, stream=None):
    """One gated decode step with log-decay g [B, H] (fp32); updates state in place, returns o [B, H, dv]."""
    B, H, dk, dv = _step_args(q, k, v, g, state, o, True)
    o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device) if o is None else o
    _cuda(q, k, v, g, state, o)
    _check("gated_ret_recurrent_step", load().gated_ret_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                                                       _ptr(state), _ptr(o), B, H, dk, dv, _dt(q),
                                                                       _stream(stream)))
    return o


@_on_device_of_tensors
def chunkwise_state(k, v, decay, chunk, gated=False, state_out=None, log2_decay=None, stream=None):
    """End state U [B, H, dk, dv] of a segment from a zero start and log2 of its total decay
    [B, H] (decay: gamma [H], or g [B, H, N] with gated=True). Returns (U, log2_decay)."""
    B, H, N, dk, dv = _seq_args(k, k, v, decay, gated, None, None, state_out)
    _expect("log2_decay", log2_decay, (B, H), torch.float32)
    state_out = torch.empty(B, H, dk, dv, dtype=torch.float32, device=k.device) if state_out is None else state_out
    log2_decay = torch.empty(B, H, dtype=torch.float32, device=k.device) if log2_decay is None else log2_decay
    _cuda(k, v, decay, state_out, log2_decay)
    name = "gated_ret_chunkwise_state" if gated else "ret_chunkwise_state"
    _check(name, getattr(load(), name)(_ptr(k), _ptr(v), _ptr(decay), _ptr(state_out), _ptr(log2_decay),
                                       B, H, N, dk, dv, int(chunk), _dt(k), _stream(stream)))
    return state_out, log2_decay


@_on_device_of_tensors
def state_prefix(seg_states, seg_log2_decay, state_in=None, stream=None):
    """Start states [R, B, H, dk, dv] of R consecutive segments and the state after all of
    them, from their end states U [R, B, H, dk, dv] and log2 decays [R, B, H]."""
    _rank("seg_states", seg_states, 5)
    R, B, H, dk, dv = seg_states.shape
    _expect("seg_states", seg_states, (R, B, H, dk, dv), torch.float32)
    _expect("seg_log2_decay", seg_log2_decay, (R, B, H), torch.float32)
    _expect("state_in", state_in, (B, H, dk, dv), torch.float32)
    starts = torch.empty_like(seg_states)
    end = torch.empty(B, H, dk, dv, dtype=torch.float32, device=seg_states.device)
    _cuda(seg_states, seg_log2_decay, state_in, starts, end)
    _check("ret_state_prefix", load().ret_state_prefix(_ptr(seg_states), _ptr(seg_log2_decay), _ptr(state_in),
                                                       _ptr(starts), _ptr(end), R, B, H, dk, dv, _stream(stream)))
    return starts, end


@_on_device_of_tensors
def chunkwise_backward(q, k, v, decay, dout, chunk, gated=False, ddecay=True, stream=None):
    """Gradients of sum(dout * o) for o = ret_chunkwise(q, k, v, decay) (gated=True:
    gated_ret_chunkwise with g = decay) from a zero initial state. Returns
    (dq, dk, dv, ddecay) with ddecay = dgamma [H] or dg [B, H, N] (fp32), or None."""
    B, H, N, dk, dv = _seq_args(q, k, v, decay, gated)
    _expect("dout", dout, (B, H, N, dv), q.dtype)
    dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dd = None
    if ddecay:
        dd = torch.empty(B, H, N, dtype=torch.float32, device=q.device) if gated else \
            torch.empty(H, dtype=torch.float32, device=q.device)
    _cuda(q, k, v, decay, dout, dq, dkk, dvv, dd)
    name = "gated_ret_chunkwise_backward" if gated else "ret_chunkwise_backward"
    _check(name, getattr(load(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(dout), _ptr(dq), _ptr(dkk),
                                       _ptr(dvv), _ptr(dd), B, H, N, dk, dv, int(chunk), _dt(q), _stream(stream)))
    return dq, dkk, dvv, dd


def chunkwise_backward_host(q, k, v, decay, dout, chunk, gated=False, ddecay=True, out=None, stream=None, sync=True):
    """chunkwise_backward on host (CPU) tensors, pinned for copy/compute overlap: the library
    copies the inputs in and the gradients out, pipelined over groups of heads, on the current
    CUDA device. out: optional (dq, dk, dv, ddecay) host tensors to write. Returns them once the
    stream has completed (sync=False: once enqueued)."""
    B, H, N, dk, dv = _seq_args(q, k, v, decay, gated)
    _expect("dout", dout, (B, H, N, dv), q.dtype)
    pin = q.is_pinned()
    if out is None:
        dd = None
        if ddecay:
            dd = torch.empty((B, H, N) if gated else (H,), dtype=torch.float32, pin_memory=pin)
        out = (torch.empty(B, H, N, dk, dtype=q.dtype, pin_memory=pin),
               torch.empty(B, H, N, dk, dtype=q.dtype, pin_memory=pin),
               torch.empty(B, H, N, dv, dtype=q.dtype, pin_memory=pin), dd)
    dq, dkk, dvv, dd = out
    _expect("dq", dq, (B, H, N, dk), q.dtype)
    _expect("dk", dkk, (B, H, N, dk), q.dtype)
    _expect("dv", dvv, (B, H, N, dv), q.dtype)
    _expect("ddecay", dd, (B, H, N) if gated else (H,), torch.float32)
    _host(*(t for t in (q, k, v, decay, dout, dq, dkk, dvv, dd) if t is not None))
    s = torch.cuda.current_stream() if stream is None else stream
    name = "gated_ret_chunkwise_backward_host" if gated else "ret_chunkwise_backward_host"
    _check(name, getattr(load(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(dout), _ptr(dq), _ptr(dkk),
                                       _ptr(dvv), _ptr(dd), B, H, N, dk, dv, int(chunk), _dt(q),
                                       ctypes.c_void_p(s.cuda_stream)))
    if sync:
        s.synchronize()
    return dq, dkk, dvv, dd


@_on_device_of_tensors
def msr_norm_gate(o, gate, eps: float = 1e-5, y=None, stream=None):
    """Multi-scale retention output epilogue: y[b, n, h] = swish(gate[b, n, h]) * RMSNorm(o[b, h, n])
    over dv (no affine weights). o [B, H, N, dv]; gate [B, N, H, dv] (same dtype);
    returns y [B, N, H, dv] (may be `gate` itself for an in-place update)."""
    _rank("o", o, 4)
    B, H, N, dv = o.shape
    if tuple(gate.shape) != (B, N, H, dv):
        raise ValueError(f"gate must be [B, N, H, dv] = {(B, N, H, dv)}, got {tuple(gate.shape)}")
    if y is None:
        y = torch.empty_like(gate)
    if gate.dtype != o.dtype or y.dtype != o.dtype or tuple(y.shape) != tuple(gate.shape):
        raise ValueError("o, gate and y must share one dtype; y has gate's shape")
    _cuda(o, gate, y)
    _check("ret_msr_norm_gate", load().ret_msr_norm_gate(_ptr(o), _ptr(gate), _ptr(y), B, H, N, dv, float(eps), _dt(o),
                                                         _stream(stream)))
    return y


# The calls below are made once per layer and token, so their host time counts: tensors are read
# once, addresses go to ctypes as integers, what is absent is not looked at, and a device or stream
# is entered only when it is not the current one.

_DTYPES = {torch.float32: RET_F32, torch.bfloat16: RET_BF16}


def _elsewhere(device, stream):
    """None when a call may go straight to the current stream of the current device; else the context in
    which it may (stream given, or the tensors' device not current). Outputs are allocated there too."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, tensors are on {device}")
        return torch.cuda.stream(stream)
    return None if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _current_stream(device) -> int:
    # the handle alone: torch.cuda.current_stream builds a Stream object around it (2 us)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _address(t):
    return None if t is None else t.data_ptr()


def msr_norm_gate_backward(dy, o, gate, eps: float = 1e-5, dout=None, dgate=None, stream=None):
    """Gradients of sum(dy * msr_norm_gate(o, gate, eps)). dy, gate [B, N, H, dv]; o [B, H, N, dv].
    Returns (dout [B, H, N, dv], dgate [B, N, H, dv]); dout may be o, dgate may be gate or dy."""
    shape, dtype, device = o.shape, o.dtype, o.device
    if len(shape) != 4:
        _rank("o", o, 4)
    B, H, N, dv = shape
    token_major = (B, N, H, dv)
    _expect("gate", gate, token_major, dtype)
    _expect("dy", dy, token_major, dtype)
    if dout is not None:
        _expect("dout", dout, shape, dtype)
    if dgate is not None:
        _expect("dgate", dgate, token_major, dtype)
    dt = _DTYPES.get(dtype)
    if dt is None:
        _dt(o)
    _cuda(o, gate, dy, dout, dgate)
    away = _elsewhere(device, stream)
    if away is not None:
        with away:
            return msr_norm_gate_backward(dy, o, gate, eps, dout, dgate)
    if dout is None:
        dout = torch.empty_like(o)
    if dgate is None:
        dgate = torch.empty_like(gate)
    _check("ret_msr_norm_gate_backward",
           (_lib or load()).ret_msr_norm_gate_backward(dy.data_ptr(), o.data_ptr(), gate.data_ptr(), dout.data_ptr(),
                                                       dgate.data_ptr(), B, H, N, dv, float(eps), dt,
                                                       _current_stream(device)))
    return dout, dgate


ROTARY_LAYOUTS = {"interleaved": 0, "half": 1}  # ret_rotary_layout in include/ret.h
_Strides = _ll * 12  # batch, token and head strides of q, k, q_out and k_out
_NO_STRIDES = (0, 0, 0, 0)


def _view(name, t, shape, dtype, device):
    """Checks one tensor of a rotary call; returns its strides and whether it is on the device."""
    if t.shape != shape or t.dtype != dtype:
        _expect(name, t, shape, dtype)
    strides = t.stride()
    if strides[3] != 1 and shape[3] > 1:
        raise ValueError(f"the head dimension of {name} must be contiguous")
    return strides, t.device == device


def _rotate(q, k, q_out, k_out, freqs, positions, starts, offset, layout, inverse, amplitude, q_scale, k_scale,
            stream):
    """One ret_rotary call. Token-major [B, N, H, d] in and head-major [B, H, N, d] out, or with
    inverse the other way round. Outputs that are None are allocated contiguous."""
    shape, dtype, device = q.shape, q.dtype, q.device
    if len(shape) != 4:
        _rank("q", q, 4)
    if inverse:
        B, Hq, N, d = shape
        q_shape = (B, N, Hq, d)
    else:
        B, N, Hq, d = shape
        q_shape = (B, Hq, N, d)
    here = q.is_cuda
    sq = q.stride()
    if sq[3] != 1 and d > 1:
        raise ValueError("the head dimension of q must be contiguous")
    Hk, sk, sko = 0, _NO_STRIDES, _NO_STRIDES
    if k is not None:
        if k.dim() != 4:
            _rank("k", k, 4)
        if inverse:
            Hk = k.shape[1]
            k_in, k_shape = (B, Hk, N, d), (B, N, Hk, d)
        else:
            Hk = k.shape[2]
            k_in, k_shape = (B, N, Hk, d), (B, Hk, N, d)
        sk, there = _view("k", k, k_in, dtype, device)
        here = here and there
    elif k_out is not None:
        raise ValueError("an output for k was given without k")
    rot = 0
    if freqs is not None:
        if freqs.dim() != 1:
            _rank("freqs", freqs, 1)
        if freqs.dtype != torch.float64:
            raise ValueError(f"freqs must be {torch.float64}, got {freqs.dtype}")
        rot = 2 * freqs.shape[0]
        if rot > d:
            raise ValueError(f"freqs rotates {rot} elements of a head of {d}")
        here = here and freqs.device == device and freqs.is_contiguous()
    if positions is not None:
        if starts is not None:
            raise ValueError("give positions or starts, not both")
        _expect("positions", positions, (B, N), torch.int64)
        here = here and positions.device == device and positions.is_contiguous()
    elif starts is not None:
        _expect("starts", starts, (B,), torch.int64)
        here = here and starts.device == device and starts.is_contiguous()
    order = ROTARY_LAYOUTS.get(layout)
    if order is None:
        raise ValueError(f"layout must be one of {tuple(ROTARY_LAYOUTS)}, got {layout!r}")
    dt = _DTYPES.get(dtype)
    if dt is None:
        _dt(q)
    if q_out is not None:
        sqo, there = _view("the output of q", q_out, q_shape, dtype, device)
        here = here and there
    if k_out is not None:
        sko, there = _view("the output of k", k_out, k_shape, dtype, device)
        here = here and there
    if not here:
        raise ValueError(f"tensors must be CUDA tensors on one device (q is on {device}), and the tables contiguous")
    away = _elsewhere(device, stream)
    if away is not None:
        with away:
            return _rotate(q, k, q_out, k_out, freqs, positions, starts, offset, layout, inverse, amplitude, q_scale,
                           k_scale, None)
    if q_out is None:
        q_out = q.new_empty(q_shape)
        sqo = q_out.stride()
    if k is not None and k_out is None:
        k_out = k.new_empty(k_shape)
        sko = k_out.stride()
    n, h = (2, 1) if inverse else (1, 2)  # token and head dimension of the inputs; the outputs have them swapped
    strides = _Strides(sq[0], sq[n], sq[h], sk[0], sk[n], sk[h], sqo[0], sqo[h], sqo[n], sko[0], sko[h], sko[n])
    at = ctypes.addressof(strides)
    _check("ret_rotary",
           (_lib or load()).ret_rotary(q.data_ptr(), None if k is None else k.data_ptr(), q_out.data_ptr(),
                                       None if k is None else k_out.data_ptr(), at, at + 24, at + 48, at + 72,
                                       None if freqs is None else freqs.data_ptr(), _address(positions),
                                       _address(starts), int(offset), B, N, Hq, Hk, d, rot, order, inverse,
                                       float(amplitude), float(q_scale), float(k_scale), dt, _current_stream(device)))
    return q_out, k_out


def rotary(q, k, freqs, positions=None, starts=None, offset=0, layout="interleaved", amplitude=1.0, q_scale=1.0,
           k_scale=1.0, q_out=None, k_out=None, stream=None):
    """Rotary prologue: q [B, N, Hq, d] and k [B, N, Hk, d] (or None) as the projections give them,
    rotated by their positions and laid out head-major for the retention calls. Returns
    (q_out [B, Hq, N, d], k_out [B, Hk, N, d] or None).

    q and k may be any strided views whose head dimension is contiguous (slices of a fused
    projection), q_out and k_out too; an output may be its own input (q_out=q.transpose(1, 2)).
    freqs [rot / 2] fp64 is radians per position of each pair (rotary.frequencies makes it), None
    for a call that only lays out and scales. The position of token n is offset + positions[b, n],
    or offset + n (+ starts[b]); positions [B, N] and starts [B] are int64. layout: "interleaved"
    pairs (2i, 2i+1) or "half" pairs (i, i + rot/2). The rotated part is multiplied by amplitude,
    the whole head by q_scale or k_scale."""
    return _rotate(q, k, q_out, k_out, freqs, positions, starts, offset, layout, False, amplitude, q_scale, k_scale,
                   stream)


def rotary_backward(dq, dk, freqs, positions=None, starts=None, offset=0, layout="interleaved", amplitude=1.0,
                    q_scale=1.0, k_scale=1.0, dq_out=None, dk_out=None, stream=None):
    """Gradient of rotary: dq [B, Hq, N, d] and dk [B, Hk, N, d] (or None), as the retention backward
    gives them, to token-major (dq_out [B, N, Hq, d], dk_out [B, N, Hk, d] or None). Arguments as
    rotary; with amplitude and scales 1 it is also its inverse."""
    return _rotate(dq, dk, dq_out, dk_out, freqs, positions, starts, offset, layout, True, amplitude, q_scale, k_scale,
                   stream)


def _norm_args(x, weight, bias):
    """x [..., D]; weight and bias [D] of x's dtype or fp32, each or both None. Returns (shape, D, dtype,
    weight dtype)."""
    shape, dtype = x.shape, x.dtype
    if not shape:
        raise ValueError("x must have at least one dimension")
    D = shape[-1]
    if D == 0:
        raise ValueError(f"x must have rows of at least one element, got shape {tuple(shape)}")
    wdtype = None
    if weight is not None:
        wdtype = weight.dtype
        if weight.shape != (D,):
            _expect("weight", weight, (D,))
    if bias is not None:
        if bias.shape != (D,):
            _expect("bias", bias, (D,))
        if wdtype is None:
            wdtype = bias.dtype
        elif bias.dtype != wdtype:
            raise ValueError(f"weight and bias must share one dtype, got {wdtype} and {bias.dtype}")
    if wdtype is None:
        wdtype = dtype
    elif wdtype != torch.float32 and wdtype != dtype:
        raise ValueError(f"weight and bias must be {dtype} or torch.float32, got {wdtype}")
    return shape, D, dtype, wdtype


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, residual=None, y=None, sum_out=None, mean=None,
               rstd=None, stream=None):
    """Layer norm over the last dimension of x [..., D], with weight and bias [D] (x's dtype or fp32, or
    None). Returns y. With a residual (x's shape and dtype) it normalises x + residual and returns
    (y, sum_out). mean and rstd (fp32, x's shape without D) receive the row statistics for
    layer_norm_backward if given. y and sum_out may each be the x or the residual tensor."""
    shape, D, dtype, wdtype = _norm_args(x, weight, bias)
    if residual is not None:
        _expect("residual", residual, shape, dtype)
    elif sum_out is not None:
        raise ValueError("sum_out was given without a residual")
    if y is not None:
        _expect("y", y, shape, dtype)
    if sum_out is not None:
        _expect("sum_out", sum_out, shape, dtype)
    if mean is not None:
        _expect("mean", mean, shape[:-1], torch.float32)
    if rstd is not None:
        _expect("rstd", rstd, shape[:-1], torch.float32)
    dt = _DTYPES.get(dtype)
    if dt is None:
        _dt(x)
    _cuda(x, weight, bias, residual, y, sum_out, mean, rstd)
    device = x.device
    away = _elsewhere(device, stream)
    if away is not None:
        with away:
            return layer_norm(x, weight, bias, eps, residual, y, sum_out, mean, rstd)
    if y is None:
        y = torch.empty_like(x)
    if residual is not None and sum_out is None:
        sum_out = torch.empty_like(x)
    _check("ret_layer_norm",
           (_lib or load()).ret_layer_norm(x.data_ptr(), _address(residual), _address(weight), _address(bias),
                                           y.data_ptr(), _address(sum_out), _address(mean), _address(rstd),
                                           x.numel() // D, D, float(eps), dt, _DTYPES[wdtype], _current_stream(device)))
    return y if residual is None else (y, sum_out)


def layer_norm_backward(dy, x, weight, mean, rstd, dsum=None, dweight=True, dbias=True, wdtype=None, dx=None,
                        stream=None):
    """Gradients of layer_norm from its statistics. x is the tensor that was normalised (with a residual,
    the forward's sum_out); dsum (x's shape) the gradient that reaches that sum by other ways, added to
    dx. Returns (dx, dweight, dbias), dweight None without a weight or with dweight=False, dbias None
    without dbias. dx may be the dy, x or dsum tensor. The dtype of dbias is the weight's, or wdtype
    (x's) where there is no weight."""
    shape, D, dtype, wd = _norm_args(x, weight, None)
    if weight is None and wdtype is not None:
        if wdtype != dtype and wdtype != torch.float32:
            raise ValueError(f"wdtype must be {dtype} or torch.float32, got {wdtype}")
        wd = wdtype
    _expect("dy", dy, shape, dtype)
    if dsum is not None:
        _expect("dsum", dsum, shape, dtype)
    if dx is not None:
        _expect("dx", dx, shape, dtype)
    _expect("mean", mean, shape[:-1], torch.float32)
    _expect("rstd", rstd, shape[:-1], torch.float32)
    dt = _DTYPES.get(dtype)
    if dt is None:
        _dt(x)
    _cuda(dy, x, weight, mean, rstd, dsum, dx)
    device = x.device
    away = _elsewhere(device, stream)
    if away is not None:
        with away:
            return layer_norm_backward(dy, x, weight, mean, rstd, dsum, dweight, dbias, wdtype, dx)
    if dx is None:
        dx = torch.empty_like(x)
    dw = torch.empty_like(weight) if dweight and weight is not None else None
    if not dbias:
        db = None
    elif weight is not None:
        db = torch.empty_like(weight)
    else:
        db = x.new_empty(D, dtype=wd)
    _check("ret_layer_norm_backward",
           (_lib or load()).ret_layer_norm_backward(dy.data_ptr(), x.data_ptr(), _address(weight), mean.data_ptr(),
                                                    rstd.data_ptr(), _address(dsum), dx.data_ptr(), _address(dw),
                                                    _address(db), x.numel() // D, D, dt, _DTYPES[wd],
                                                    _current_stream(device)))
    return dx, dw, db


def last_device_error(stream=None) -> int:
    return int(load().ret_last_device_error(_stream(stream)))


def selftest_wait_timeout(limit_us: int, stream=None) -> int:
    """Launch the failure-path self-test (a bounded wait that runs out); returns the launch status."""
    return int(load().ret_selftest_wait_timeout(limit_us, _stream(stream)))


def chunkwise_launches(B: int, H: int, N: int, dk: int, dv: int, chunk: int, dtype: torch.dtype) -> int:
    return int(load().ret_chunkwise_launches(B, H, N, dk, dv, chunk, RET_BF16 if dtype == torch.bfloat16 else RET_F32))


def chunkwise_state_launches(B: int, H: int, N: int, dk: int, dv: int, chunk: int, dtype: torch.dtype) -> int:
    return int(load().ret_chunkwise_state_launches(B, H, N, dk, dv, chunk,
                                                   RET_BF16 if dtype == torch.bfloat16 else RET_F32))


def chunkwise_backward_launches(B: int, H: int, N: int, dk: int, dv: int, chunk: int, dtype: torch.dtype,
                                gated: bool = False, ddecay: bool = True) -> int:
    return int(load().ret_chunkwise_backward_launches(B, H, N, dk, dv, chunk,
                                                      RET_BF16 if dtype == torch.bfloat16 else RET_F32,
                                                      int(gated), int(ddecay)))


def chunkwise_path(dk: int, dv: int, chunk: int, dtype: torch.dtype) -> int:
    return int(load().ret_chunkwise_path(dk, dv, chunk, RET_BF16 if dtype == torch.bfloat16 else RET_F32))


def noalloc_scratch_bytes(B: int, H: int, N: int, dk: int, dv: int, chunk: int, dtype: torch.dtype,
                          in_place: bool = False) -> int:
    """Bytes of the fixed buffer ret_chunkwise_noalloc would use on the current device (0: none,
    -1: invalid sizes); above NOALLOC_SCRATCH_BYTES the call is rejected with RET_ERR_SCRATCH."""
    return int(load().ret_chunkwise_noalloc_scratch_bytes(B, H, N, dk, dv, chunk,
                                                          RET_BF16 if dtype == torch.bfloat16 else RET_F32,
                                                          int(in_place)))


NOALLOC_SCRATCH_BYTES = 16 << 20  # RET_NOALLOC_SCRATCH_BYTES in include/ret.h
