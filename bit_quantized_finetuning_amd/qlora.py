"""Thin Python binding over libqlora.so (ctypes).

Argument marshalling only: every step of the layer runs in the HIP library.
PyTorch supplies device memory and the current HIP stream; the library itself
allocates nothing. If the library is missing this module raises at import --
there is no fallback path. (_marshal.so, the same marshalling in C++ for the
calls made most often, may be missing: those calls then take longer on the host.)

Function names follow the C ABI in include/qlora.h:
    qlora_quantize, qlora_dequantize, qlora_merge, qlora_forward, qlora_forward_noalloc, qlora_backward,
    qlora_adamw_step, qlora_adamw_step_host, qlora_workspace_fallbacks, qlora_workspace_set_wait_limit, qlora_storage_bytes,
    qlora_storage_bytes_absmax,
    qlora_workspace_bytes, qlora_nf4_codebook, qlora_nf4_thresholds, qlora_status_string,
    qlora_fp8_quantize, qlora_fp8_quantize_rows, qlora_fp8_forward, qlora_fp8_backward, qlora_fp8_storage_bytes,
    qlora_fp8_workspace_bytes, qlora_stream_capture_id, qlora_rmsnorm_forward, qlora_rmsnorm_backward, qlora_adamw_many

The C ABI sees only pointers, so every tensor argument is checked here before the call: its shape against the
weight and the other operands, its dtype, contiguity, and that it lives on the weight's GPU. A mismatch raises
TypeError (dtype) or ValueError (shape, layout, device) and nothing is launched.
"""

from __future__ import annotations

import bisect
import contextlib
import ctypes
import os
import threading
import warnings
from dataclasses import dataclass
from typing import NamedTuple

import torch

BLOCK = 64
GROUP = 256
MAX_RANK = 256
# The workspace starts with a counter region (u32 words) that must be zero before
# the first call and that every call leaves zero, except its last word, which
# counts the waits that ran out of time (qlora_workspace_fallbacks).
COUNTER_BYTES = 16384 * 4
STATIC_SCRATCH_BYTES = 1 << 20  # QLORA_STATIC_SCRATCH_BYTES: scratch of qlora_forward_noalloc per GPU

F32, BF16 = 0, 1

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqlora.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python -m bit_quantized_finetuning_amd.build` (hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)

try:
    from . import _marshal  # native marshalling of the calls made most often (csrc/binding.cpp)
except ImportError as e:  # not built, or against another torch: every call has its Python marshalling too
    _marshal = None
    warnings.warn(f"{os.path.dirname(LIB_PATH)}/_marshal.so does not load ({e}): calls are marshalled in Python, which "
                  "takes a few times as long per call; run `python -m bit_quantized_finetuning_amd.build`", RuntimeWarning)


class _Nf4Weight(ctypes.Structure):
    _fields_ = [("d_out", ctypes.c_int64), ("d_in", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("qscale", ctypes.c_void_p), ("smax", ctypes.c_void_p)]


_vp, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_W = ctypes.POINTER(_Nf4Weight)

_lib.qlora_quantize.argtypes = [_vp, ctypes.c_int, _W, _vp, _vp]
_lib.qlora_quantize.restype = ctypes.c_int
_lib.qlora_quantize_many.argtypes = [ctypes.POINTER(_vp), ctypes.c_int, _W, _i32, _vp, _vp]
_lib.qlora_quantize_many.restype = ctypes.c_int
_lib.qlora_dequantize.argtypes = [_W, ctypes.c_int, _vp, _vp]
_lib.qlora_dequantize.restype = ctypes.c_int
_lib.qlora_merge.argtypes = [_W, _vp, _vp, _i32, _f32, _vp, _vp]
_lib.qlora_merge.restype = ctypes.c_int
_lib.qlora_adamw_step.argtypes = [ctypes.c_void_p, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.qlora_adamw_step.restype = ctypes.c_int
_lib.qlora_adamw_step_host.argtypes = [ctypes.c_void_p, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i32]
_lib.qlora_adamw_step_host.restype = ctypes.c_int
_lib.qlora_forward.argtypes = [_W, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _sz, _vp]
_lib.qlora_forward.restype = ctypes.c_int


class _ForwardJob(ctypes.Structure):
    _fields_ = [("W", _W), ("x", _vp), ("T", _i64), ("A", _vp), ("B", _vp), ("r", _i32), ("alpha", _f32),
                ("h", _vp), ("u_out", _vp)]


_lib.qlora_forward_many.argtypes = [ctypes.POINTER(_ForwardJob), _i32, _vp, _sz, _vp]
_lib.qlora_forward_many.restype = ctypes.c_int
_lib.qlora_forward_many_workspace_bytes.argtypes = [_i32]
_lib.qlora_forward_many_workspace_bytes.restype = _sz
_lib.qlora_forward_noalloc.argtypes = [_W, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp]
_lib.qlora_forward_noalloc.restype = ctypes.c_int
_lib.qlora_workspace_fallbacks.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint32), _vp]
_lib.qlora_workspace_fallbacks.restype = ctypes.c_int
_lib.qlora_workspace_set_wait_limit.argtypes = [_vp, ctypes.c_uint32, _vp]
_lib.qlora_workspace_set_wait_limit.restype = ctypes.c_int
_lib.qlora_backward.argtypes = [_W, _vp, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.qlora_backward.restype = ctypes.c_int
_lib.qlora_storage_bytes.argtypes = [_i64, _i64]
_lib.qlora_storage_bytes.restype = _sz
_lib.qlora_storage_bytes_absmax.argtypes = [_i64, _i64]
_lib.qlora_storage_bytes_absmax.restype = _sz
_lib.qlora_workspace_bytes.argtypes = [_i64, _i64, _i64, _i32]
_lib.qlora_workspace_bytes.restype = _sz
_lib.qlora_nf4_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
_lib.qlora_nf4_codebook.restype = None
_lib.qlora_nf4_thresholds.argtypes = [ctypes.POINTER(ctypes.c_float)]
_lib.qlora_nf4_thresholds.restype = None
_lib.qlora_status_string.argtypes = [ctypes.c_int]
_lib.qlora_status_string.restype = ctypes.c_char_p

class _Fp8Weight(ctypes.Structure):
    _fields_ = [("d_out", _i64), ("d_in", _i64), ("codes", _vp), ("scales", _vp)]


class _AdamWJob(ctypes.Structure):
    _fields_ = [("grad", _vp), ("param", _vp), ("n", _i64)]


class _AdamWManyHparams(ctypes.Structure):
    _fields_ = [(k, ctypes.c_double) for k in ("lr", "beta1", "beta2", "eps", "weight_decay")]


class _AdamWState(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp), ("master", _vp)]


for _name, _args, _res in (
        ("qlora_fp8_quantize", [_vp, ctypes.c_int, ctypes.POINTER(_Fp8Weight), _vp], ctypes.c_int),
        ("qlora_fp8_quantize_rows", [_vp, ctypes.c_int, _i64, _i64, ctypes.c_int, _vp, _vp, _vp], ctypes.c_int),
        ("qlora_fp8_storage_bytes", [_i64, _i64], _sz),
        ("qlora_fp8_workspace_bytes", [_i64, _i64, _i64, _i32], _sz),
        ("qlora_fp8_forward", [ctypes.POINTER(_Fp8Weight), _vp, _vp, ctypes.c_int, _vp, _i64, _vp, _vp, _i32, _f32, _vp,
                               _vp, _vp, _sz, _vp], ctypes.c_int),
        ("qlora_fp8_backward", [ctypes.POINTER(_Fp8Weight), _vp, _vp, ctypes.c_int, _i64, _vp, _vp, _i32, _f32, _vp, _vp,
                                _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
        ("qlora_stream_capture_id", [ctypes.POINTER(ctypes.c_uint64), _vp], ctypes.c_int),
        ("qlora_rmsnorm_forward", [_vp, _i64, _vp, _i64, ctypes.c_int, _i64, _i64, _vp, ctypes.c_int, _f32, _vp, _vp, _vp,
                                   _vp, ctypes.c_int, _vp, _vp], ctypes.c_int),
        ("qlora_rmsnorm_workspace_bytes", [_i64, _i64], _sz),
        ("qlora_rmsnorm_backward", [_vp, _i64, _vp, _i64, _vp, _i64, ctypes.c_int, _i64, _i64, _vp, ctypes.c_int, _vp, _vp,
                                    _vp, _vp, _sz, _vp], ctypes.c_int),
        ("qlora_adamw_many_workspace_bytes", [_i32], _sz),
        ("qlora_adamw_many", [_vp, _i64, ctypes.POINTER(_AdamWJob), _i32, ctypes.c_int, ctypes.c_int,
                              ctypes.POINTER(_AdamWState), _f32, _vp, ctypes.c_uint32, _vp, _sz, _vp], ctypes.c_int)):
    getattr(_lib, _name).argtypes, getattr(_lib, _name).restype = _args, _res

lib = _lib  # raw handle, for tests of the C ABI itself


class QloraError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_lib.qlora_status_string(status).decode()} (status {status})")
        self.status = status


def _check(status: int, where: str):
    if status != 0:
        raise QloraError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream of a device index, as an integer


def _stream(device: torch.device):
    """The current stream of a tensor's device."""
    return ctypes.c_void_p(_raw_stream(device.index))


# ---------------------------------------------------------------------------
# host helpers (no GPU needed)
# ---------------------------------------------------------------------------

def qlora_nf4_codebook():
    buf = (ctypes.c_float * 16)()
    _lib.qlora_nf4_codebook(buf)
    return list(buf)


def qlora_nf4_thresholds():
    buf = (ctypes.c_float * 15)()
    _lib.qlora_nf4_thresholds(buf)
    return list(buf)


def qlora_storage_bytes(d_out: int, d_in: int) -> int:
    return int(_lib.qlora_storage_bytes(d_out, d_in))


def qlora_storage_bytes_absmax(d_out: int, d_in: int) -> int:
    return int(_lib.qlora_storage_bytes_absmax(d_out, d_in))


def qlora_workspace_bytes(d_out: int, d_in: int, T: int, r: int) -> int:
    return int(_lib.qlora_workspace_bytes(d_out, d_in, T, r))


def qlora_status_string(status: int) -> str:
    return _lib.qlora_status_string(status).decode()


# ---------------------------------------------------------------------------
# device entry points
# ---------------------------------------------------------------------------

@dataclass
class NF4Weight:
    """A quantized frozen weight: the three buffers of qlora_nf4_weight plus its shape.

    qscale None is the absmax-only storage (4.5 bits per weight): smax then holds the float32 absmax of
    every 64-weight block instead of one maximum per group of 256 blocks.
    """
    d_out: int
    d_in: int
    codes: torch.Tensor           # uint8 [d_out*d_in/2]
    qscale: torch.Tensor | None   # uint8 [d_out*d_in/64], or None
    smax: torch.Tensor            # float32 [ceil(d_out*d_in/64/256)], or [d_out*d_in/64] without qscale

    @property
    def double_quant(self) -> bool:
        return self.qscale is not None

    def _c(self):
        return _Nf4Weight(self.d_out, self.d_in, self.codes.data_ptr(),
                          None if self.qscale is None else self.qscale.data_ptr(), self.smax.data_ptr())

    @staticmethod
    def empty(d_out: int, d_in: int, device, double_quant: bool = True) -> "NF4Weight":
        n = d_out * d_in
        nb = n // BLOCK
        ng = (nb + GROUP - 1) // GROUP
        # 16-byte aligned allocations (torch's caching allocator aligns to >= 512 bytes)
        return NF4Weight(d_out, d_in,
                         torch.empty(n // 2, dtype=torch.uint8, device=device),
                         torch.empty(nb, dtype=torch.uint8, device=device) if double_quant else None,
                         torch.empty(ng if double_quant else nb, dtype=torch.float32, device=device))


_workspaces: dict = {}  # (device type, device index, stream) -> workspace
_captured: dict = {}    # the same key -> (capture, workspace of the calls of that capture)
# Held from the choice of a shared workspace to the call's last launch: threads that use one stream enqueue whole calls
# one after another. (Reentrant: an allocation in between may collect garbage.)
_enqueue = threading.RLock()


def _stream_id(dev: torch.device) -> int:
    """The current stream of a device as an integer (0 for a device without streams)."""
    return torch.cuda.current_stream(dev).cuda_stream if dev.type == "cuda" else 0


def _capture_id(dev: torch.device, stream: int) -> int:
    """A number for the graph capture that the stream takes part in, 0 when it is not being captured."""
    if dev.type != "cuda":
        return 0
    n = ctypes.c_uint64(0)
    _check(_lib.qlora_stream_capture_id(ctypes.byref(n), ctypes.c_void_p(stream)), "qlora_stream_capture_id")
    return int(n.value)


def workspace(device, nbytes: int) -> torch.Tensor:
    """The zero-initialised workspace cached for the device's current stream (the library leaves its counters zero after
    each call).

    Every call that does not pass a workspace of its own (`ws=`) uses the cached one of the stream it runs on, so calls
    on different streams may overlap. Calls captured into a graph share one from the graph's memory pool, cleared by a
    kernel at its first use in the graph, so that replays share nothing with eager calls or other graphs. A workspace
    that the caller passes serves one call at a time, in whatever streams; it is zeroed once, e.g. with
    `torch.zeros(qlora_workspace_bytes(...), dtype=torch.uint8, device=...)`.
    """
    dev = torch.device(device)
    stream = _stream_id(dev)
    key = (dev.type, dev.index, stream)
    capture = _capture_id(dev, stream)
    with _enqueue:
        if capture:
            of, ws = _captured.get(key, (0, None))
            if of != capture or ws.numel() < nbytes:
                ws = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
                ws[:COUNTER_BYTES].zero_()
                _captured[key] = (capture, ws)
            return ws
        ws = _workspaces.get(key)
        if ws is None or ws.numel() < nbytes:
            # (allocated on this stream, and replaced in its order: nothing has to be waited for)
            ws = torch.zeros(max(nbytes, 1 << 20, 0 if ws is None else 2 * ws.numel()), dtype=torch.uint8, device=dev)
            _workspaces[key] = ws
        return ws


def _own_workspace(ws: torch.Tensor, nbytes: int) -> torch.Tensor:
    if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.numel() < nbytes:
        raise ValueError(f"ws must be a contiguous uint8 tensor of at least {nbytes} bytes")
    return ws


class _ws_for:
    """The caller's workspace, or the stream's cached one, for as long as the call enqueues its launches."""
    __slots__ = ("ws", "dev", "nbytes")

    def __init__(self, ws, dev: torch.device, nbytes: int):
        self.ws, self.dev, self.nbytes = ws, dev, nbytes

    def __enter__(self) -> torch.Tensor:
        if self.ws is not None:
            return _own_workspace(self.ws, self.nbytes)
        _enqueue.acquire()
        try:
            ws, index = None, self.dev.index
            if self.dev.type == "cuda" and index == torch.cuda.current_device():
                ws = _cached_ws(index, _raw_stream(index))
            return workspace(self.dev, self.nbytes) if ws is None or ws.numel() < self.nbytes else ws
        except BaseException:
            _enqueue.release()
            raise

    def __exit__(self, *exc):
        if self.ws is None:
            _enqueue.release()


def _cached_ws(dev: int, stream: int):
    """The workspace cached for the current device's stream (None while a graph is captured, see workspace)."""
    return None if torch.cuda.is_current_stream_capturing() else _workspaces.get(("cuda", dev, stream))


def _bits(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.bfloat16:
        raise TypeError(f"expected a bfloat16 tensor, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t


def _arg(t, name: str, dtype, shape):
    """dtype, shape and contiguity of one tensor argument (None passes)."""
    if t is None:
        return
    if not torch.is_tensor(t):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_weight(w: "NF4Weight"):
    n = w.d_out * w.d_in
    if w.d_in % BLOCK or n <= 0:
        raise ValueError(f"weight shape {w.d_out}x{w.d_in}: d_in must be a positive multiple of {BLOCK}")
    nb = n // BLOCK
    _arg(w.codes, "codes", torch.uint8, (n // 2,))
    if w.qscale is not None:
        _arg(w.qscale, "qscale", torch.uint8, (nb,))
        _arg(w.smax, "smax", torch.float32, ((nb + GROUP - 1) // GROUP,))
    else:
        _arg(w.smax, "smax", torch.float32, (nb,))


def _check_devices(device, **tensors):
    """Every given tensor on `device`, a GPU (the checks that come last, so that the shape rules can be
    exercised without one)."""
    if device.type != "cuda":
        raise ValueError(f"the weight must be on a GPU, got {device}")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the weight on {device}")


def _adapter_rank(w: "NF4Weight", A, B) -> int:
    if (A is None) != (B is None):
        raise ValueError("give both A and B, or neither")
    if A is None:
        return 0
    if A.dim() != 2:
        raise ValueError(f"A must be [r, d_in], got shape {tuple(A.shape)}")
    r = A.shape[0]
    if r < 0 or r > MAX_RANK or r % 8:
        raise ValueError(f"rank {r} outside 0..{MAX_RANK} or not a multiple of 8")
    _arg(A, "A", torch.bfloat16, (r, w.d_in))
    _arg(B, "B", torch.bfloat16, (w.d_out, r))
    return r


def qlora_quantize(W: torch.Tensor, out: NF4Weight | None = None, flags: torch.Tensor | None = None,
                   double_quant: bool = True) -> NF4Weight:
    """NF4-quantize W; double_quant=False keeps each block's float32 absmax (ignored when `out` is given)."""
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D tensor")
    if W.dtype == torch.float32:
        dt = F32
    elif W.dtype == torch.bfloat16:
        dt = BF16
    else:
        raise TypeError(f"W must be float32 or bfloat16, got {W.dtype}")
    d_out, d_in = W.shape
    if out is None:
        out = NF4Weight.empty(d_out, d_in, W.device, double_quant)
    if (out.d_out, out.d_in) != (d_out, d_in):
        raise ValueError(f"out is {out.d_out}x{out.d_in}, W is {d_out}x{d_in}")
    _check_weight(out)
    if flags is not None and (flags.dtype not in (torch.int32, torch.uint32) or flags.numel() < 1):
        raise TypeError("flags must be a 32-bit integer tensor of at least one element")
    _check_devices(W.device, codes=out.codes, qscale=out.qscale, smax=out.smax, flags=flags)
    cw = out._c()
    _check(_lib.qlora_quantize(_ptr(W), dt, ctypes.byref(cw), _ptr(flags), _stream(W.device)), "qlora_quantize")
    return out


def qlora_quantize_many(Ws, outs=None, flags: torch.Tensor | None = None,
                        double_quant: bool = True) -> list:
    """NF4-quantize several weights of one dtype in shared launches (the results equal one qlora_quantize per
    weight); `outs` (optional) names each weight's output buffers."""
    Ws = list(Ws)
    if not Ws:
        return []
    dtypes = {W.dtype for W in Ws}
    if len(dtypes) != 1 or dtypes.pop() not in (torch.float32, torch.bfloat16):
        raise TypeError("all weights must be float32, or all bfloat16")
    dt = F32 if Ws[0].dtype == torch.float32 else BF16
    if outs is None:
        outs = [None] * len(Ws)
    outs = list(outs)
    if len(outs) != len(Ws):
        raise ValueError(f"{len(Ws)} weights but {len(outs)} outputs")
    if flags is not None and (flags.dtype not in (torch.int32, torch.uint32) or flags.numel() < 1):
        raise TypeError("flags must be a 32-bit integer tensor of at least one element")
    for i, W in enumerate(Ws):
        if W.dim() != 2 or not W.is_contiguous():
            raise ValueError("every W must be a contiguous 2-D tensor")
        if outs[i] is None:
            outs[i] = NF4Weight.empty(W.shape[0], W.shape[1], W.device, double_quant)
        o = outs[i]
        if (o.d_out, o.d_in) != tuple(W.shape):
            raise ValueError(f"out {i} is {o.d_out}x{o.d_in}, W is {W.shape[0]}x{W.shape[1]}")
        _check_weight(o)
        _check_devices(Ws[0].device, W=W, codes=o.codes, qscale=o.qscale, smax=o.smax, flags=flags)
    wp = (_vp * len(Ws))(*[W.data_ptr() for W in Ws])
    cw = (_Nf4Weight * len(Ws))(*[o._c() for o in outs])
    _check(_lib.qlora_quantize_many(wp, dt, cw, len(Ws), _ptr(flags), _stream(Ws[0].device)),
           "qlora_quantize_many")
    return outs


def qlora_dequantize(w: NF4Weight, dtype=torch.bfloat16) -> torch.Tensor:
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    _check_weight(w)
    _check_devices(w.codes.device, qscale=w.qscale, smax=w.smax)
    out = torch.empty(w.d_out, w.d_in, dtype=dtype, device=w.codes.device)
    dt = BF16 if dtype == torch.bfloat16 else F32
    cw = w._c()
    _check(_lib.qlora_dequantize(ctypes.byref(cw), dt, _ptr(out), _stream(out.device)), "qlora_dequantize")
    return out


def qlora_merge(w: NF4Weight, A: torch.Tensor | None, B: torch.Tensor | None, alpha: float,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [d_out, d_in] = bf16(W_hat + (alpha/r) B A): the adapter merged into the restored weight."""
    _check_weight(w)
    r = _adapter_rank(w, A, B)
    _arg(out, "out", torch.bfloat16, (w.d_out, w.d_in))
    dev = w.codes.device
    _check_devices(dev, qscale=w.qscale, smax=w.smax, A=A, B=B, out=out)
    if out is None:
        out = torch.empty(w.d_out, w.d_in, dtype=torch.bfloat16, device=dev)
    cw = w._c()
    _check(_lib.qlora_merge(ctypes.byref(cw), _ptr(A), _ptr(B), r, alpha, _ptr(out), _stream(out.device)),
           "qlora_merge")
    return out


class AdamWHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float)]


def qlora_adamw_step(step: int, grad: torch.Tensor, master: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                     param: torch.Tensor | None = None, lr: float = 1e-4, beta1: float = 0.9, beta2: float = 0.999,
                     eps: float = 1e-8, weight_decay: float = 0.0, stream: torch.cuda.Stream | None = None):
    """One AdamW step over float32 master/m/v (device or pinned host tensors, updated in place) from a device
    float32 gradient; param (device bf16, optional) receives bf16(master). Enqueued on `stream` (default: the
    current stream of grad's device)."""
    for t in (grad, master, m, v):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise TypeError("grad, master, m and v must be contiguous float32 tensors")
    n = grad.numel()
    if any(t.numel() != n for t in (master, m, v)) or (param is not None and param.numel() != n):
        raise ValueError("all tensors must have the same number of elements")
    if param is not None:
        _bits(param)
    if grad.device.type != "cuda":
        raise ValueError(f"grad must be on a GPU, got {grad.device}")
    _check_devices(grad.device, param=param)
    for name, t in (("master", master), ("m", m), ("v", v)):
        if t.device != grad.device and not (t.device.type == "cpu" and t.is_pinned()):
            raise ValueError(f"{name} must be on the gradient's GPU or in pinned host memory, got {t.device}")
    hp = AdamWHparams(lr, beta1, beta2, eps, weight_decay)
    st = ctypes.c_void_p((stream or torch.cuda.current_stream(grad.device)).cuda_stream)
    _check(_lib.qlora_adamw_step(ctypes.byref(hp), step, n, _ptr(grad), _ptr(master), _ptr(m), _ptr(v),
                                 _ptr(param), st), "qlora_adamw_step")


def qlora_adamw_step_host(step: int, grad: torch.Tensor, master: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                          param: torch.Tensor | None = None, lr: float = 1e-4, beta1: float = 0.9,
                          beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0, threads: int = 0):
    """The same AdamW step run by the host CPU: every tensor in host memory (pinned, so that the caller's copies
    to and from the device are DMA copies); param (bf16, optional) receives bf16(master). Blocks until done."""
    for t in (grad, master, m, v):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise TypeError("grad, master, m and v must be contiguous float32 tensors")
    n = grad.numel()
    if any(t.numel() != n for t in (master, m, v)) or (param is not None and param.numel() != n):
        raise ValueError("all tensors must have the same number of elements")
    if param is not None:
        _bits(param)
    for name, t in (("grad", grad), ("master", master), ("m", m), ("v", v), ("param", param)):
        if t is not None and t.device.type != "cpu":
            raise ValueError(f"{name} must be in host memory, got {t.device}")
    hp = AdamWHparams(lr, beta1, beta2, eps, weight_decay)
    _check(_lib.qlora_adamw_step_host(ctypes.byref(hp), step, n, _ptr(grad), _ptr(master), _ptr(m), _ptr(v),
                                      _ptr(param), int(threads)), "qlora_adamw_step_host")


def _check_no_overlap(inputs: dict, outputs: dict):
    """The kernels read their inputs while they write their outputs and workspace: no output may overlap an
    input or another output (in-place calls are not supported)."""
    named = [(n, _span(t), False) for n, t in inputs.items()] + [(n, _span(t), True) for n, t in outputs.items()]
    for i, (n1, s1, out1) in enumerate(named):
        if not out1 or s1 is None:
            continue
        for k, (n2, s2, _) in enumerate(named):
            if k != i and s2 is not None and s1[0] < s2[1] and s2[0] < s1[1]:
                raise ValueError(f"{n1} overlaps {n2}: outputs and workspace must not share memory with any "
                                 "other argument")


def _forward_args(w, x, A, B, h, u, save_u, ws=None):
    _check_weight(w)
    if not torch.is_tensor(x) or x.dim() != 2:
        raise ValueError("x must be a 2-D [T, d_in] tensor")
    T = x.shape[0]
    _arg(x, "x", torch.bfloat16, (T, w.d_in))
    r = _adapter_rank(w, A, B)
    _arg(h, "h", torch.bfloat16, (T, w.d_out))
    if u is not None and r == 0:
        raise ValueError("u is given but there is no adapter")
    _arg(u, "u", torch.float32, (T, r))
    if ws is not None:
        _own_workspace(ws, qlora_workspace_bytes(w.d_out, w.d_in, T, r))
    _check_no_overlap({"x": x, "A": A, "B": B, "codes": w.codes, "qscale": w.qscale, "smax": w.smax},
                      {"h": h, "u": u, "ws": ws})
    dev = w.codes.device
    _check_devices(dev, qscale=w.qscale, smax=w.smax, x=x, A=A, B=B, h=h, u=u, ws=ws)
    if h is None:
        h = torch.empty(T, w.d_out, dtype=torch.bfloat16, device=dev)
    if u is None and save_u and r > 0:
        u = torch.empty(T, r, dtype=torch.float32, device=dev)
    return T, r, h, u


def qlora_forward(w: NF4Weight, x: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None, alpha: float,
                  save_u: bool = False, h: torch.Tensor | None = None, u: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None):
    """h = x W_hat^T + (alpha/r) (x A^T) B^T. Returns (h, u); u is float32 [T, r] when save_u or given, else None.

    h and u may be passed in (preallocated outputs); otherwise they are allocated here.
    """
    T, r, h, u = _forward_args(w, x, A, B, h, u, save_u, ws)
    cw = w._c()
    with _ws_for(ws, x.device, qlora_workspace_bytes(w.d_out, w.d_in, T, r)) as ws:
        _check(_lib.qlora_forward(ctypes.byref(cw), _ptr(x), T, _ptr(A), _ptr(B), r, alpha, _ptr(h), _ptr(u),
                                  _ptr(ws), ws.numel(), _stream(x.device)), "qlora_forward")
    return h, u


MAX_FORWARD_JOBS = 64  # QLORA_MAX_FORWARD_JOBS


def _span(t):
    return None if t is None or t.numel() == 0 else (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())


def _check_independent(args):
    """The jobs of one grouped launch run at the same time: no output may overlap an input or output of any job
    (its own inputs included)."""
    spans = []
    for i, (w, x, T, A, B, r, alpha, h, u) in enumerate(args):
        for name, t in (("x", x), ("A", A), ("B", B), ("codes", w.codes), ("qscale", w.qscale), ("smax", w.smax)):
            spans.append((i, name, False, _span(t)))
        for name, t in (("h", h), ("u", u)):
            spans.append((i, name, True, _span(t)))
    for i, n1, out1, s1 in spans:
        if not out1 or s1 is None:
            continue
        for k, n2, out2, s2 in spans:
            if s2 is None or (k == i and n2 == n1):
                continue
            if s1[0] < s2[1] and s2[0] < s1[1]:
                raise ValueError(f"job {i}'s {n1} overlaps job {k}'s {n2}: the jobs of a grouped call must be "
                                 "independent")


def qlora_forward_many_workspace_bytes(count: int) -> int:
    return int(_lib.qlora_forward_many_workspace_bytes(int(count)))


def qlora_forward_many(jobs, ws: torch.Tensor | None = None):
    """Several independent forwards of T <= 16 tokens in as few launches as possible (qlora_forward_many).

    jobs: a sequence of dicts with keys w, x, A, B, alpha and optionally h, u (preallocated outputs) and save_u,
    as for qlora_forward. Returns [(h, u), ...] in job order. No job's output may overlap another job's input
    or output.
    """
    jobs = list(jobs)
    if not 1 <= len(jobs) <= MAX_FORWARD_JOBS:
        raise ValueError(f"between 1 and {MAX_FORWARD_JOBS} jobs, got {len(jobs)}")
    args, outs = [], []
    dev = None
    for i, j in enumerate(jobs):
        w = j["w"]
        T, r, h, u = _forward_args(w, j["x"], j.get("A"), j.get("B"), j.get("h"), j.get("u"), j.get("save_u", False))
        if T > 16:
            raise ValueError(f"job {i}: T = {T}; the grouped forward takes T <= 16")
        if dev is None:
            dev = w.codes.device
        elif w.codes.device != dev:
            raise ValueError(f"job {i} is on {w.codes.device}, job 0 on {dev}")
        args.append((w, j["x"], T, j.get("A"), j.get("B"), r, float(j["alpha"]), h, u))
        outs.append((h, u))
    _check_independent(args)
    nbytes = qlora_forward_many_workspace_bytes(len(jobs))
    if ws is not None:
        _check_devices(dev, ws=ws)
    cws = [a[0]._c() for a in args]  # kept alive for the call
    arr = (_ForwardJob * len(args))()
    for k, (a, cw) in enumerate(zip(args, cws)):
        w, x, T, A, B, r, alpha, h, u = a
        arr[k] = _ForwardJob(ctypes.pointer(cw), _ptr(x), T, _ptr(A), _ptr(B), r, alpha, _ptr(h), _ptr(u))
    with _ws_for(ws, dev, nbytes) as ws:
        _check(_lib.qlora_forward_many(arr, len(args), _ptr(ws), ws.numel(), _stream(dev)), "qlora_forward_many")
    return outs


def qlora_forward_noalloc(w: NF4Weight, x: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None,
                          alpha: float, h: torch.Tensor, u: torch.Tensor | None = None):
    """qlora_forward for T <= 16 on the library's static per-GPU scratch array instead of a workspace: no
    allocation in the library or here (h, and u when wanted, are the caller's). Calls that overlap on one GPU
    share the array and must be serialized by the caller."""
    if h is None:
        raise ValueError("qlora_forward_noalloc writes into a given h (it allocates nothing)")
    T, r, h, u = _forward_args(w, x, A, B, h, u, False)
    cw = w._c()
    _check(_lib.qlora_forward_noalloc(ctypes.byref(cw), _ptr(x), T, _ptr(A), _ptr(B), r, alpha, _ptr(h), _ptr(u),
                                      _stream(x.device)), "qlora_forward_noalloc")
    return h, u


def qlora_workspace_fallbacks(ws: torch.Tensor) -> int:
    """How many waits on this workspace ran out of time and took their fallback path (the results are the same;
    a nonzero count means launches on other streams held the compute units). Synchronizes the current stream."""
    _own_workspace(ws, COUNTER_BYTES)
    _check_devices(ws.device)
    n = ctypes.c_uint32(0)
    _check(_lib.qlora_workspace_fallbacks(_ptr(ws), ctypes.byref(n), _stream(ws.device)), "qlora_workspace_fallbacks")
    return int(n.value)


def qlora_workspace_set_wait_limit(ws: torch.Tensor, ticks: int) -> None:
    """A testing aid: later calls on this workspace give up a wait after `ticks` ticks of the 100 MHz clock and
    take the fallback path (1 sends every wait that does not succeed at once there); 0 restores the built-in
    limit. Synchronizes the current stream."""
    _own_workspace(ws, COUNTER_BYTES)
    _check_devices(ws.device)
    if not 0 <= int(ticks) < 1 << 32:
        raise ValueError("ticks must fit in 32 bits")
    _check(_lib.qlora_workspace_set_wait_limit(_ptr(ws), int(ticks), _stream(ws.device)),
           "qlora_workspace_set_wait_limit")


def qlora_backward(w: NF4Weight, x: torch.Tensor | None, dY: torch.Tensor, A: torch.Tensor | None,
                   B: torch.Tensor | None, alpha: float, u_saved: torch.Tensor | None = None,
                   need_dx: bool = True, need_dA: bool = True, need_dB: bool = True,
                   dX: torch.Tensor | None = None, dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None):
    """Returns (dX bf16 [T, d_in] | None, dA f32 [r, d_in] | None, dB f32 [d_out, r] | None).

    Outputs passed in are written in place (and count as needed); the others are allocated when needed.
    """
    _check_weight(w)
    if not torch.is_tensor(dY) or dY.dim() != 2:
        raise ValueError("dY must be a 2-D [T, d_out] tensor")
    T = dY.shape[0]
    _arg(dY, "dY", torch.bfloat16, (T, w.d_out))
    _arg(x, "x", torch.bfloat16, (T, w.d_in))
    r = _adapter_rank(w, A, B)
    if r == 0 and (dA is not None or dB is not None or u_saved is not None):
        raise ValueError("dA, dB and u_saved need an adapter")
    _arg(u_saved, "u_saved", torch.float32, (T, r))
    _arg(dX, "dX", torch.bfloat16, (T, w.d_in))
    _arg(dA, "dA", torch.float32, (r, w.d_in))
    _arg(dB, "dB", torch.float32, (w.d_out, r))
    nbytes = qlora_workspace_bytes(w.d_out, w.d_in, T, r)
    if ws is not None:
        _own_workspace(ws, nbytes)
    _check_no_overlap({"x": x, "dY": dY, "A": A, "B": B, "u_saved": u_saved, "codes": w.codes, "qscale": w.qscale,
                       "smax": w.smax}, {"dX": dX, "dA": dA, "dB": dB, "ws": ws})
    dev = w.codes.device
    _check_devices(dev, qscale=w.qscale, smax=w.smax, x=x, dY=dY, A=A, B=B, u_saved=u_saved, dX=dX, dA=dA, dB=dB,
                   ws=ws)
    if dX is None and need_dx:
        dX = torch.empty(T, w.d_in, dtype=torch.bfloat16, device=dev)
    if dA is None and need_dA and r > 0:
        dA = torch.empty(r, w.d_in, dtype=torch.float32, device=dev)
    if dB is None and need_dB and r > 0:
        dB = torch.empty(w.d_out, r, dtype=torch.float32, device=dev)
    cw = w._c()
    with _ws_for(ws, dev, nbytes) as ws:
        _check(_lib.qlora_backward(ctypes.byref(cw), _ptr(x), _ptr(dY), T, _ptr(A), _ptr(B), r, alpha, _ptr(u_saved),
                                   _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(), _stream(dev)), "qlora_backward")
    return dX, dA, dB


# ---------------------------------------------------------------------------
# the 8-bit frozen base
# ---------------------------------------------------------------------------

FP8_GROUP = 128     # QLORA_FP8_GROUP
ADAMW_BLOCK = 256   # QLORA_ADAMW_BLOCK
NORM_MAX_DIM = 32768  # QLORA_NORM_MAX_DIM
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
_FMT = {E4M3: 2, E5M2: 3}
_FLOAT = {torch.float32: F32, torch.bfloat16: BF16}


def _fmt(fmt) -> int:
    if fmt not in _FMT:
        raise TypeError(f"fmt must be torch.float8_e4m3fn or torch.float8_e5m2, got {fmt}")
    return _FMT[fmt]


def _float(t, name: str) -> int:
    if not torch.is_tensor(t):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in _FLOAT:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return _FLOAT[t.dtype]


def _groups(d: int) -> int:
    return -(-d // FP8_GROUP)


def _done(answer, where: str):
    """The results of a call that the native marshalling made; a status it got is raised."""
    if type(answer) is int:
        _check(answer, where)
    return answer


def _on(dev):
    """The library launches on the current device: make `dev` current where it is not."""
    return contextlib.nullcontext() if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


@dataclass
class Fp8Weight:
    """A frozen weight in e4m3 with one float32 scale per 128 x 128 block: the buffers of qlora_fp8_weight."""
    d_out: int
    d_in: int
    codes: torch.Tensor   # float8_e4m3fn [d_out, d_in]
    scales: torch.Tensor  # float32 [ceil(d_out / 128), ceil(d_in / 128)]

    def _c(self):
        return _Fp8Weight(self.d_out, self.d_in, self.codes.data_ptr(), self.scales.data_ptr())

    @staticmethod
    def empty(d_out: int, d_in: int, device) -> "Fp8Weight":
        return Fp8Weight(d_out, d_in, torch.empty(d_out, d_in, dtype=E4M3, device=device),
                         torch.empty(_groups(d_out), _groups(d_in), dtype=torch.float32, device=device))


def qlora_fp8_storage_bytes(d_out: int, d_in: int) -> int:
    return int(_lib.qlora_fp8_storage_bytes(d_out, d_in))


def qlora_fp8_workspace_bytes(d_out: int, d_in: int, T: int, r: int) -> int:
    return int(_lib.qlora_fp8_workspace_bytes(d_out, d_in, T, r))


def _check_fp8_weight(w: Fp8Weight):
    if w.d_out < 16 or w.d_in < 16 or w.d_out % 16 or w.d_in % 16:
        raise ValueError(f"weight shape {w.d_out}x{w.d_in}: both must be positive multiples of 16")
    _arg(w.codes, "codes", E4M3, (w.d_out, w.d_in))
    _arg(w.scales, "scales", torch.float32, (_groups(w.d_out), _groups(w.d_in)))


def qlora_fp8_quantize(W: torch.Tensor, out: Fp8Weight | None = None) -> Fp8Weight:
    """W (float32 or bfloat16 [d_out, d_in]) to e4m3 with scale amax / 448 per 128 x 128 block."""
    dt = _float(W, "W")
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D tensor")
    d_out, d_in = W.shape
    if out is None:
        if d_out % 16 or d_in % 16:
            raise ValueError(f"weight shape {d_out}x{d_in}: both must be positive multiples of 16")
        out = Fp8Weight.empty(d_out, d_in, W.device)
    if (out.d_out, out.d_in) != (d_out, d_in):
        raise ValueError(f"out is {out.d_out}x{out.d_in}, W is {d_out}x{d_in}")
    _check_fp8_weight(out)
    _check_no_overlap({"W": W}, {"codes": out.codes, "scales": out.scales})
    _check_devices(W.device, codes=out.codes, scales=out.scales)
    cw = out._c()
    with _on(W.device):
        _check(_lib.qlora_fp8_quantize(_ptr(W), dt, ctypes.byref(cw), _stream(W.device)), "qlora_fp8_quantize")
    return out


def qlora_fp8_quantize_rows(x: torch.Tensor, fmt=E4M3, xq: torch.Tensor | None = None, xs: torch.Tensor | None = None):
    """Rows x [T, d] (float32 or bfloat16, d % 16 == 0) to 8 bits in groups of 128 with power-of-two scales.
    Returns (xq fmt [T, d], xs float32 [T, ceil(d / 128)])."""
    dt, f = _float(x, "x"), _fmt(fmt)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D tensor")
    T, d = x.shape
    if T < 1 or d < 16 or d % 16:
        raise ValueError(f"x must be [T >= 1, d] with d a positive multiple of 16, got {tuple(x.shape)}")
    _arg(xq, "xq", fmt, (T, d))
    _arg(xs, "xs", torch.float32, (T, _groups(d)))
    _check_no_overlap({"x": x}, {"xq": xq, "xs": xs})
    _check_devices(x.device, xq=xq, xs=xs)
    if xq is None:
        xq = torch.empty(T, d, dtype=fmt, device=x.device)
    if xs is None:
        xs = torch.empty(T, _groups(d), dtype=torch.float32, device=x.device)
    with _on(x.device):
        _check(_lib.qlora_fp8_quantize_rows(_ptr(x), dt, T, d, f, _ptr(xq), _ptr(xs), _stream(x.device)),
               "qlora_fp8_quantize_rows")
    return xq, xs


def qlora_fp8_forward(w: Fp8Weight, x: torch.Tensor | None, A: torch.Tensor | None, B: torch.Tensor | None,
                      alpha: float, xq: torch.Tensor | None = None, xs: torch.Tensor | None = None, fmt=E4M3,
                      save_u: bool = False, h: torch.Tensor | None = None, u: torch.Tensor | None = None,
                      ws: torch.Tensor | None = None):
    """h = xq W_hat^T (block-scaled) + (alpha/r) (x A^T) B^T over the 8-bit base. Returns (h bf16 [T, d_out], u).

    xq, xs: the 8-bit rows of a norm or of qlora_fp8_quantize_rows, in fmt; without them x (bf16 [T, d_in]) is
    quantized to fmt within the call. x itself is needed then, and for the adapter. u is float32 [T, r] when
    save_u or given, else None."""
    f = _fmt(fmt)
    if _marshal is not None and h is None and u is None and ws is None and w.codes.is_cuda:
        dev = torch.cuda.current_device()
        stream = _raw_stream(dev)
        with _enqueue:
            out = _marshal.fp8_forward(w.codes, w.scales, w.d_out, w.d_in, x, A, B, alpha, xq, xs, f, save_u,
                                       _cached_ws(dev, stream), dev, stream)
        if out is not None:
            return _done(out, "qlora_fp8_forward")
    _check_fp8_weight(w)
    if (xq is None) != (xs is None):
        raise ValueError("give both xq and xs, or neither")
    lead = x if x is not None else xq
    if lead is None:
        raise ValueError("give x, or xq and xs")
    if not torch.is_tensor(lead) or lead.dim() != 2:
        raise ValueError("x and xq must be 2-D [T, d_in] tensors")
    T = lead.shape[0]
    if T < 1:
        raise ValueError("x must have at least one row")
    _arg(x, "x", torch.bfloat16, (T, w.d_in))
    _arg(xq, "xq", fmt, (T, w.d_in))
    _arg(xs, "xs", torch.float32, (T, _groups(w.d_in)))
    r = _adapter_rank(w, A, B)
    if r and x is None:
        raise ValueError("the adapter needs x")
    _arg(h, "h", torch.bfloat16, (T, w.d_out))
    if u is not None and r == 0:
        raise ValueError("u is given but there is no adapter")
    _arg(u, "u", torch.float32, (T, r))
    nbytes = qlora_fp8_workspace_bytes(w.d_out, w.d_in, T, r)
    if h is not None or u is not None or ws is not None:
        _check_no_overlap({"x": x, "xq": xq, "xs": xs, "A": A, "B": B, "codes": w.codes, "scales": w.scales},
                          {"h": h, "u": u, "ws": ws})
    dev = w.codes.device
    _check_devices(dev, scales=w.scales, x=x, xq=xq, xs=xs, A=A, B=B, h=h, u=u, ws=ws)
    if h is None:
        h = torch.empty(T, w.d_out, dtype=torch.bfloat16, device=dev)
    if u is None and save_u and r > 0:
        u = torch.empty(T, r, dtype=torch.float32, device=dev)
    cw = w._c()
    with _on(dev), _ws_for(ws, dev, nbytes) as ws:
        _check(_lib.qlora_fp8_forward(ctypes.byref(cw), _ptr(xq), _ptr(xs), f, _ptr(x), T, _ptr(A), _ptr(B), r, alpha,
                                      _ptr(h), _ptr(u), _ptr(ws), ws.numel(), _stream(dev)), "qlora_fp8_forward")
    return h, u


def qlora_fp8_backward(w: Fp8Weight, x: torch.Tensor | None, dY: torch.Tensor, A: torch.Tensor | None,
                       B: torch.Tensor | None, alpha: float, u_saved: torch.Tensor | None = None, need_dx: bool = True,
                       need_dA: bool = True, need_dB: bool = True, fmt=E4M3, dX: torch.Tensor | None = None,
                       dA: torch.Tensor | None = None, dB: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Returns (dX bf16 [T, d_in] | None, dA f32 [r, d_in] | None, dB f32 [d_out, r] | None); dY is quantized to fmt
    within the call for dX's product with the base, and used as it is for the adapter."""
    f = _fmt(fmt)
    if _marshal is not None and dX is None and dA is None and dB is None and ws is None and w.codes.is_cuda:
        dev = torch.cuda.current_device()
        stream = _raw_stream(dev)
        with _enqueue:
            out = _marshal.fp8_backward(w.codes, w.scales, w.d_out, w.d_in, x, dY, A, B, alpha, u_saved, need_dx, need_dA,
                                        need_dB, f, _cached_ws(dev, stream), dev, stream)
        if out is not None:
            return _done(out, "qlora_fp8_backward")
    _check_fp8_weight(w)
    if not torch.is_tensor(dY) or dY.dim() != 2 or dY.shape[0] < 1:
        raise ValueError("dY must be a 2-D [T >= 1, d_out] tensor")
    T = dY.shape[0]
    _arg(dY, "dY", torch.bfloat16, (T, w.d_out))
    _arg(x, "x", torch.bfloat16, (T, w.d_in))
    r = _adapter_rank(w, A, B)
    if r == 0 and (dA is not None or dB is not None or u_saved is not None):
        raise ValueError("dA, dB and u_saved need an adapter")
    _arg(u_saved, "u_saved", torch.float32, (T, r))
    _arg(dX, "dX", torch.bfloat16, (T, w.d_in))
    _arg(dA, "dA", torch.float32, (r, w.d_in))
    _arg(dB, "dB", torch.float32, (w.d_out, r))
    need_dA, need_dB = r > 0 and (need_dA or dA is not None), r > 0 and (need_dB or dB is not None)
    if x is None and (need_dA or (need_dB and u_saved is None)):
        raise ValueError("dA needs x, and dB needs x or u_saved")
    nbytes = qlora_fp8_workspace_bytes(w.d_out, w.d_in, T, r)
    if dX is not None or dA is not None or dB is not None or ws is not None:
        _check_no_overlap({"x": x, "dY": dY, "A": A, "B": B, "u_saved": u_saved, "codes": w.codes, "scales": w.scales},
                          {"dX": dX, "dA": dA, "dB": dB, "ws": ws})
    dev = w.codes.device
    _check_devices(dev, scales=w.scales, x=x, dY=dY, A=A, B=B, u_saved=u_saved, dX=dX, dA=dA, dB=dB, ws=ws)
    if dX is None and need_dx:
        dX = torch.empty(T, w.d_in, dtype=torch.bfloat16, device=dev)
    if dA is None and need_dA:
        dA = torch.empty(r, w.d_in, dtype=torch.float32, device=dev)
    if dB is None and need_dB:
        dB = torch.empty(w.d_out, r, dtype=torch.float32, device=dev)
    cw = w._c()
    with _on(dev), _ws_for(ws, dev, nbytes) as ws:
        _check(_lib.qlora_fp8_backward(ctypes.byref(cw), _ptr(x), _ptr(dY), f, T, _ptr(A), _ptr(B), r, alpha,
                                       _ptr(u_saved), _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(), _stream(dev)),
               "qlora_fp8_backward")
    return dX, dA, dB


# ---------------------------------------------------------------------------
# the root-mean-square norm
# ---------------------------------------------------------------------------

class RMSNormOut(NamedTuple):
    y: torch.Tensor | None     # x's dtype [T, d]
    yq: torch.Tensor | None    # fmt [T, d]
    ys: torch.Tensor | None    # float32 [T, ceil(d / 128)]
    s: torch.Tensor | None     # x + residual in x's dtype, when a residual was given
    rstd: torch.Tensor | None  # float32 [T]


def _rows(t, name: str, dtype, T: int, d: int):
    """A [T, d] tensor of `dtype` whose rows are dense (any row stride of at least d)."""
    if t is None:
        return
    if not torch.is_tensor(t):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] != T or t.shape[1] != d:
        raise ValueError(f"{name} must have shape {(T, d)}, got {tuple(t.shape)}")
    if (d > 1 and t.stride(1) != 1) or (T > 1 and t.stride(0) < d):
        raise ValueError(f"{name} must have dense rows that do not overlap, got strides {t.stride()}")


def _row_stride(t, d: int) -> int:
    return d if t is None or t.shape[0] <= 1 else t.stride(0)


def _norm_weight(weight, d: int) -> int:
    if weight is None:
        return F32
    wd = _float(weight, "weight")
    _arg(weight, "weight", weight.dtype, (d,))
    return wd


def qlora_rmsnorm_forward(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                          eps: float = 1e-6, want_y: bool = True, fmt=None, save_rstd: bool = False) -> RMSNormOut:
    """s = x + residual (rounded to x's dtype); y = s / sqrt(mean(s^2) + eps) * weight over the rows of x [T, d]
    (float32 or bfloat16, any row stride). y comes in x's dtype (want_y) and / or as 8-bit rows with scales (fmt:
    torch.float8_e4m3fn or torch.float8_e5m2), as qlora_fp8_forward takes them."""
    f = 0 if fmt is None else _fmt(fmt)
    if _marshal is not None and torch.is_tensor(x) and x.is_cuda:
        dev = torch.cuda.current_device()
        out = _marshal.rmsnorm_forward(x, weight, residual, eps, want_y, f, save_rstd, dev, _raw_stream(dev))
        if out is not None:
            return RMSNormOut(*_done(out, "qlora_rmsnorm_forward"))
    dt = _float(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a 2-D [T, d] tensor")
    T, d = x.shape
    if not 1 <= d <= NORM_MAX_DIM:
        raise ValueError(f"rows of {d} values: 1 to {NORM_MAX_DIM}")
    _rows(x, "x", x.dtype, T, d)
    _rows(residual, "residual", x.dtype, T, d)
    wd = _norm_weight(weight, d)
    if not want_y and fmt is None:
        raise ValueError("nothing to write: want_y is false and fmt is None")
    dev = x.device
    _check_devices(dev, weight=weight, residual=residual)
    y = torch.empty(T, d, dtype=x.dtype, device=dev) if want_y else None
    s = torch.empty(T, d, dtype=x.dtype, device=dev) if residual is not None else None
    yq = ys = None
    if fmt is not None:
        yq = torch.empty(T, d, dtype=fmt, device=dev)
        ys = torch.empty(T, _groups(d), dtype=torch.float32, device=dev)
    rstd = torch.empty(T, dtype=torch.float32, device=dev) if save_rstd else None
    with _on(dev):
        _check(_lib.qlora_rmsnorm_forward(_ptr(x), _row_stride(x, d), _ptr(residual), _row_stride(residual, d), dt, T, d,
                                          _ptr(weight), wd, eps, _ptr(s), _ptr(y), _ptr(yq), _ptr(ys), f, _ptr(rstd),
                                          _stream(dev)), "qlora_rmsnorm_forward")
    return RMSNormOut(y, yq, ys, s, rstd)


def qlora_rmsnorm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor | None, rstd: torch.Tensor,
                           ds: torch.Tensor | None = None, need_dw: bool = False, ws: torch.Tensor | None = None):
    """Returns (dx, dw): dx in s's dtype is the gradient of x and of the residual; dw float32 [d] when need_dw. dy is
    the gradient of y, ds the one that reaches s past the norm (both in s's dtype, any row stride)."""
    if _marshal is not None and ws is None and torch.is_tensor(s) and s.is_cuda:
        dev = torch.cuda.current_device()
        out = _marshal.rmsnorm_backward(dy, s, weight, rstd, ds, need_dw, dev, _raw_stream(dev))
        if out is not None:
            return _done(out, "qlora_rmsnorm_backward")
    dt = _float(s, "s")
    if s.dim() != 2:
        raise ValueError("s must be a 2-D [T, d] tensor")
    T, d = s.shape
    if not 1 <= d <= NORM_MAX_DIM:
        raise ValueError(f"rows of {d} values: 1 to {NORM_MAX_DIM}")
    _rows(s, "s", s.dtype, T, d)
    if dy is None:
        raise TypeError("dy must be a tensor")
    _rows(dy, "dy", s.dtype, T, d)
    _rows(ds, "ds", s.dtype, T, d)
    wd = _norm_weight(weight, d)
    if rstd is None:
        raise TypeError("rstd must be a tensor")
    _arg(rstd, "rstd", torch.float32, (T,))
    dev = s.device
    _check_devices(dev, dy=dy, ds=ds, weight=weight, rstd=rstd, ws=ws)
    dx = torch.empty(T, d, dtype=s.dtype, device=dev)
    dw = torch.empty(d, dtype=torch.float32, device=dev) if need_dw else None
    with _on(dev):
        nbytes = 0
        if need_dw:  # the partial sums of dw: scratch of this call alone
            nbytes = int(_lib.qlora_rmsnorm_workspace_bytes(T, d))
            if ws is not None:
                _check_no_overlap({"dy": dy, "s": s, "ds": ds, "weight": weight, "rstd": rstd},
                                  {"ws": _own_workspace(ws, nbytes)})
            else:
                ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check(_lib.qlora_rmsnorm_backward(_ptr(dy), _row_stride(dy, d), _ptr(s), _row_stride(s, d), _ptr(ds),
                                           _row_stride(ds, d), dt, T, d, _ptr(weight), wd, _ptr(rstd), _ptr(dx), _ptr(dw),
                                           _ptr(ws) if need_dw else None, nbytes, _stream(dev)),
               "qlora_rmsnorm_backward")
    return dx, dw


# ---------------------------------------------------------------------------
# AdamW over many tensors
# ---------------------------------------------------------------------------

def _neighbours(spans):
    spans.sort()
    return zip(spans, spans[1:])


def _meets(span, spans) -> bool:
    """Whether a span overlaps one of `spans` (sorted, none overlapping another)."""
    i = bisect.bisect_left(spans, (span[1],))  # the first that starts at or past its end
    return i > 0 and spans[i - 1][1] > span[0]


def adamw_state_elements(sizes) -> int:
    """Elements of the flat state of tensors of these sizes: each starts at a multiple of 256."""
    return sum(-(-n // ADAMW_BLOCK) * ADAMW_BLOCK for n in sizes)


def qlora_adamw_many(step: int, grads, params, m: torch.Tensor, v: torch.Tensor, m_scale: torch.Tensor | None = None,
                     v_scale: torch.Tensor | None = None, master: torch.Tensor | None = None, lr: float = 1e-4,
                     beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                     max_norm: float | None = None, seed: int = 0, norm: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None) -> torch.Tensor | None:
    """One AdamW step over lists of gradients (all float32 or all bfloat16; None leaves that parameter and its moments
    as they are) and parameters (all float32, or all bfloat16 with a float32 `master` copy), in place.

    m, v, master are flat: tensor i's elements start after those of the tensors before it, each rounded up to a
    multiple of 256 (adamw_state_elements of the sizes in all). float32 m and v hold the moments; float8_e4m3fn ones
    hold 8-bit codes of m and sqrt(v), with float32 m_scale and v_scale per 256 elements, rounded stochastically by
    bits that depend on (seed, step, place) alone. max_norm: gradients are scaled to at most that global norm first,
    and a norm that is not finite leaves everything as it was; the norm is returned (float32 [1], on the device)."""
    grads, params = list(grads), list(params)
    if (_marshal is not None and ws is None and (max_norm is None or max_norm > 0) and torch.is_tensor(m)
            and m.is_cuda):
        dev = torch.cuda.current_device()
        out = _marshal.adamw_many(step, grads, params, m, v, m_scale, v_scale, master, lr, beta1, beta2, eps,
                                  weight_decay, 0.0 if max_norm is None else max_norm, seed, norm, dev, _raw_stream(dev))
        if out is not None:
            return _done(out, "qlora_adamw_many")[0]
    count = len(grads)
    if len(params) != count:
        raise ValueError(f"{count} gradients but {len(params)} parameters")
    if not torch.is_tensor(m) or not torch.is_tensor(v):
        raise TypeError("m and v must be tensors")
    dev = m.device
    gd = next((g.dtype for g in grads if g is not None), torch.float32)
    pd = params[0].dtype if count else torch.float32
    if gd not in _FLOAT or pd not in _FLOAT:
        raise TypeError(f"gradients and parameters must be float32 or bfloat16, got {gd} and {pd}")
    jobs = (_AdamWJob * max(count, 1))()
    total, spans = 0, []
    for i in range(count):
        g, p = grads[i], params[i]
        n = p.numel()
        if (g is not None and g.dtype is not gd) or p.dtype is not pd:
            raise TypeError(f"tensor {i}: all gradients must be {gd} and all parameters {pd}")
        if not p.is_contiguous() or (g is not None and (g.numel() != n or not g.is_contiguous())):
            raise ValueError(f"tensor {i}: gradient and parameter must be contiguous and of one size")
        if p.device != dev or (g is not None and g.device != dev):
            raise ValueError(f"tensor {i} is not on {dev}, where the state is")
        j = jobs[i]
        at = p.data_ptr()
        j.grad, j.param, j.n = None if g is None else g.data_ptr(), at, n
        total += -(-n // ADAMW_BLOCK) * ADAMW_BLOCK
        if n:
            spans.append((at, at + n * p.element_size()))
    if any(a[1] > b[0] for a, b in _neighbours(spans)):
        raise ValueError("parameters overlap (is one listed twice?)")
    bits8 = m.dtype == E4M3
    if not bits8 and m.dtype != torch.float32:
        raise TypeError(f"m must be float32 or float8_e4m3fn, got {m.dtype}")
    _arg(m, "m", m.dtype, (total,))
    _arg(v, "v", m.dtype, (total,))
    if bits8 != (m_scale is not None) or bits8 != (v_scale is not None):
        raise ValueError("8-bit moments need m_scale and v_scale, 32-bit ones take none")
    _arg(m_scale, "m_scale", torch.float32, (total // ADAMW_BLOCK,))
    _arg(v_scale, "v_scale", torch.float32, (total // ADAMW_BLOCK,))
    if count and (pd == torch.bfloat16) != (master is not None):
        raise ValueError("bfloat16 parameters need a float32 master copy, float32 ones take none")
    _arg(master, "master", torch.float32, (total,))
    if not 0 <= int(seed) < 1 << 32:
        raise ValueError("seed must fit in 32 bits")
    _arg(norm, "norm", torch.float32, (1,))
    if ws is not None and max_norm is not None:
        _own_workspace(ws, int(_lib.qlora_adamw_many_workspace_bytes(count)))
    for t in (m, v, m_scale, v_scale, master, norm, ws if max_norm is not None else None):
        if t is not None and t.numel():
            spans.append(_span(t))
    if any(a[1] > b[0] for a, b in _neighbours(spans)):
        raise ValueError("the state, the parameters, norm and workspace must not overlap")
    if any(_meets(_span(g), spans) for g in grads if g is not None and g.numel()):
        raise ValueError("a gradient overlaps a parameter, the state, norm or the workspace")
    if max_norm is None and norm is not None:
        raise ValueError("norm is given but max_norm is not")
    if max_norm is not None and not ctypes.c_float(max_norm).value > 0:
        raise ValueError(f"max_norm must be positive in float32, got {max_norm}")
    _check_devices(dev, v=v, m_scale=m_scale, v_scale=v_scale, master=master, norm=norm, ws=ws)
    hp = _AdamWManyHparams(lr, beta1, beta2, eps, weight_decay)
    st = _AdamWState(2 if bits8 else 0, m.data_ptr(), v.data_ptr(), _ptr(m_scale), _ptr(v_scale), _ptr(master))
    with _on(dev):
        nbytes = 0
        if max_norm is not None:
            if norm is None:
                norm = torch.empty(1, dtype=torch.float32, device=dev)
            nbytes = int(_lib.qlora_adamw_many_workspace_bytes(count))
            # partial sums, scratch of this call alone
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if ws is None else _own_workspace(ws, nbytes)
        _check(_lib.qlora_adamw_many(ctypes.byref(hp), step, jobs, count, _FLOAT[gd], _FLOAT[pd], ctypes.byref(st),
                                     0.0 if max_norm is None else max_norm, _ptr(norm), int(seed),
                                     None if max_norm is None else _ptr(ws), nbytes, _stream(dev)), "qlora_adamw_many")
    return norm
