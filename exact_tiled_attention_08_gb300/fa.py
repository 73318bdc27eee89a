"""Thin Python binding of the C ABI in ``include/fa.h`` (ctypes).

Every function here has the name of the C entry point it wraps and does
argument marshalling only: it checks dtypes, shapes, contiguity and devices of
the torch tensors it is given, passes their device pointers and sizes to the
library, and raises ``FaError`` on a non-OK status.  All arithmetic runs in the
library's CUDA kernels; there is no other implementation behind these names.
If the compiled library is missing, loading fails loudly.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import struct

import torch

from .build import LIB_PATH

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_MISALIGNED = 2
FA_ERR_UNSUPPORTED = 3
FA_ERR_CUDA = 4
FA_ERR_TIMEOUT = 5

_STATUS_NAMES = {
    FA_OK: "FA_OK",
    FA_ERR_INVALID_ARG: "FA_ERR_INVALID_ARG",
    FA_ERR_MISALIGNED: "FA_ERR_MISALIGNED",
    FA_ERR_UNSUPPORTED: "FA_ERR_UNSUPPORTED",
    FA_ERR_CUDA: "FA_ERR_CUDA",
    FA_ERR_TIMEOUT: "FA_ERR_TIMEOUT",
}


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS_NAMES.get(status, status)}")


# The argument structs of the *_packed entry points (fa_rows: Pqqq).  One struct
# costs a call a fraction of what twenty ctypes arguments do.
_PACKED = {
    "fa_cross_fwd": struct.Struct("@7PN6ifP").pack,
    "fa_cross_bwd": struct.Struct("@11PN6ifP").pack,
    "fa_tree_fwd": struct.Struct("@9PN6ifP").pack,
    "fa_rope_fwd": struct.Struct("@PqqqPqqqPqqq8P8i2fiP").pack,
    "fa_rope_bwd": struct.Struct("@PqqqPqqq7PPqqqPqqqPqqq3PN7i2fiP").pack,
}
_entries = {}  # name -> (packed entry point, pack)

_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libfa.so (built by ``build.build_library``); raises if it is absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libfa.so not found at {p}: run __graft_entry__.build() (no fallback exists)")
    lib = ctypes.CDLL(p)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_fp8_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_fwd_fp8_workspace_bytes.restype = sz
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, f, i, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_bwd_preprocess.argtypes = [vp, vp, vp, i, i, i, i, vp]
    lib.fa_bwd_preprocess.restype = i
    lib.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_bwd_workspace_bytes.restype = sz
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, f, i, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_deterministic.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, f, i, vp]
    lib.fa_bwd_deterministic.restype = i
    lib.fa_bwd_static_scratch.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_bwd_static_scratch.restype = i
    lib.fa_cross_fwd_workspace_bytes.argtypes = [i] * 6
    lib.fa_cross_fwd_workspace_bytes.restype = sz
    lib.fa_cross_fwd.argtypes = [vp] * 7 + [sz] + [i] * 6 + [f, vp]
    lib.fa_cross_fwd.restype = i
    lib.fa_cross_bwd_workspace_bytes.argtypes = [i] * 6
    lib.fa_cross_bwd_workspace_bytes.restype = sz
    lib.fa_cross_bwd.argtypes = [vp] * 11 + [sz] + [i] * 6 + [f, vp]
    lib.fa_cross_bwd.restype = i
    lib.fa_tree_fwd_workspace_bytes.argtypes = [i] * 6
    lib.fa_tree_fwd_workspace_bytes.restype = sz
    lib.fa_tree_fwd.argtypes = [vp] * 9 + [sz] + [i] * 6 + [f, vp]
    lib.fa_tree_fwd.restype = i
    rows = vp  # fa_rows: an address, or its 32 bytes
    for entry in _PACKED:
        getattr(lib, entry + "_packed").argtypes = [vp]
        getattr(lib, entry + "_packed").restype = i
    lib.fa_rope_fwd.argtypes = [rows] * 3 + [vp] * 8 + [i] * 8 + [f, f, i, vp]
    lib.fa_rope_fwd.restype = i
    lib.fa_rope_bwd_workspace_bytes.argtypes = [i] * 5
    lib.fa_rope_bwd_workspace_bytes.restype = sz
    lib.fa_rope_bwd.argtypes = [rows] * 2 + [vp] * 7 + [rows] * 3 + [vp] * 3 + [sz] + [i] * 7 + [f, f, i, vp]
    lib.fa_rope_bwd.restype = i
    lib.fa_check_device_status.argtypes = [vp]
    lib.fa_check_device_status.restype = i
    lib.fa_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.fa_set_wait_limit_ns.restype = None
    lib.fa_debug_stall.argtypes = [i]
    lib.fa_debug_stall.restype = None
    lib.fa_set_bwd_pair_mma.argtypes = [i]
    lib.fa_set_bwd_pair_mma.restype = None
    lib.fa_set_exp2_split.argtypes = [i]
    lib.fa_set_exp2_split.restype = i
    lib.fa_set_timing_events.argtypes = [vp, vp, vp, vp]
    lib.fa_set_timing_events.restype = None
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def _stream_handle(stream, device=None) -> int:
    """The raw handle of ``stream``: None is the current stream of ``device``
    (or of the current device); a torch stream must live on ``device``."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if device is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return stream.cuda_stream
    return int(stream)


def _on_device(device: torch.device):
    """The library launches on the current device, so each call makes the
    tensors' device current for its duration."""
    return torch.cuda.device(device) if device.type == "cuda" else contextlib.nullcontext()


def _shape4(t: torch.Tensor, name: str):
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, N, d], got {tuple(t.shape)}")
    return tuple(t.shape)


def _check(t: torch.Tensor, name: str, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")


def _raise(status: int, where: str):
    if status != FA_OK:
        raise FaError(status, where)


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(int(status)).decode()


def fa_set_wait_limit_ns(limit_ns: int) -> None:
    load_library().fa_set_wait_limit_ns(int(limit_ns))


def fa_debug_stall(enable: bool) -> None:
    """Test hook: kernels launched while enabled stall on a barrier nothing signals."""
    load_library().fa_debug_stall(int(bool(enable)))


def fa_set_bwd_pair_mma(enable: bool) -> None:
    """fa_bwd_deterministic at d = 128: dK, dV products as 2-CTA (256-row) MMAs on CTA pairs."""
    load_library().fa_set_bwd_pair_mma(int(bool(enable)))


def fa_set_exp2_split(soft_quarters: int) -> None:
    """0 (default): every forward exponential on the special-function unit;
    1 or 2: that many of every four pairs by the cubic 2^n p(f) on the FMA pipe."""
    _raise(load_library().fa_set_exp2_split(int(soft_quarters)), "fa_set_exp2_split")


def _event_handle(ev) -> int:
    if ev is None:
        return 0
    if isinstance(ev, torch.cuda.Event):
        if ev.cuda_event == 0:
            raise ValueError("record a torch.cuda.Event once before passing it (it is created lazily)")
        return ev.cuda_event
    return int(ev)


def fa_set_timing_events(fwd_start=None, fwd_stop=None, bwd_start=None, bwd_stop=None) -> None:
    """Events recorded around the forward kernel and the main backward kernel (profiling)."""
    load_library().fa_set_timing_events(_event_handle(fwd_start), _event_handle(fwd_stop),
                                        _event_handle(bwd_start), _event_handle(bwd_stop))


def fa_check_device_status(stream=None) -> int:
    """Synchronize the stream; return (and clear) the status word of the
    stream's device (of the current device for None or a raw handle)."""
    dev = stream.device if isinstance(stream, torch.cuda.Stream) else None
    with (torch.cuda.device(dev) if dev is not None else contextlib.nullcontext()):
        return int(load_library().fa_check_device_status(_stream_handle(stream)))


def fa_fwd(q, k, v, o, lse, scale: float, causal: bool, stream=None) -> None:
    """O and LSE of softmax(scale Q K^T) V; tensors [B,H,N,d] bf16 and [B,H,N] fp32."""
    B, H, N, d = _shape4(q, "q")
    dev = q.device
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _check(t, name, torch.bfloat16, (B, H, N, d), dev)
    _check(lse, "lse", torch.float32, (B, H, N), dev)
    with _on_device(dev):
        st = load_library().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                   B, H, N, d, float(scale), int(bool(causal)), _stream_handle(stream, dev))
    _raise(st, "fa_fwd")


def fa_fwd_fp8_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().fa_fwd_fp8_workspace_bytes(B, H, N, d))


def fa_fwd_fp8(q, k, v, signs, o, lse, workspace, scale: float, causal: bool, stream=None) -> None:
    """FP8 forward: Q, K rotated by diag(signs) H / sqrt(d) and quantised per
    128-row block, V per channel, E4M3 products; signs is an int8 device
    tensor of +1 / -1 [d]; workspace a uint8 device tensor."""
    B, H, N, d = _shape4(q, "q")
    dev = q.device
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _check(t, name, torch.bfloat16, (B, H, N, d), dev)
    _check(lse, "lse", torch.float32, (B, H, N), dev)
    _check(signs, "signs", torch.int8, (d,), dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    ws_bytes = workspace.numel() * workspace.element_size()
    with _on_device(dev):
        st = load_library().fa_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), signs.data_ptr(), o.data_ptr(),
                                       lse.data_ptr(), workspace.data_ptr(), ws_bytes, B, H, N, d, float(scale),
                                       int(bool(causal)), _stream_handle(stream, dev))
    _raise(st, "fa_fwd_fp8")


def fa_bwd_preprocess(o, dout, delta, stream=None) -> None:
    """delta = rowsum(dO * O) in fp32, [B,H,N]."""
    B, H, N, d = _shape4(o, "o")
    dev = o.device
    _check(o, "o", torch.bfloat16, (B, H, N, d), dev)
    _check(dout, "dout", torch.bfloat16, (B, H, N, d), dev)
    _check(delta, "delta", torch.float32, (B, H, N), dev)
    with _on_device(dev):
        st = load_library().fa_bwd_preprocess(o.data_ptr(), dout.data_ptr(), delta.data_ptr(), B, H, N, d,
                                              _stream_handle(stream, dev))
    _raise(st, "fa_bwd_preprocess")


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().fa_bwd_workspace_bytes(B, H, N, d))


def _bwd_call(entry: str, q, k, v, o, dout, lse, dq, dk, dv, workspace, scale: float, causal: bool, stream):
    B, H, N, d = _shape4(q, "q")
    dev = q.device
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, name, torch.bfloat16, (B, H, N, d), dev)
    _check(lse, "lse", torch.float32, (B, H, N), dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    ws_bytes = workspace.numel() * workspace.element_size()
    with _on_device(dev):
        st = getattr(load_library(), entry)(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                            dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                            dv.data_ptr(), workspace.data_ptr(), ws_bytes, B, H, N, d, float(scale),
                                            int(bool(causal)), _stream_handle(stream, dev))
    _raise(st, entry)


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale: float, causal: bool, stream=None) -> None:
    """dQ, dK, dV of attention by recomputation; workspace is a uint8 device tensor."""
    _bwd_call("fa_bwd", q, k, v, o, dout, lse, dq, dk, dv, workspace, scale, causal, stream)


def fa_bwd_deterministic(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale: float, causal: bool,
                         stream=None) -> None:
    """fa_bwd with dQ summed by a separate query-major pass: bitwise repeatable."""
    _bwd_call("fa_bwd_deterministic", q, k, v, o, dout, lse, dq, dk, dv, workspace, scale, causal, stream)


FA_STATIC_SCRATCH_BYTES = 72 * 1024 * 1024


def fa_bwd_static_scratch(q, k, v, o, dout, lse, dq, dk, dv, scale: float, causal: bool, stream=None) -> None:
    """fa_bwd without a workspace argument, for callers that cannot allocate device
    memory at call time: the scratch is a fixed array inside the library (see
    include/fa.h for the size limit, the first-call set-up and the rule that
    calls overlapping on the GPU race)."""
    B, H, N, d = _shape4(q, "q")
    dev = q.device
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, name, torch.bfloat16, (B, H, N, d), dev)
    _check(lse, "lse", torch.float32, (B, H, N), dev)
    with _on_device(dev):
        st = load_library().fa_bwd_static_scratch(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                                  dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                                  dv.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
                                                  _stream_handle(stream, dev))
    _raise(st, "fa_bwd_static_scratch")


# ---------------------------------------------------------------------------
# cross attention, attention over a cache, head norm and rotation
# ---------------------------------------------------------------------------
# Single tokens are launched every few microseconds, so the checks below look at
# each property once and leave the messages to _check; the library's device and
# stream are taken without a context manager where they are current already.
def _ptr(t, name: str, dtype, shape, device) -> int:
    """Address of a tensor, checked."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device.index or not t.is_contiguous():
        _check(t, name, dtype, shape, device)
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t.data_ptr()


def _given(t, name: str, dtype, shape, device) -> int:
    """Address of an optional tensor (0 for None), checked."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device.index or not t.is_contiguous():
        return _ptr(t, name, dtype, shape, device)
    return t.data_ptr()


@functools.lru_cache(maxsize=1)
def _only_device() -> bool:
    """Whether the process sees one GPU, which is then always the current one."""
    return torch.cuda.device_count() == 1


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(name: str, device: torch.device, stream, *args) -> None:
    """The entry point on (*args, stream) with the tensors' device current; raises on a status."""
    if device.type != "cuda":
        raise ValueError(f"{name} needs CUDA tensors, got {device}")
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(device.index)
    else:
        handle = _stream_handle(stream, device)
    if name not in _entries:
        _entries[name] = getattr(load_library(), name + "_packed"), _PACKED[name]
    entry, pack = _entries[name]
    try:
        packed = pack(*args, handle)
    except (struct.error, OverflowError, TypeError) as e:
        raise ValueError(f"{name}: {e}") from None  # a number that the C type does not hold
    if _only_device() or torch.cuda.current_device() == device.index:
        st = entry(packed)
    else:
        with torch.cuda.device(device):
            st = entry(packed)
    if st != FA_OK:
        raise FaError(st, name)


def _workspace(workspace, device):
    if workspace.get_device() != device.index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace.data_ptr(), workspace.nbytes


def _cross_sizes(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q and k must be [B, H, N, d], got {tuple(q.shape)} and {tuple(k.shape)}")
    B, H, Nq, d = q.shape
    _, Hkv, Nk, _ = k.shape
    return B, H, Hkv, Nq, Nk, d


@functools.lru_cache(maxsize=1024)
def fa_cross_fwd_workspace_bytes(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    return int(load_library().fa_cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d))


def fa_cross_fwd(q, k, v, key_lens, o, lse, workspace, scale: float, stream=None) -> None:
    """Attention of q [B,H,Nq,d] to k, v [B,Hkv,Nk,d] of another length; key_lens
    int32 [B] (or None: all Nk); o like q, lse [B,H,Nq] fp32."""
    B, H, Hkv, Nq, Nk, d = _cross_sizes(q, k)
    dev, bf, rows, keys = q.device, torch.bfloat16, (B, H, Nq, d), (B, Hkv, Nk, d)
    _call("fa_cross_fwd", dev, stream, _ptr(q, "q", bf, rows, dev),
          _ptr(k, "k", bf, keys, dev), _ptr(v, "v", bf, keys, dev),
          _given(key_lens, "key_lens", torch.int32, (B,), dev), _ptr(o, "o", bf, rows, dev),
          _ptr(lse, "lse", torch.float32, (B, H, Nq), dev), *_workspace(workspace, dev), B, H, Hkv, Nq, Nk, d, scale)


@functools.lru_cache(maxsize=1024)
def fa_cross_bwd_workspace_bytes(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    return int(load_library().fa_cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d))


def fa_cross_bwd(q, k, v, key_lens, o, dout, lse, dq, dk, dv, workspace, scale: float, stream=None) -> None:
    """dQ, dK, dV of fa_cross_fwd by recomputation; dk, dv like k, v."""
    B, H, Hkv, Nq, Nk, d = _cross_sizes(q, k)
    dev, bf, rows, keys = q.device, torch.bfloat16, (B, H, Nq, d), (B, Hkv, Nk, d)
    _call("fa_cross_bwd", dev, stream, _ptr(q, "q", bf, rows, dev),
          _ptr(k, "k", bf, keys, dev), _ptr(v, "v", bf, keys, dev),
          _given(key_lens, "key_lens", torch.int32, (B,), dev), _ptr(o, "o", bf, rows, dev),
          _ptr(dout, "dout", bf, rows, dev), _ptr(lse, "lse", torch.float32, (B, H, Nq), dev),
          _ptr(dq, "dq", bf, rows, dev), _ptr(dk, "dk", bf, keys, dev), _ptr(dv, "dv", bf, keys, dev), *_workspace(workspace, dev),
          B, H, Hkv, Nq, Nk, d, scale)


@functools.lru_cache(maxsize=1024)
def fa_tree_fwd_workspace_bytes(B: int, H: int, Hkv: int, T: int, C: int, d: int) -> int:
    return int(load_library().fa_tree_fwd_workspace_bytes(B, H, Hkv, T, C, d))


def fa_tree_fwd(q, k_cache, v_cache, cache_lens, draft_lens, draft_masks, o, lse, workspace, scale: float,
                stream=None) -> None:
    """Attention of T new tokens q [B,H,T,d] over a cache [B,Hkv,C,d] that holds
    cache_lens[b] tokens and then the new ones.  draft_lens int32 [B] (or
    None: T); draft_masks int64 [B,T], bit t of word n: token n sees token t
    (or None: each sees the ones before it and itself; see tree_masks)."""
    B, H, Hkv, T, C, d = _cross_sizes(q, k_cache)
    dev, bf, rows, keys = q.device, torch.bfloat16, (B, H, T, d), (B, Hkv, C, d)
    _call("fa_tree_fwd", dev, stream, _ptr(q, "q", bf, rows, dev),
          _ptr(k_cache, "k_cache", bf, keys, dev), _ptr(v_cache, "v_cache", bf, keys, dev),
          _ptr(cache_lens, "cache_lens", torch.int32, (B,), dev),
          _given(draft_lens, "draft_lens", torch.int32, (B,), dev),
          _given(draft_masks, "draft_masks", torch.int64, (B, T), dev), _ptr(o, "o", bf, rows, dev),
          _ptr(lse, "lse", torch.float32, (B, H, T), dev), *_workspace(workspace, dev), B, H, Hkv, T, C, d, scale)


def tree_masks(parents: torch.Tensor) -> torch.Tensor:
    """draft_masks of fa_tree_fwd for trees given by parents int [B,T]: parents[b,n]
    is the token that n was drafted after (always an earlier one), or -1 for
    one that follows the request's own tokens.  On the tensor's device."""
    if parents.dim() != 2 or parents.dtype not in (torch.int32, torch.int64):
        raise ValueError("parents must be int32 or int64 [B, T]")
    B, T = parents.shape
    if T > 64:
        raise ValueError("at most 64 drafted tokens have masks")
    place = torch.arange(T, device=parents.device)
    if bool(((parents < -1) | (parents >= place)).any()):
        raise ValueError("a parent must be -1 or an earlier token")
    words = torch.zeros((B, T), dtype=torch.int64, device=parents.device)
    for n in range(T):
        up = torch.gather(words, 1, parents[:, n:n + 1].long().clamp(min=0))[:, 0]
        words[:, n] = torch.where(parents[:, n] >= 0, up, 0) | (1 << n if n < 63 else -(1 << 63))
    return words


def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, scale: float = 1.0,
                     trained_len: int = 0, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(inv_freq, factor) of fa_rope_fwd: frequencies base^(-2i/rotary_dim) in fp64, and
    the factor of the rotated values.  For contexts ``scale`` times the trained one:
    ``"linear"`` divides every frequency by scale; ``"base"`` raises the base to
    base * scale^(rotary_dim / (rotary_dim - 2)), which slows the lowest frequency
    by scale and leaves the highest; ``"parts"`` keeps frequencies that turn at
    least ``fast`` times over trained_len positions, divides by scale those that
    turn at most ``slow`` times, blends between, with factor 0.1 ln(scale) + 1."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not base > 1.0 or not scale >= 1.0:
        raise ValueError("base must be above 1 and scale at least 1")
    factor = 1.0
    if scaling == "base":
        if rotary_dim == 2:
            raise ValueError("scaling by the base needs rotary_dim above 2")
        base = base * scale ** (rotary_dim / (rotary_dim - 2))
    freq = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    if scaling == "linear":
        freq = freq / scale
    elif scaling == "parts":
        if trained_len < 1 or not fast > slow > 0:
            raise ValueError("scaling by parts needs trained_len and fast > slow > 0")
        turns = trained_len * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        freq = freq * (keep + (1.0 - keep) / scale)
        factor = 0.1 * math.log(scale) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(device), factor


_NO_ROWS = (0, 0, 0, 0)


def _rows(t, name: str, shape, device):
    """``fa_rows`` (address and strides) of a [B, N, heads, d] tensor whose d values lie
    next to each other; None: no such rows."""
    if t is None:
        return _NO_ROWS
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    sb, sn, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must have its last dimension contiguous")
    if t.get_device() != device.index:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    # (the stride of a dimension of one is any number: it is never used)
    return t.data_ptr(), sb if shape[0] > 1 else 0, sn if shape[1] > 1 else 0, sh if shape[2] > 1 else 0


def _rope_sizes(q, k, v, names):
    """B, N, H, Hkv, d and device of the token-major tensors that are given."""
    kv = k if k is not None else v
    first = q if q is not None else kv
    if first is None:
        raise ValueError(f"one of {', '.join(names)} must be given")
    if first.dim() != 4 or (kv is not None and kv.dim() != 4):
        raise ValueError(f"{', '.join(names)} must be [B, N, heads, d]")
    B, N, _, d = first.shape
    return B, N, (q.shape[2] if q is not None else 1), (kv.shape[2] if kv is not None else 1), d, first.device


def _frequencies(inv_freq, device):
    if inv_freq is None:
        return 0, 0
    n = inv_freq.numel()
    return _ptr(inv_freq, "inv_freq", torch.float64, (n,), device), 2 * n


def fa_rope_fwd(q, k, v, q_weight, k_weight, inv_freq, positions, starts, q_out, k_out, v_out, *, eps=None,
                factor: float = 1.0, interleaved: bool = False, stream=None) -> None:
    """RMS norm of each head (with eps; None: no norm) and rotation of the first
    2 * len(inv_freq) values by position: q [B,N,H,d], k and v [B,N,Hkv,d] (any
    strides with d contiguous) into q_out [B,H,N,d] and rows starts[b].. of
    k_out, v_out [B,Hkv,C,d].  q, k or v may be None with its output; weights
    fp32 [d] or None; inv_freq fp64 or None (no rotation); positions int32
    [B,N] or None (starts[b] + n); starts int32 [B] or None (0)."""
    B, N, H, Hkv, d, dev = _rope_sizes(q, k, v, ("q", "k", "v"))
    if eps is None and (q_weight is not None or k_weight is not None):
        raise ValueError("weights need eps: without it there is no norm")
    cache = k_out if k_out is not None else v_out
    C = N if cache is None else _shape4(cache, "k_out")[2]
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    freq, rot = _frequencies(inv_freq, dev)
    _call("fa_rope_fwd", dev, stream, *_rows(q, "q", (B, N, H, d), dev),
          *_rows(k, "k", (B, N, Hkv, d), dev), *_rows(v, "v", (B, N, Hkv, d), dev),
          _given(q_weight, "q_weight", f32, (d,), dev), _given(k_weight, "k_weight", f32, (d,), dev), freq,
          _given(positions, "positions", i32, (B, N), dev), _given(starts, "starts", i32, (B,), dev),
          _given(q_out, "q_out", bf, (B, H, N, d), dev), _given(k_out, "k_out", bf, (B, Hkv, C, d), dev),
          _given(v_out, "v_out", bf, (B, Hkv, C, d), dev), B, N, H, Hkv, C, d, rot, 0 if eps is None else 1,
          eps or 0.0, factor, 1 if interleaved else 0)


@functools.lru_cache(maxsize=1024)
def fa_rope_bwd_workspace_bytes(B: int, H: int, Hkv: int, N: int, d: int) -> int:
    return int(load_library().fa_rope_bwd_workspace_bytes(B, H, Hkv, N, d))


def fa_rope_bwd(q, k, q_weight, k_weight, inv_freq, positions, dq_out, dk_out, dv_out, dq, dk, dv, dq_weight,
                dk_weight, workspace=None, *, eps=None, factor: float = 1.0, interleaved: bool = False,
                stream=None) -> None:
    """Gradients of fa_rope_fwd (without starts): dq_out [B,H,N,d], dk_out and dv_out
    [B,Hkv,N,d] into token-major dq, dk, dv like q, k, v, and fp32 dq_weight,
    dk_weight [d] (or None).  q and k are read only with eps; any of the three
    gradients may be None with its output; workspace is needed for weights."""
    B, N, H, Hkv, d, dev = _rope_sizes(dq, dk, dv, ("dq", "dk", "dv"))
    if eps is None and any(t is not None for t in (q_weight, k_weight, dq_weight, dk_weight)):
        raise ValueError("weights need eps: without it there is no norm")
    norm = eps is not None
    bf, f32 = torch.bfloat16, torch.float32
    freq, rot = _frequencies(inv_freq, dev)
    ws, ws_bytes = (0, 0) if workspace is None else _workspace(workspace, dev)
    _call("fa_rope_bwd", dev, stream,
          *(_rows(q, "q", (B, N, H, d), dev) if norm and dq is not None else _NO_ROWS),
          *(_rows(k, "k", (B, N, Hkv, d), dev) if norm and dk is not None else _NO_ROWS),
          _given(q_weight, "q_weight", f32, (d,), dev), _given(k_weight, "k_weight", f32, (d,), dev), freq,
          _given(positions, "positions", torch.int32, (B, N), dev),
          _given(dq_out, "dq_out", bf, (B, H, N, d), dev), _given(dk_out, "dk_out", bf, (B, Hkv, N, d), dev),
          _given(dv_out, "dv_out", bf, (B, Hkv, N, d), dev), *_rows(dq, "dq", (B, N, H, d), dev),
          *_rows(dk, "dk", (B, N, Hkv, d), dev), *_rows(dv, "dv", (B, N, Hkv, d), dev),
          _given(dq_weight, "dq_weight", f32, (d,), dev), _given(dk_weight, "dk_weight", f32, (d,), dev), ws, ws_bytes,
          B, N, H, Hkv, d, rot, 1 if norm else 0, eps or 0.0, factor, 1 if interleaved else 0)


# ---------------------------------------------------------------------------
# conveniences that allocate the outputs with torch and call the entry points.
# With check_status (the default) they wait for the work and raise FaError if
# a kernel reported a timeout, so what they return is known to be valid; pass
# check_status=False to keep the call asynchronous and check later with
# fa_check_device_status.  Outputs and workspaces are allocated (and filled) on
# the call's stream, and outputs are marked as used on the current one too, so that
# neither stream gets memory back that the other still works on.
# ---------------------------------------------------------------------------
@contextlib.contextmanager
def _allocating(stream, device: torch.device):
    """Makes ``stream`` current; yields a function that marks tensors made there as
    used on the stream that was current before."""
    if stream is None or device.type != "cuda":
        yield lambda *tensors: None
        return
    handle = _stream_handle(stream, device)
    if not isinstance(stream, torch.cuda.Stream):
        # (0 and 1 are both the legacy default stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle > 1 else torch.cuda.default_stream(device)
    before = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        yield lambda *tensors: [t.record_stream(before) for t in tensors] if before != stream else None


def _checked(stream, device, where: str):
    with _on_device(device):
        st = int(load_library().fa_check_device_status(_stream_handle(stream, device)))
    _raise(st, where)


def attention_forward(q, k, v, scale: float, causal: bool = False, stream=None, check_status: bool = True):
    B, H, N, d = _shape4(q, "q")
    with _allocating(stream, q.device) as used:
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
        used(o, lse)
        fa_fwd(q, k, v, o, lse, scale, causal, stream)
    if check_status:
        _checked(stream, q.device, "attention_forward")
    return o, lse


def attention_forward_fp8(q, k, v, signs, scale: float, causal: bool = False, workspace=None, stream=None,
                          check_status: bool = True):
    B, H, N, d = _shape4(q, "q")
    with _allocating(stream, q.device) as used:
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
        used(o, lse)
        if workspace is None:
            workspace = torch.empty(fa_fwd_fp8_workspace_bytes(B, H, N, d), dtype=torch.uint8, device=q.device)
        fa_fwd_fp8(q, k, v, signs, o, lse, workspace, scale, causal, stream)
    if check_status:
        _checked(stream, q.device, "attention_forward_fp8")
    return o, lse


def attention_backward(q, k, v, o, dout, lse, scale: float, causal: bool = False, workspace=None, stream=None,
                       deterministic: bool = False, check_status: bool = True):
    B, H, N, d = _shape4(q, "q")
    with _allocating(stream, q.device) as used:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        used(dq, dk, dv)
        if workspace is None:
            workspace = torch.empty(fa_bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8, device=q.device)
        (fa_bwd_deterministic if deterministic else fa_bwd)(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale, causal,
                                                            stream)
    if check_status:
        _checked(stream, q.device, "attention_backward")
    return dq, dk, dv


def cross_attention_forward(q, k, v, scale: float, key_lens=None, workspace=None, stream=None,
                            check_status: bool = True):
    B, H, Nq, d = _shape4(q, "q")
    _, Hkv, Nk, _ = _shape4(k, "k")
    with _allocating(stream, q.device) as used:
        o = torch.empty_like(q)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        used(o, lse)
        if workspace is None:
            workspace = torch.empty(fa_cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d), dtype=torch.uint8, device=q.device)
        fa_cross_fwd(q, k, v, key_lens, o, lse, workspace, scale, stream)
    if check_status:
        _checked(stream, q.device, "cross_attention_forward")
    return o, lse


def cross_attention_backward(q, k, v, o, dout, lse, scale: float, key_lens=None, workspace=None, stream=None,
                             check_status: bool = True):
    B, H, Nq, d = _shape4(q, "q")
    _, Hkv, Nk, _ = _shape4(k, "k")
    with _allocating(stream, q.device) as used:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        used(dq, dk, dv)
        if workspace is None:
            workspace = torch.empty(fa_cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d), dtype=torch.uint8, device=q.device)
        fa_cross_bwd(q, k, v, key_lens, o, dout, lse, dq, dk, dv, workspace, scale, stream)
    if check_status:
        _checked(stream, q.device, "cross_attention_backward")
    return dq, dk, dv


def tree_attention_forward(q, k_cache, v_cache, cache_lens, scale: float, draft_lens=None, draft_masks=None,
                           workspace=None, stream=None, check_status: bool = True):
    """Rows of tokens that a request does not have come out as O = 0, LSE = -inf."""
    B, H, T, d = _shape4(q, "q")
    _, Hkv, C, _ = _shape4(k_cache, "k_cache")
    with _allocating(stream, q.device) as used:
        o = torch.zeros_like(q)
        lse = torch.full((B, H, T), -math.inf, dtype=torch.float32, device=q.device)
        used(o, lse)
        if workspace is None:
            workspace = torch.empty(fa_tree_fwd_workspace_bytes(B, H, Hkv, T, C, d), dtype=torch.uint8, device=q.device)
        fa_tree_fwd(q, k_cache, v_cache, cache_lens, draft_lens, draft_masks, o, lse, workspace, scale, stream)
    if check_status:
        _checked(stream, q.device, "tree_attention_forward")
    return o, lse
