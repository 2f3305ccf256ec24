"""Python binding of libringattn (GB300 / sm_103a blockwise ring attention).

Every call marshals torch tensors into the C ABI declared in
``include/ringattn.h`` and launches the library's CUDA kernels on the current
torch stream.  torch only provides device memory and streams; no step of the
computation runs in Python or in torch.  There is no fallback: if the shared
library is missing or a tensor is not on a CUDA device the call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import math
import os

import torch

__all__ = [
    "LAYOUTS", "RingAttnError", "lib_path", "load", "ring_attn_fwd", "ring_attn_fwd_step", "ring_attn_bwd",
    "ring_attn_varlen_fwd", "ring_attn_varlen_bwd", "lse_merge", "ring_attn_permute", "ring_attn_unpermute",
    "ring_attn_workspace_size", "ring_attn_check_device_error", "ring_attn_set_knob", "ring_attn_version",
    "ring_attn_timing_enable", "ring_attn_timing_read", "ring_attn_bwd_static_scratch", "EXPORTED_SYMBOLS",
    "KERNELS", "RA_STATIC_SCRATCH_BYTES", "ring_attn_qkvpacked_fwd", "ring_attn_qkvpacked_bwd", "ring_attn_kvpacked_fwd",
    "ring_attn_kvpacked_bwd", "ring_attn_varlen_qkvpacked_fwd", "ring_attn_varlen_qkvpacked_bwd",
    "ring_attn_varlen_kvpacked_fwd", "ring_attn_varlen_kvpacked_bwd", "ring_attn_varlen_permute",
    "ring_attn_varlen_unpermute", "ring_attn_llama3_varlen_fwd", "ring_attn_llama3_varlen_bwd", "CuSeqlens",
    "KVCache", "ring_attn_cache_append", "ring_attn_cache_read", "ring_attn_cache_fwd", "ring_attn_cache_workspace_size",
    "ring_attn_cache_workspace", "Scores", "ring_attn_rope", "ring_attn_rope_bwd",
]

LAYOUTS = {"contiguous": 0, "zigzag": 1, "stripe": 2}
RA_BF16, RA_FP32, RA_E2M1X2, RA_E4M3 = 0, 1, 2, 3
RA_OP_FWD, RA_OP_BWD = 0, 1
RA_KNOB_WAIT_LIMIT_NS, RA_KNOB_DEBUG_FLAGS, RA_KNOB_DKDV_PAIR = 0, 1, 2

# Every extern "C" symbol include/ringattn.h declares.
EXPORTED_SYMBOLS = (
    "ring_attn_fwd", "ring_attn_fwd_step", "lse_merge", "ring_attn_bwd", "ring_attn_varlen_fwd",
    "ring_attn_varlen_bwd", "ring_attn_permute", "ring_attn_unpermute", "ring_attn_workspace_size",
    "ring_attn_check_device_error", "ring_attn_set_knob", "ring_attn_timing_enable", "ring_attn_timing_read",
    "ra_status_string", "ring_attn_version", "ring_attn_bwd_static_scratch", "ring_attn_varlen_permute",
    "ring_attn_varlen_unpermute", "ring_attn_llama3_varlen_fwd", "ring_attn_llama3_varlen_bwd",
    "ring_attn_debug_bounds", "ring_attn_varlen_workspace_size", "ring_attn_cache_append", "ring_attn_cache_read",
    "ring_attn_cache_fwd", "ring_attn_cache_workspace_size", "ring_attn_rope", "ring_attn_scored_fwd",
    "ring_attn_scored_fwd_step", "ring_attn_scored_bwd", "ring_attn_scored_varlen_fwd", "ring_attn_scored_varlen_bwd",
    "ring_attn_scored_llama3_varlen_fwd", "ring_attn_scored_llama3_varlen_bwd", "ring_attn_scored_cache_fwd",
)
RA_STATIC_SCRATCH_BYTES = 16 << 20
KERNELS = {"fwd": 0, "bwd_dkdv": 1, "bwd_pre": 2, "bwd_dq": 3, "permute": 4, "lse_merge": 5, "cache_append": 6,
           "cache_read": 7, "cache_fwd": 8, "cache_join": 9}
_KINDS = {**KERNELS, "rope": 10}


class RingAttnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class _KVCache(ctypes.Structure):
    _fields_ = [("k", _Tensor), ("k_scale", _Tensor), ("v", _Tensor), ("v_scale", _Tensor)]


class _KVSeqs(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("page_table_stride", ctypes.c_int64), ("kv_lens", ctypes.c_void_p),
                ("cu_seqlens_dev", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p),
                ("max_pages", ctypes.c_int32), ("n_seqs", ctypes.c_int32)]


class _Scores(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p)]


class _RopePositions(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("stride_axis", ctypes.c_int64), ("stride_b", ctypes.c_int64),
                ("stride_s", ctypes.c_int64), ("pair_axis", ctypes.c_void_p), ("n_axes", ctypes.c_int32)]


_LIB = None


def lib_path() -> str:
    """libringattn.so, or the debug-bounds variant libringattn_dbg.so when
    RA_LIB_VARIANT=debug_bounds (build it with build(debug_bounds=True))."""
    variant = os.environ.get("RA_LIB_VARIANT", "")
    if variant not in ("", "debug_bounds"):
        raise ValueError(f"RA_LIB_VARIANT={variant!r}: expected 'debug_bounds' or unset")
    name = "libringattn_dbg.so" if variant == "debug_bounds" else "libringattn.so"
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), name)


def load():
    """Loads libringattn.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with ring_attn_gb300.build.build() "
                           "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(path)
    P, I32, I64, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    T = ctypes.POINTER(_Tensor)
    C, S = ctypes.POINTER(_KVCache), ctypes.POINTER(_KVSeqs)
    Z = ctypes.POINTER(_Scores)
    sig = {
        "ring_attn_fwd": [T, T, T, I32, I32, I32, F32, T, T, P, SZ, P],
        "ring_attn_fwd_step": [T, T, T, I32, I32, I32, F32, I32, T, T, P],
        "lse_merge": [T, T, T, T, P],
        "ring_attn_bwd": [T, T, T, T, T, T, I32, I32, I32, F32, T, T, T, P, SZ, P],
        "ring_attn_bwd_static_scratch": [T, T, T, T, T, T, I32, I32, I32, F32, T, T, T, P],
        "ring_attn_varlen_fwd": [T, T, T, P, P, I32, I32, I32, I32, I32, F32, T, T, P, SZ, P],
        "ring_attn_varlen_bwd": [T, T, T, T, T, T, P, P, I32, I32, I32, I32, I32, F32, T, T, T, P, SZ, P],
        "ring_attn_varlen_permute": [T, T, P, P, I32, I32, I32, I32, P],
        "ring_attn_llama3_varlen_fwd": [T, T, T, P, P, I32, I32, I32, I32, I32, F32, T, T, P],
        "ring_attn_llama3_varlen_bwd": [T, T, T, T, T, T, P, P, I32, I32, I32, I32, I32, F32, T, T, T, P, SZ, P],
        "ring_attn_varlen_unpermute": [T, T, P, P, I32, I32, I32, I32, P],
        "ring_attn_permute": [T, T, I32, I32, I32, P],
        "ring_attn_unpermute": [T, T, I32, I32, I32, P],
        "ring_attn_cache_append": [T, T, T, T, T, I32, P, C, S, T, P],
        "ring_attn_cache_read": [C, S, T, T, P],
        "ring_attn_cache_fwd": [T, C, S, I32, F32, I32, T, T, P, SZ, P],
        "ring_attn_rope": [T, T, T, T, I32, ctypes.POINTER(_RopePositions), I32, I32, I32, T, T, P],
        "ring_attn_scored_fwd": [T, T, T, I32, I32, I32, F32, Z, T, T, P],
        "ring_attn_scored_fwd_step": [T, T, T, I32, I32, I32, F32, Z, I32, T, T, P],
        "ring_attn_scored_bwd": [T, T, T, T, T, T, I32, I32, I32, F32, Z, T, T, T, P, SZ, P],
        "ring_attn_scored_varlen_fwd": [T, T, T, P, P, I32, I32, I32, I32, I32, F32, Z, T, T, P, SZ, P],
        "ring_attn_scored_varlen_bwd": [T, T, T, T, T, T, P, P, I32, I32, I32, I32, I32, F32, Z, T, T, T, P, SZ, P],
        "ring_attn_scored_llama3_varlen_fwd": [T, T, T, P, P, I32, I32, I32, I32, I32, F32, Z, T, T, P],
        "ring_attn_scored_llama3_varlen_bwd": [T, T, T, T, T, T, P, P, I32, I32, I32, I32, I32, F32, Z, T, T, T, P, SZ,
                                               P],
        "ring_attn_scored_cache_fwd": [T, C, S, I32, F32, Z, I32, T, T, P, SZ, P],
        "ring_attn_check_device_error": [P, ctypes.POINTER(I32)],
        "ring_attn_set_knob": [I32, I64],
        "ring_attn_timing_enable": [I32],
        "ring_attn_timing_read": [I32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I64)],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = I32
    lib.ring_attn_workspace_size.argtypes = [I32, I64, I64, I64, I64, I32]
    lib.ring_attn_workspace_size.restype = SZ
    lib.ring_attn_varlen_workspace_size.argtypes = [I32, I64, I64, I64, I32, I32]
    lib.ring_attn_varlen_workspace_size.restype = SZ
    lib.ring_attn_cache_workspace_size.argtypes = [I64, I64, I64, I64, I64, I32]
    lib.ring_attn_cache_workspace_size.restype = SZ
    lib.ra_status_string.argtypes = [I32]
    lib.ra_status_string.restype = ctypes.c_char_p
    lib.ring_attn_version.argtypes = []
    lib.ring_attn_version.restype = I32
    lib.ring_attn_debug_bounds.argtypes = []
    lib.ring_attn_debug_bounds.restype = I32
    _LIB = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        msg = load().ra_status_string(status).decode()
        raise RingAttnError(status, f"{what}: {msg}")


def _layout(layout) -> int:
    if isinstance(layout, str):
        if layout not in LAYOUTS:
            raise ValueError(f"unknown layout {layout!r}")
        return LAYOUTS[layout]
    return int(layout)


def _t(x: torch.Tensor) -> _Tensor:
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("ring_attn_gb300 takes CUDA tensors only")
    if x.dtype == torch.bfloat16:
        dt = RA_BF16
    elif x.dtype == torch.float32:
        dt = RA_FP32
    else:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if x.dim() > 4 or x.dim() < 1:
        raise ValueError("tensors must have 1 to 4 dimensions")
    t = _Tensor()
    t.data = x.data_ptr()
    t.dtype = dt
    t.ndim = x.dim()
    for i in range(x.dim()):
        t.shape[i] = x.shape[i]
        t.stride[i] = x.stride(i)
    return t


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _scale(scale, d):
    return float(1.0 / math.sqrt(d) if scale is None else scale)


class Scores:
    """What a model does to its scores besides the product, for the `scores` argument of the attention calls.

    With x = softmax_scale * q.k of tokens i and j (of a sequence, whatever the layout):
    softcap: y = softcap * tanh(x / softcap), 2^-10 to 2^20 (0: y = x).
    slopes: (h,) fp32, one per query head: z = y - slopes[h] * |i - j|.
    prefix: (b,) int32, or (n_seqs,) for varlen and cache calls: with causal, every token of a
    sequence sees its first prefix tokens, so that those see each other both ways.
    out, lse and the gradients of q, k and v are those of attention with z; softcap and slopes
    are constants.  The handle keeps the tensors; the kernels read their contents (so a captured call
    follows them), from where the tensors are at the call.  Other tensors are another handle."""

    softcap, slopes, prefix = (property(lambda self, i=i: self._parts[i]) for i in range(3))

    def __init__(self, softcap=0.0, slopes=None, prefix=None):
        self._parts = (float(softcap), slopes, prefix)
        self._check()
        if slopes is not None and prefix is not None and slopes.device != prefix.device:
            raise ValueError("slopes and prefix must be on one device")

    def __reduce__(self):  # copies and pickles describe their own tensors
        return type(self), self._parts

    @property
    def device(self):
        return next((x.device for x in self._parts[1:] if x is not None), None)

    def _check(self):
        for name, x, dtype in (("slopes", self.slopes, torch.float32), ("prefix", self.prefix, torch.int32)):
            if x is None:
                continue
            if not isinstance(x, torch.Tensor) or not x.is_cuda:
                raise ValueError("ring_attn_gb300 takes CUDA tensors only")
            if x.dtype != dtype or x.dim() != 1 or not x.is_contiguous():
                raise ValueError(f"{name} must be a contiguous 1-D {dtype} tensor")

    def _arg(self, device, h, n):
        """The C argument for a call of h query heads and n batches or sequences on the device."""
        self._check()
        for name, x, m, of in (("slopes", self.slopes, h, "query heads"), ("prefix", self.prefix, n, "sequences")):
            if x is None:
                continue
            if x.device != device:
                raise ValueError(f"scores on {x.device}, call on {device}")
            if x.numel() != m:
                raise ValueError(f"{name} must have one entry for each of the {m} {of}")
        return ctypes.byref(_Scores(self.softcap, None if self.slopes is None else self.slopes.data_ptr(),
                                    None if self.prefix is None else self.prefix.data_ptr()))


def _place(scores, q, stream):
    """Where a call with scores runs and allocates: the stream given, or q's device."""
    if scores is None:
        return contextlib.nullcontext()
    if not isinstance(scores, Scores):
        raise ValueError("scores must be a Scores")
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("ring_attn_gb300 takes CUDA tensors only")
    if stream is None:
        return torch.cuda.device(q.device)
    if stream.device != q.device:
        raise ValueError(f"stream on {stream.device}, q on {q.device}")
    return torch.cuda.stream(stream)


def _of(scores):
    if not isinstance(scores, Scores):
        raise ValueError("scores must be a Scores")
    return scores._parts


def _scored_call(name, q, stream, *args):
    """Runs a call of the compiled marshaller on the given stream (None: the current one of q's device); its results."""
    f = getattr(_EXT or _ext(), name)
    if stream is None:
        r = f(*args)
    else:
        if isinstance(q, torch.Tensor) and stream.device != q.device:
            raise ValueError(f"stream on {stream.device}, q on {q.device}")
        with torch.cuda.stream(stream):  # outputs and workspace belong to it, too
            r = f(*args)
    if r[0] != 0:
        _check(r[0], "ring_attn_" + name)
    return r[1:]


def _cu_arrays(cu_seqlens, q, stream):
    """(device, host) arrays of cu_seqlens, copied where q is if it is not a CuSeqlens."""
    if not isinstance(cu_seqlens, CuSeqlens):
        if not isinstance(q, torch.Tensor) or not q.is_cuda:
            raise ValueError("ring_attn_gb300 takes CUDA tensors only")
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(q.device):
            cu_seqlens = CuSeqlens(cu_seqlens, q.device)
    return cu_seqlens.dev, cu_seqlens.host


def _call(name, scores, device, h, n, at, *args):
    """lib.ring_attn_<name>(*args), or its scored form with the scores at place `at`; checks the status."""
    if scores is None:
        _check(getattr(load(), "ring_attn_" + name)(*args), "ring_attn_" + name)
    else:
        z = scores._arg(device, h, n)
        _check(getattr(load(), "ring_attn_scored_" + name)(*args[:at], z, *args[at:]), "ring_attn_scored_" + name)


def ring_attn_fwd(q, k, v, layout="contiguous", n_shards=1, causal=False, softmax_scale=None, out=None, lse=None,
                  stream=None, scores=None):
    """Ring forward with the fp32 LSE merge fused.  q, k, v: (b, h, s, d) bf16 in layout order
    (k and v may have hk heads, hk dividing h: query head i uses key / value head i // (h // hk)).
    scores: a Scores, or None for plain ones.

    Returns (out (b, h, s, d) bf16, lse (b, h, s) fp32), both in layout order."""
    if scores is not None:
        return _scored_call("scored_fwd", q, stream, q, k, v, _layout(layout), n_shards, causal,
                            _scale(softmax_scale, q.shape[-1]), _of(scores), out, lse)
    lib = load()
    b, h, s, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((b, h, s), dtype=torch.float32, device=q.device)
    tq, tk, tv, to, tl = _t(q), _t(k), _t(v), _t(out), _t(lse)
    _check(lib.ring_attn_fwd(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv), _layout(layout), int(n_shards),
                             int(bool(causal)), _scale(softmax_scale, d), ctypes.byref(to), ctypes.byref(tl),
                             None, 0, _stream(stream)), "ring_attn_fwd")
    return out, lse


def ring_attn_fwd_step(q, k, v, step, layout="contiguous", n_shards=1, causal=False, softmax_scale=None,
                       out_blk=None, lse_blk=None, out_dtype=torch.float32, stream=None, scores=None):
    """One ring step: every Q shard r against KV shard (r - step) mod N; block out and lse."""
    load()
    with _place(scores, q, stream):
        b, h, s, d = q.shape
        if out_blk is None:
            out_blk = torch.empty((b, h, s, d), dtype=out_dtype, device=q.device)
        if lse_blk is None:
            lse_blk = torch.empty((b, h, s), dtype=torch.float32, device=q.device)
        tq, tk, tv, to, tl = _t(q), _t(k), _t(v), _t(out_blk), _t(lse_blk)
        _call("fwd_step", scores, q.device, h, b, 7, ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
              _layout(layout), int(n_shards), int(bool(causal)), _scale(softmax_scale, d), int(step),
              ctypes.byref(to), ctypes.byref(tl), _stream(stream))
    return out_blk, lse_blk


def lse_merge(out_acc, lse_acc, out_blk, lse_blk, stream=None):
    """In-place merge of a block result into (out_acc fp32, lse_acc fp32)."""
    lib = load()
    a, b_, c, d = _t(out_acc), _t(lse_acc), _t(out_blk), _t(lse_blk)
    _check(lib.lse_merge(ctypes.byref(a), ctypes.byref(b_), ctypes.byref(c), ctypes.byref(d), _stream(stream)),
           "lse_merge")
    return out_acc, lse_acc


def ring_attn_workspace_size(op, b, h, s, d, n_shards=1) -> int:
    return int(load().ring_attn_workspace_size(int(op), int(b), int(h), int(s), int(d), int(n_shards)))


def ring_attn_varlen_workspace_size(op, total, h, d, layout="contiguous", n_shards=1) -> int:
    """Bytes of a varlen call's workspace (for zigzag: the original-order copies, see the C header)."""
    return int(load().ring_attn_varlen_workspace_size(int(op), int(total), int(h), int(d), _layout(layout),
                                                      int(n_shards)))


def _ws_arg(workspace):
    """(pointer, bytes) of an optional workspace tensor."""
    if workspace is None:
        return None, 0
    return ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()


def ring_attn_bwd(dout, q, k, v, out, lse, layout="contiguous", n_shards=1, causal=False, softmax_scale=None,
                  dq=None, dk=None, dv=None, workspace=None, stream=None, scores=None):
    """Gradients (dq like q, dk and dv like k and v), bf16, layout order; scores as in the forward."""
    if scores is not None:
        return _scored_call("scored_bwd", q, stream, dout, q, k, v, out, lse, _layout(layout), n_shards, causal,
                            _scale(softmax_scale, q.shape[-1]), _of(scores), dq, dk, dv, workspace)
    lib = load()
    b, h, s, d = q.shape
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ws_bytes = ring_attn_workspace_size(RA_OP_BWD, b, h, s, d, n_shards)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ts = [_t(x) for x in (dout, q, k, v, out, lse, dq, dk, dv)]
    r = [ctypes.byref(x) for x in ts]
    _check(lib.ring_attn_bwd(r[0], r[1], r[2], r[3], r[4], r[5], _layout(layout), int(n_shards), int(bool(causal)),
                             _scale(softmax_scale, d), r[6], r[7], r[8], ctypes.c_void_p(workspace.data_ptr()),
                             workspace.numel() * workspace.element_size(), _stream(stream)), "ring_attn_bwd")
    return dq, dk, dv


def ring_attn_bwd_static_scratch(dout, q, k, v, out, lse, layout="contiguous", n_shards=1, causal=False,
                                 softmax_scale=None, dq=None, dk=None, dv=None, stream=None):
    """ring_attn_bwd with the library's static device scratch instead of a workspace.

    The library call allocates nothing; only the outputs this wrapper creates when
    dq, dk or dv is None are allocated here, so callers that cannot allocate pass
    all three.  Calls that may overlap on the GPU race on the shared scratch."""
    lib = load()
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ts = [_t(x) for x in (dout, q, k, v, out, lse, dq, dk, dv)]
    r = [ctypes.byref(x) for x in ts]
    _check(lib.ring_attn_bwd_static_scratch(r[0], r[1], r[2], r[3], r[4], r[5], _layout(layout), int(n_shards),
                                            int(bool(causal)), _scale(softmax_scale, q.shape[-1]), r[6], r[7], r[8],
                                            _stream(stream)), "ring_attn_bwd_static_scratch")
    return dq, dk, dv


class CuSeqlens:
    """One cu_seqlens prepared once for repeated varlen calls.

    Holds the int32 host copy that the library validates before each launch and
    the device copy that its kernels read, so that a call given a CuSeqlens
    copies and allocates nothing for it (a plain list or tensor passed to a
    varlen call is copied to the device on every call)."""

    def __init__(self, cu_seqlens, device):
        if isinstance(cu_seqlens, torch.Tensor):
            host = cu_seqlens.detach().to("cpu", torch.int32).contiguous()
        else:
            host = torch.tensor(list(cu_seqlens), dtype=torch.int32)
        if host.dim() != 1 or host.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-D array of n_seqs + 1 prefix sums")
        self.host = host
        self.dev = host.to(device)
        self.n_seqs = host.numel() - 1
        self.total = int(host[-1])
        self.max_seqlen = int((host[1:] - host[:-1]).max())


def _max_len(cu_seqlens, host):
    if isinstance(cu_seqlens, CuSeqlens):
        return cu_seqlens.max_seqlen
    return int((host[1:] - host[:-1]).max())


def _cu_pair(cu_seqlens, device):
    """(host, device) copies of cu_seqlens; a CuSeqlens is used as it is."""
    if isinstance(cu_seqlens, CuSeqlens):
        if cu_seqlens.dev.device != torch.device(device):
            raise ValueError(f"CuSeqlens was prepared for {cu_seqlens.dev.device}, not {device}")
        return cu_seqlens.host, cu_seqlens.dev
    c = CuSeqlens(cu_seqlens, device)
    return c.host, c.dev


def ring_attn_varlen_fwd(q, k, v, cu_seqlens, max_seqlen=None, n_shards=1, causal=True, softmax_scale=None,
                         out=None, lse=None, stream=None, layout="contiguous", workspace=None, scores=None):
    """Packed sequences, one cu_seqlens.  q, k, v: (total, h, d) or (h, total, d) bf16 in
    layout order ("contiguous" slices of the packed buffer, or "zigzag" per sequence);
    k and v may have fewer heads than q (grouped-query attention, as in ring_attn_fwd).

    workspace: None allocates what ring_attn_varlen_workspace_size asks for (for
    zigzag, the original-order copies the library computes in); pass a tensor to
    reuse one (an empty tensor runs the zigzag kernels directly).
    Returns (out like q, lse (h, total) fp32)."""
    if scores is not None:
        return _scored_call("scored_varlen_fwd", q, stream, q, k, v, *_cu_arrays(cu_seqlens, q, stream), max_seqlen,
                            _layout(layout), n_shards, causal, _scale(softmax_scale, q.shape[-1]), _of(scores), out,
                            lse, workspace)
    lib = load()
    host, dev = _cu_pair(cu_seqlens, q.device)
    n = host.numel() - 1
    total = int(host[-1])
    if max_seqlen is None:
        max_seqlen = _max_len(cu_seqlens, host)
    h = q.shape[1] if q.shape[0] == total else q.shape[0]
    d = q.shape[2]
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((h, total), dtype=torch.float32, device=q.device) if lse is None else lse
    if workspace is None:
        need = ring_attn_varlen_workspace_size(RA_OP_FWD, total, h, d, layout, n_shards)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    wp, wb = _ws_arg(workspace)
    tq, tk, tv, to, tl = _t(q), _t(k), _t(v), _t(out), _t(lse)
    _check(lib.ring_attn_varlen_fwd(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                    ctypes.c_void_p(dev.data_ptr()), ctypes.c_void_p(host.data_ptr()), n,
                                    int(max_seqlen), _layout(layout), int(n_shards), int(bool(causal)),
                                    _scale(softmax_scale, d), ctypes.byref(to), ctypes.byref(tl), wp, wb,
                                    _stream(stream)),
           "ring_attn_varlen_fwd")
    return out, lse


def ring_attn_varlen_bwd(dout, q, k, v, out, lse, cu_seqlens, max_seqlen=None, n_shards=1, causal=True,
                         softmax_scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None,
                         layout="contiguous", scores=None):
    if scores is not None:
        return _scored_call("scored_varlen_bwd", q, stream, dout, q, k, v, out, lse,
                            *_cu_arrays(cu_seqlens, q, stream), max_seqlen, _layout(layout), n_shards, causal,
                            _scale(softmax_scale, q.shape[-1]), _of(scores), dq, dk, dv, workspace)
    lib = load()
    host, dev = _cu_pair(cu_seqlens, q.device)
    n = host.numel() - 1
    total = int(host[-1])
    if max_seqlen is None:
        max_seqlen = _max_len(cu_seqlens, host)
    h = q.shape[1] if q.shape[0] == total else q.shape[0]
    d = q.shape[2]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        ws_bytes = ring_attn_varlen_workspace_size(RA_OP_BWD, total, h, d, layout, n_shards)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ts = [_t(x) for x in (dout, q, k, v, out, lse, dq, dk, dv)]
    r = [ctypes.byref(x) for x in ts]
    _check(lib.ring_attn_varlen_bwd(r[0], r[1], r[2], r[3], r[4], r[5], ctypes.c_void_p(dev.data_ptr()),
                                    ctypes.c_void_p(host.data_ptr()), n, int(max_seqlen), _layout(layout),
                                    int(n_shards), int(bool(causal)), _scale(softmax_scale, d), r[6], r[7], r[8],
                                    ctypes.c_void_p(workspace.data_ptr()),
                                    workspace.numel() * workspace.element_size(), _stream(stream)),
           "ring_attn_varlen_bwd")
    return dq, dk, dv


# ---------------------------------------------------------------------------- llama3 form
def _heads_of(x, rows):
    return x.shape[1] if x.shape[0] == rows else x.shape[0]


def ring_attn_llama3_varlen_fwd(q, k, v, cu_seqlens, rank, n_shards, causal=True, softmax_scale=None, max_seqlen=None,
                                out=None, lse=None, stream=None, scores=None):
    """One rank of the llama3 form: q (L, h, d) or (h, L, d), the rank's contiguous slice of the
    packed buffer (L = total / n_shards); k, v: all total rows.  Returns (out like q, lse (h, L))."""
    load()
    with _place(scores, q, stream):
        host, dev = _cu_pair(cu_seqlens, q.device)
        n = host.numel() - 1
        total = int(host[-1])
        if max_seqlen is None:
            max_seqlen = _max_len(cu_seqlens, host)
        L = total // int(n_shards)
        h, d = _heads_of(q, L), q.shape[2]
        out = torch.empty_like(q) if out is None else out
        lse = torch.empty((h, L), dtype=torch.float32, device=q.device) if lse is None else lse
        t = [_t(x) for x in (q, k, v, out, lse)]
        _call("llama3_varlen_fwd", scores, q.device, h, n, 11, ctypes.byref(t[0]), ctypes.byref(t[1]),
              ctypes.byref(t[2]), ctypes.c_void_p(dev.data_ptr()), ctypes.c_void_p(host.data_ptr()), n,
              int(max_seqlen), int(rank), int(n_shards), int(bool(causal)), _scale(softmax_scale, d),
              ctypes.byref(t[3]), ctypes.byref(t[4]), _stream(stream))
    return out, lse


def ring_attn_llama3_varlen_bwd(dout, q, k, v, out, lse, cu_seqlens, rank, n_shards, causal=True, softmax_scale=None,
                                max_seqlen=None, dq=None, dk=None, dv=None, workspace=None, stream=None, scores=None):
    """Gradient of one rank of the llama3 form: (dq of the rank's rows, the rank's contributions to dk, dv)."""
    load()
    with _place(scores, q, stream):
        host, dev = _cu_pair(cu_seqlens, q.device)
        n = host.numel() - 1
        total = int(host[-1])
        if max_seqlen is None:
            max_seqlen = _max_len(cu_seqlens, host)
        L = total // int(n_shards)
        h, d = _heads_of(q, L), q.shape[2]
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        ws_bytes = ring_attn_workspace_size(RA_OP_BWD, 1, h, L, d, 1)
        if workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        ts = [_t(x) for x in (dout, q, k, v, out, lse, dq, dk, dv)]
        r = [ctypes.byref(x) for x in ts]
        _call("llama3_varlen_bwd", scores, q.device, h, n, 14, r[0], r[1], r[2], r[3], r[4], r[5],
              ctypes.c_void_p(dev.data_ptr()), ctypes.c_void_p(host.data_ptr()), n, int(max_seqlen), int(rank),
              int(n_shards), int(bool(causal)), _scale(softmax_scale, d), r[6], r[7], r[8],
              ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(), _stream(stream))
    return dq, dk, dv


# ---------------------------------------------------------------------------- packed forms
# The "kvpacked" / "qkvpacked" entry points of the "Ring Flash Attention" README
# (API list) take k and v, or q, k and v, stacked in one tensor.  They are
# strided views over the calls above: the kernels read the packed tensors in
# place through their strides, and the gradients are written into one packed
# tensor the same way.  Batched forms use the flash-attention packing
# (b, s, 3 or 2, h, d) with out and dout as (b, s, h, d); varlen forms use
# (total, 3 or 2, h, d) with out and dout as (total, h, d).  The sequence axis
# is in layout order, as everywhere in this library.

def _bshd(x):
    """(b, s, h, d) -> the (b, h, s, d) view the calls take."""
    return x.transpose(1, 2)


def ring_attn_qkvpacked_fwd(qkv, layout="contiguous", n_shards=1, causal=False, softmax_scale=None, out=None,
                            lse=None, stream=None, scores=None):
    """qkv: (b, s, 3, h, d) bf16.  Returns (out (b, s, h, d) bf16, lse (b, h, s) fp32)."""
    b, s, three, h, d = qkv.shape
    if three != 3:
        raise ValueError("qkv must be (b, s, 3, h, d)")
    out = torch.empty((b, s, h, d), dtype=qkv.dtype, device=qkv.device) if out is None else out
    _, lse = ring_attn_fwd(_bshd(qkv[:, :, 0]), _bshd(qkv[:, :, 1]), _bshd(qkv[:, :, 2]), layout, n_shards, causal,
                           softmax_scale, out=_bshd(out), lse=lse, stream=stream, scores=scores)
    return out, lse


def ring_attn_qkvpacked_bwd(dout, qkv, out, lse, layout="contiguous", n_shards=1, causal=False, softmax_scale=None,
                            dqkv=None, workspace=None, stream=None, scores=None):
    """Gradient of ring_attn_qkvpacked_fwd: dqkv (b, s, 3, h, d) bf16."""
    dqkv = torch.empty_like(qkv) if dqkv is None else dqkv
    ring_attn_bwd(_bshd(dout), _bshd(qkv[:, :, 0]), _bshd(qkv[:, :, 1]), _bshd(qkv[:, :, 2]), _bshd(out), lse,
                  layout, n_shards, causal, softmax_scale, dq=_bshd(dqkv[:, :, 0]), dk=_bshd(dqkv[:, :, 1]),
                  dv=_bshd(dqkv[:, :, 2]), workspace=workspace, stream=stream, scores=scores)
    return dqkv


def ring_attn_kvpacked_fwd(q, kv, layout="contiguous", n_shards=1, causal=False, softmax_scale=None, out=None,
                           lse=None, stream=None, scores=None):
    """q: (b, s, h, d), kv: (b, s, 2, h, d) bf16.  Returns (out (b, s, h, d), lse (b, h, s))."""
    if kv.dim() != 5 or kv.shape[2] != 2:
        raise ValueError("kv must be (b, s, 2, h, d)")
    out = torch.empty_like(q) if out is None else out
    _, lse = ring_attn_fwd(_bshd(q), _bshd(kv[:, :, 0]), _bshd(kv[:, :, 1]), layout, n_shards, causal,
                           softmax_scale, out=_bshd(out), lse=lse, stream=stream, scores=scores)
    return out, lse


def ring_attn_kvpacked_bwd(dout, q, kv, out, lse, layout="contiguous", n_shards=1, causal=False, softmax_scale=None,
                           dq=None, dkv=None, workspace=None, stream=None, scores=None):
    """Gradient of ring_attn_kvpacked_fwd: (dq (b, s, h, d), dkv (b, s, 2, h, d))."""
    dq = torch.empty_like(q) if dq is None else dq
    dkv = torch.empty_like(kv) if dkv is None else dkv
    ring_attn_bwd(_bshd(dout), _bshd(q), _bshd(kv[:, :, 0]), _bshd(kv[:, :, 1]), _bshd(out), lse, layout, n_shards,
                  causal, softmax_scale, dq=_bshd(dq), dk=_bshd(dkv[:, :, 0]), dv=_bshd(dkv[:, :, 1]),
                  workspace=workspace, stream=stream, scores=scores)
    return dq, dkv


def ring_attn_varlen_qkvpacked_fwd(qkv, cu_seqlens, max_seqlen=None, n_shards=1, causal=True, softmax_scale=None,
                                   out=None, lse=None, stream=None, layout="contiguous", scores=None):
    """qkv: (total, 3, h, d) bf16.  Returns (out (total, h, d), lse (h, total))."""
    if qkv.dim() != 4 or qkv.shape[1] != 3:
        raise ValueError("qkv must be (total, 3, h, d)")
    out = torch.empty_like(qkv[:, 0]) if out is None else out
    return ring_attn_varlen_fwd(qkv[:, 0], qkv[:, 1], qkv[:, 2], cu_seqlens, max_seqlen, n_shards, causal,
                                softmax_scale, out=out, lse=lse, stream=stream, layout=layout, scores=scores)


def ring_attn_varlen_qkvpacked_bwd(dout, qkv, out, lse, cu_seqlens, max_seqlen=None, n_shards=1, causal=True,
                                   softmax_scale=None, dqkv=None, workspace=None, stream=None, layout="contiguous", scores=None):
    """Gradient of ring_attn_varlen_qkvpacked_fwd: dqkv (total, 3, h, d)."""
    dqkv = torch.empty_like(qkv) if dqkv is None else dqkv
    ring_attn_varlen_bwd(dout, qkv[:, 0], qkv[:, 1], qkv[:, 2], out, lse, cu_seqlens, max_seqlen, n_shards, causal,
                         softmax_scale, dq=dqkv[:, 0], dk=dqkv[:, 1], dv=dqkv[:, 2], workspace=workspace,
                         stream=stream, layout=layout, scores=scores)
    return dqkv


def ring_attn_varlen_kvpacked_fwd(q, kv, cu_seqlens, max_seqlen=None, n_shards=1, causal=True, softmax_scale=None,
                                  out=None, lse=None, stream=None, layout="contiguous", scores=None):
    """q: (total, h, d), kv: (total, 2, h, d).  Returns (out (total, h, d), lse (h, total))."""
    if kv.dim() != 4 or kv.shape[1] != 2:
        raise ValueError("kv must be (total, 2, h, d)")
    return ring_attn_varlen_fwd(q, kv[:, 0], kv[:, 1], cu_seqlens, max_seqlen, n_shards, causal, softmax_scale,
                                out=out, lse=lse, stream=stream, layout=layout, scores=scores)


def ring_attn_varlen_kvpacked_bwd(dout, q, kv, out, lse, cu_seqlens, max_seqlen=None, n_shards=1, causal=True,
                                  softmax_scale=None, dq=None, dkv=None, workspace=None, stream=None,
                                  layout="contiguous", scores=None):
    """Gradient of ring_attn_varlen_kvpacked_fwd: (dq (total, h, d), dkv (total, 2, h, d))."""
    dq = torch.empty_like(q) if dq is None else dq
    dkv = torch.empty_like(kv) if dkv is None else dkv
    ring_attn_varlen_bwd(dout, q, kv[:, 0], kv[:, 1], out, lse, cu_seqlens, max_seqlen, n_shards, causal,
                         softmax_scale, dq=dq, dk=dkv[:, 0], dv=dkv[:, 1], workspace=workspace, stream=stream, scores=scores,
                         layout=layout)
    return dq, dkv


def ring_attn_varlen_permute(x, cu_seqlens, layout, n_shards, seq_dim=0, out=None, stream=None):
    """Packed original order -> layout order along seq_dim for one cu_seqlens (bit copy)."""
    lib = load()
    host, dev = _cu_pair(cu_seqlens, x.device)
    out = torch.empty_like(x) if out is None else out
    a, b_ = _t(x), _t(out)
    _check(lib.ring_attn_varlen_permute(ctypes.byref(a), ctypes.byref(b_), ctypes.c_void_p(dev.data_ptr()),
                                        ctypes.c_void_p(host.data_ptr()), host.numel() - 1, _layout(layout),
                                        int(n_shards), int(seq_dim), _stream(stream)), "ring_attn_varlen_permute")
    return out


def ring_attn_varlen_unpermute(y, cu_seqlens, layout, n_shards, seq_dim=0, out=None, stream=None):
    """Layout order -> packed original order along seq_dim (bit copy)."""
    lib = load()
    host, dev = _cu_pair(cu_seqlens, y.device)
    out = torch.empty_like(y) if out is None else out
    a, b_ = _t(y), _t(out)
    _check(lib.ring_attn_varlen_unpermute(ctypes.byref(a), ctypes.byref(b_), ctypes.c_void_p(dev.data_ptr()),
                                          ctypes.c_void_p(host.data_ptr()), host.numel() - 1, _layout(layout),
                                          int(n_shards), int(seq_dim), _stream(stream)), "ring_attn_varlen_unpermute")
    return out


def ring_attn_permute(x, layout, n_shards, seq_dim=2, out=None, stream=None):
    """Original token order -> layout order along seq_dim (bit copy)."""
    lib = load()
    out = torch.empty_like(x) if out is None else out
    a, b_ = _t(x), _t(out)
    _check(lib.ring_attn_permute(ctypes.byref(a), ctypes.byref(b_), _layout(layout), int(n_shards), int(seq_dim),
                                 _stream(stream)), "ring_attn_permute")
    return out


def ring_attn_unpermute(y, layout, n_shards, seq_dim=2, out=None, stream=None):
    """Layout order -> original token order along seq_dim (bit copy)."""
    lib = load()
    out = torch.empty_like(y) if out is None else out
    a, b_ = _t(y), _t(out)
    _check(lib.ring_attn_unpermute(ctypes.byref(a), ctypes.byref(b_), _layout(layout), int(n_shards),
                                   int(seq_dim), _stream(stream)), "ring_attn_unpermute")
    return out


# ---------------------------------------------------------------------------- paged 4-bit cache
class KVCache:
    """A paged key / value cache in 4 bits, as the ring_attn_cache_* calls take it.

    k, v: (n_pages, hk, page, d // 2) uint8, two e2m1 numbers per byte; k_scale, v_scale:
    (n_pages, hk, page, d // 16) float8_e4m3fn.  Any order of the first three dimensions in
    memory (pass a transposed view).  The handle keeps the tensors, which the caller
    allocates, and their description, so that a call marshals nothing for them (so k, k_scale,
    v and v_scale cannot be replaced: other tensors are another handle); copies describe their
    own tensors.  KVCache.empty allocates a cache of zeros.

    The stored scales go from 2^-9 to 448 and there is no other: keys and values of size 0.03 to
    400 are kept best.  Multiply others by a factor before they are appended, and divide
    softmax_scale (keys) or the result (values) by it."""

    k, k_scale, v, v_scale = (property(lambda self, i=i: self._tensors[i]) for i in range(4))

    def __init__(self, k, k_scale, v, v_scale):
        self._tensors = (k, k_scale, v, v_scale)
        for name, x, dtype in (("k", k, torch.uint8), ("k_scale", k_scale, torch.float8_e4m3fn),
                               ("v", v, torch.uint8), ("v_scale", v_scale, torch.float8_e4m3fn)):
            if not isinstance(x, torch.Tensor) or not x.is_cuda:
                raise ValueError("ring_attn_gb300 takes CUDA tensors only")
            if x.dtype != dtype or x.dim() != 4:
                raise ValueError(f"{name} must be a 4-D {dtype} tensor")
            if x.device != k.device:
                raise ValueError("the cache's tensors must be on one device")
        self.device = k.device
        self.n_pages, self.hk, self.page, self.d = k.shape[0], k.shape[1], k.shape[2], 2 * k.shape[3]
        self._c = _KVCache(_desc(k, RA_E2M1X2), _desc(k_scale, RA_E4M3), _desc(v, RA_E2M1X2), _desc(v_scale, RA_E4M3))
        self.scale = 1.0 / math.sqrt(max(self.d, 1))  # the default softmax scale
        self._call = (ctypes.addressof(self._c), k.get_device(), self.hk, self.d)

    def __reduce__(self):  # copies and pickles (which take no 8-bit floats: as bytes)
        return _cache_of_bytes, (type(self), *(x.view(torch.uint8) for x in self._tensors))

    @classmethod
    def empty(cls, n_pages, page, hk, d, device="cuda"):
        code = lambda w: torch.zeros((n_pages, hk, page, w), dtype=torch.uint8, device=device)  # noqa: E731
        return cls(code(d // 2), code(d // 16).view(torch.float8_e4m3fn), code(d // 2),
                   code(d // 16).view(torch.float8_e4m3fn))


def _cache_of_bytes(cls, k, k_scale, v, v_scale):
    return cls(k, k_scale.view(torch.float8_e4m3fn), v, v_scale.view(torch.float8_e4m3fn))


_I64x4 = ctypes.c_int64 * 4


def _desc(x, dtype):
    """The ra_tensor of x (1-D to 4-D)."""
    return _Tensor(x.data_ptr(), dtype, x.dim(), _I64x4(*x.shape), _I64x4(*x.stride()))


_EXT = None


def _ext():
    """The compiled marshaller of the cache calls, the rotation and attention with scores, bound to the loaded library."""
    global _EXT
    if _EXT is None:
        lib = load()
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_ra_binding.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with ring_attn_gb300.build.build() "
                               "(or __graft_entry__.build()); there is no fallback path")
        spec = importlib.util.spec_from_file_location("_ra_binding", path)
        ext = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(ext)
        ext.use(*(ctypes.cast(getattr(lib, "ring_attn_" + f), ctypes.c_void_p).value
                  for f in ("cache_append", "cache_read", "cache_fwd", "cache_workspace_size", "scored_cache_fwd", "rope",
                            "scored_fwd", "scored_bwd", "scored_varlen_fwd", "scored_varlen_bwd", "workspace_size",
                            "varlen_workspace_size")))
        _EXT = ext
    return _EXT


def _cache_call(name, cache, cu_seqlens, stream, *args):
    """Runs a cache call on the given stream (None: the current one of the cache's device) and checks its status."""
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    f = getattr(_EXT or _ext(), name)
    if stream is None:
        if not isinstance(cu_seqlens, CuSeqlens):
            with torch.cuda.device(cache.device):
                cu_seqlens = CuSeqlens(cu_seqlens, cache.device)
        r = f(cache._call, cu_seqlens.dev, cu_seqlens.host, *args)
    else:
        if stream.device != cache.device:
            raise ValueError(f"stream on {stream.device}, cache on {cache.device}")
        with torch.cuda.stream(stream):  # outputs, workspace and cu_seqlens belong to it, too
            if not isinstance(cu_seqlens, CuSeqlens):
                cu_seqlens = CuSeqlens(cu_seqlens, cache.device)
            r = f(cache._call, cu_seqlens.dev, cu_seqlens.host, *args)
    if r[0] != 0:
        _check(r[0], "ring_attn_" + name)
    return r


def ring_attn_cache_append(k, v, cache, page_table, kv_lens, cu_seqlens, q=None, rope=None, positions=None,
                           interleaved=False, q_out=None, stream=None):
    """Rotates k and q and puts k and v into the paged 4-bit cache.

    k, v: (rows, hk, d) bf16, the new tokens of every sequence (cu_seqlens over them, a CuSeqlens
    to copy nothing); kv_lens: (n_seqs,) int32, the sequences' lengths after this call; page_table:
    (n_seqs, max_pages) int32.  q: (rows, h, d) bf16 or None; q_out may be q.  rope: (cos, sin), each
    (positions, r // 2) fp32, or None; positions: (rows,) int32, or None for the tokens' cache indices.
    Rows past cu_seqlens[-1] are left as they were.  Returns q_out (None without q)."""
    cos, sin = rope if rope is not None else (None, None)
    return _cache_call("cache_append", cache, cu_seqlens, stream, k, v, page_table, kv_lens, q, cos, sin, positions,
                       interleaved, q_out)[1]


def ring_attn_cache_read(cache, page_table, kv_lens, cu_seqlens, k_out=None, v_out=None, stream=None):
    """The last cu_seqlens[i + 1] - cu_seqlens[i] cached tokens of every sequence as bf16.

    Returns (k, v), each (rows, hk, d): input for the attention calls."""
    return _cache_call("cache_read", cache, cu_seqlens, stream, page_table, kv_lens, k_out, v_out)[1:]


def ring_attn_cache_workspace_size(total, max_new, h, hk, d, n_seqs) -> int:
    """Bytes of ring_attn_cache_fwd's workspace for `total` new tokens, at most max_new of one sequence."""
    return int(load().ring_attn_cache_workspace_size(int(total), int(max_new), int(h), int(hk), int(d), int(n_seqs)))


def ring_attn_cache_workspace(q, cache, cu_seqlens):
    """A workspace for ring_attn_cache_fwd calls with this q, cache and CuSeqlens (calls on one stream can share it)."""
    n = ring_attn_cache_workspace_size(cu_seqlens.total, cu_seqlens.max_seqlen, q.shape[1], cache.hk, cache.d,
                                       cu_seqlens.n_seqs)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def ring_attn_cache_fwd(q, cache, page_table, kv_lens, cu_seqlens, causal=True, softmax_scale=None, max_kv_len=0,
                        out=None, lse=None, out_dtype=torch.bfloat16, workspace=None, stream=None, scores=None):
    """Attention of new tokens over the paged 4-bit cache.

    q: (rows, h, d) bf16, rotated, h a multiple of the cache's heads; the new tokens are already in
    the cache (ring_attn_cache_append), the last ones of each sequence.  causal: a token sees the
    cache up to itself; else the whole sequence.  max_kv_len: an upper bound of kv_lens (0: what the
    page table can hold).  workspace: from ring_attn_cache_workspace, or None to allocate it.
    scores: a Scores (prefix per sequence; distances between cache indices), or None.
    Returns (out (rows, h, d) bf16 or fp32, lse (h, rows) fp32); rows that see nothing get 0 and -inf."""
    if out is None and out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"unsupported dtype {out_dtype}")
    if softmax_scale is None and isinstance(cache, KVCache):
        softmax_scale = cache.scale
    if scores is not None and not isinstance(scores, Scores):
        raise ValueError("scores must be a Scores")
    return _cache_call("cache_fwd", cache, cu_seqlens, stream, q, page_table, kv_lens, causal, softmax_scale, max_kv_len,
                       out, lse, out_dtype is torch.float32, workspace, scores and scores._parts)[1:]


# ---------------------------------------------------------------------------- rotary positions
def ring_attn_rope(q, k, rope, positions=None, axes=None, interleaved=False, layout="contiguous", n_shards=1, q_out=None,
                   k_out=None, stream=None):
    """Rotates q and k (or None) by their positions, on one axis or several.

    q: (b, h, s, d), k: (b, hk, s, d), or both (rows, heads, d); bf16 or fp32.  rope: (cos, sin), each
    (positions, r // 2) fp32; pairs (i, i + r / 2) of head dims turn, or (2 i, 2 i + 1) if interleaved.
    positions: int32, (b, s) or (rows), or with a leading dimension of axes: pair f then goes by
    the position on axis axes[f] (r // 2 numbers, as [0] * 16 + [1] * 24 + [2] * 24 for time, height and width).
    None: the rows' original tokens, in the order of layout and n_shards.
    q_out may be q and k_out k.  Returns (q_out, k_out)."""
    return _rope_call(False, q, k, rope, positions, axes, interleaved, layout, n_shards, q_out, k_out, stream)


def ring_attn_rope_bwd(dq, dk, rope, positions=None, axes=None, interleaved=False, layout="contiguous", n_shards=1,
                       dq_out=None, dk_out=None, stream=None):
    """Gradient of ring_attn_rope: those of the rotated q and k (or None) in, of the unrotated ones out."""
    return _rope_call(True, dq, dk, rope, positions, axes, interleaved, layout, n_shards, dq_out, dk_out, stream)


def _axes(axes):
    """The axes of the pairs as bytes (bytes(n) of a number would be n zeros, of an array its memory)."""
    if axes is None or isinstance(axes, bytes):
        return axes
    if not isinstance(axes, (list, tuple)):
        try:
            axes = [int(a) for a in axes]
        except TypeError:
            raise ValueError("axes must name an axis for each pair") from None
    return bytes(axes)


def _rope_call(inverse, q, k, rope, positions, axes, interleaved, layout, n_shards, q_out, k_out, stream):
    f = (_EXT or _ext()).rope
    args = (q, k, rope[0], rope[1], positions, _axes(axes), interleaved, inverse,
            _layout(layout), int(n_shards), q_out, k_out)
    if stream is None:
        r = f(*args)
    else:
        if isinstance(q, torch.Tensor) and stream.device != q.device:
            raise ValueError(f"stream on {stream.device}, q on {q.device}")
        with torch.cuda.stream(stream):
            r = f(*args)
    if r[0] != 0:
        _check(r[0], "ring_attn_rope")
    return r[1:]


def ring_attn_check_device_error(stream=None):
    """Synchronises the stream and returns (status, info); status 0 = no device-side error."""
    info = ctypes.c_int32(0)
    st = load().ring_attn_check_device_error(_stream(stream), ctypes.byref(info))
    return int(st), int(info.value)


def ring_attn_set_knob(knob: int, value: int):
    _check(load().ring_attn_set_knob(int(knob), int(value)), "ring_attn_set_knob")


def ring_attn_timing_enable(on: bool = True):
    """Bracket every library kernel launch with CUDA events (see ring_attn_timing_read)."""
    _check(load().ring_attn_timing_enable(int(bool(on))), "ring_attn_timing_enable")


def ring_attn_timing_read(kernel) -> tuple:
    """(total device ms, launches) of one kernel kind (of KERNELS, or "rope") since the last read; resets it."""
    k = _KINDS[kernel] if isinstance(kernel, str) else int(kernel)
    ms = ctypes.c_double(0.0)
    n = ctypes.c_int64(0)
    _check(load().ring_attn_timing_read(k, ctypes.byref(ms), ctypes.byref(n)), "ring_attn_timing_read")
    return float(ms.value), int(n.value)


def ring_attn_version() -> int:
    return int(load().ring_attn_version())
