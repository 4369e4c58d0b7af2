"""Python binding of the cache operators' C ABI (include/mono_cache.h): attention over a paged
fp8 cache, eviction by accumulated attention weight, verification of drafted tokens.

Argument marshalling and checks only; the operators run in the library's CUDA kernels.  Tensors
must be CUDA tensors of one device and stay valid until the enqueued work has run.  A wrong
dtype, shape, stride or device raises ValueError, what the library refuses raises MonoError.
"""
from __future__ import annotations

import ctypes as C
import struct

import torch

import moe_decode_layer_mxfp8_gb300 as _m


class CacheSpec(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_q_heads", "head_dim", "kv_dim", "block_size",
                                         "kv_record_bytes", "max_rows", "max_req")]


class AttendArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("o", C.c_void_p), ("q_stride", C.c_int64),
                ("o_stride", C.c_int64), ("positions", C.c_void_p), ("row_req", C.c_void_p),
                ("block_table", C.c_void_p), ("max_blocks", C.c_int32), ("n_req", C.c_int32),
                ("rows", C.c_int32), ("window", C.c_int32), ("sinks", C.c_int32),
                ("causal", C.c_int32), ("scale", C.c_float), ("kv_cache", C.c_void_p),
                ("kv_stride_block", C.c_int64), ("kv_stride_tok", C.c_int64),
                ("kv_num_blocks", C.c_int64), ("lse", C.c_void_p), ("weights", C.c_void_p),
                ("weights_stride", C.c_int64), ("weights_cols", C.c_int64)]


class EvictArgs(C.Structure):
    _fields_ = [("weights", C.c_void_p), ("weights_out", C.c_void_p),
                ("weights_stride", C.c_int64), ("weights_out_stride", C.c_int64),
                ("lengths", C.c_void_p), ("new_lengths", C.c_void_p), ("kept", C.c_void_p),
                ("kept_stride", C.c_int64), ("budget", C.c_int32), ("sinks", C.c_int32),
                ("recent", C.c_int32), ("n_req", C.c_int32), ("block_table", C.c_void_p),
                ("max_blocks", C.c_int32), ("kv_cache", C.c_void_p),
                ("kv_stride_block", C.c_int64), ("kv_stride_tok", C.c_int64),
                ("kv_num_blocks", C.c_int64), ("dst_table", C.c_void_p),
                ("dst_max_blocks", C.c_int32), ("dst_cache", C.c_void_p),
                ("dst_stride_block", C.c_int64), ("dst_stride_tok", C.c_int64),
                ("dst_num_blocks", C.c_int64), ("weights_cols", C.c_int64),
                ("weights_out_cols", C.c_int64)]


class VerifyArgs(C.Structure):
    _fields_ = [("target", C.c_void_p), ("draft", C.c_void_p), ("target_stride", C.c_int64),
                ("draft_stride", C.c_int64), ("dtype", C.c_int32), ("vocab", C.c_int32),
                ("rows", C.c_int32), ("n_req", C.c_int32), ("row_start", C.c_void_p),
                ("draft_tokens", C.c_void_p), ("u", C.c_void_p), ("r", C.c_void_p),
                ("greedy", C.c_void_p), ("accepted", C.c_void_p), ("tokens", C.c_void_p)]


# The same structures packed at once: setting ctypes fields one by one took most of a call.
_ATTEND = struct.Struct("@PPqqPPPiiiiiifPqqqPPqq")
_EVICT = struct.Struct("@PPqqPPPqiiiiPiPqqqPiPqqqqq")
_VERIFY = struct.Struct("@PPqqiiiiPPPPPPP")

CACHE_EXPORTS = ["mono_cache_build", "mono_cache_free", "mono_cache_status", "mono_cache_attend",
                 "mono_cache_evict", "mono_verify_drafts"]


def _lib() -> C.CDLL:
    L = _m.lib()
    if not getattr(L, "_mono_cache_ready", False):
        L.mono_cache_build.argtypes = [C.POINTER(CacheSpec), C.POINTER(C.c_void_p)]
        L.mono_cache_free.argtypes = [C.c_void_p]
        L.mono_cache_free.restype = None
        L.mono_cache_status.argtypes = [C.c_void_p, C.c_int]
        L.mono_cache_attend.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p]
        L.mono_cache_evict.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p]
        L.mono_verify_drafts.argtypes = [C.c_void_p, C.c_void_p]
        L._mono_cache_ready = True
    return L


def _bad(t, name, dtypes, shape, device, packed):
    """What is wrong with a tensor that failed the checks below."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is not a tensor")
    if t.dtype not in dtypes:
        names = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} is {t.dtype}, not {names}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not cuda:{device}")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not "
                         f"({', '.join('*' if w is None else str(w) for w in shape)})")
    raise ValueError(f"{name} is not contiguous" + ("" if packed else " in its last dimension, or is "
                     f"broadcast: strides {t.stride()}"))


def _vec(t, name, dtype, n, device):
    """Address of a contiguous vector of n elements."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != (n,) or not t.is_contiguous():
        _bad(t, name, (dtype,), (n,), device, True)
    return t.data_ptr()


def _mat(t, name, dtypes, rows, cols, device):
    """(address, row stride) of a [rows, cols] matrix (None: any) with contiguous rows."""
    shape, stride = t.shape, t.stride()
    if (t.dtype not in dtypes or t.get_device() != device or len(shape) != 2
            or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols)
            or (shape[1] > 1 and stride[1] != 1) or (shape[0] > 1 and stride[0] < shape[1])):
        _bad(t, name, dtypes, (rows, cols), device, False)
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1]


def _weights(t, name, rows, device):
    """(address, row stride, columns) of a f32 [rows, tokens] matrix."""
    p, stride = _mat(t, name, _F32, rows, None, device)
    if t.shape[1] == 0:
        raise ValueError(f"{name} has no columns")
    return p, stride, t.shape[1]


def _table(t, name, rows, device):
    if (t.dtype is not torch.int32 or t.get_device() != device or t.dim() != 2
            or (rows is not None and t.shape[0] != rows) or not t.is_contiguous()):
        _bad(t, name, (torch.int32,), (rows, None), device, True)
    return t.data_ptr()


def _pack(layout, *values):
    try:
        return layout.pack(*values)
    except struct.error as e:
        raise ValueError(f"an argument is not a 32-bit integer: {e}") from None


_BF16, _F32 = (torch.bfloat16,), (torch.float32,)
_LEAST, _MOST = 2.0 ** -149, (2.0 - 2.0 ** -23) * 2.0 ** 127  # an f32 above 0
_PROBS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


# What torch.cuda.current_stream and current_device ask, without their wrappers (2 us of a call); not
# in a torch built without CUDA.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _call(name, device, stream, *args):
    """Calls the library with `device` current, on `stream` or torch's current one."""
    if stream is None:
        raw = _raw_stream(device)
    elif stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, not cuda:{device}")
    else:
        raw = stream.cuda_stream
    fn = getattr(_lib(), name)
    if _current_device() == device:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, raw)
    if rc != _m.MONO_OK:
        raise _m.MonoError(rc, name)


class Cache:
    """The operators on one cache layout (``spec``: n_q_heads, head_dim, kv_dim, block_size,
    kv_record_bytes, as in a layer's spec), with a workspace for steps of up to ``max_rows`` rows
    of ``max_requests`` requests on the current device.  Calls on one Cache share the workspace:
    order them on the GPU."""

    def __init__(self, spec: dict, max_rows: int, max_requests: int):
        self.spec = {k: int(spec[k]) for k in ("n_q_heads", "head_dim", "kv_dim", "block_size",
                                               "kv_record_bytes")}
        self._h = C.c_void_p()
        self.max_rows, self.max_requests = int(max_rows), int(max_requests)
        s = CacheSpec(**self.spec, max_rows=self.max_rows, max_req=self.max_requests)
        rc = _lib().mono_cache_build(C.byref(s), C.byref(self._h))
        if rc != _m.MONO_OK:
            raise _m.MonoError(rc, "mono_cache_build")
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._dev = self.device.index
        self._width = self.spec["n_q_heads"] * self.spec["head_dim"]

    def _view(self, t, name):
        if t.dim() != 3 or t.dtype is not torch.uint8 or t.get_device() != self._dev:
            raise ValueError(f"{name} is a uint8 [blocks, block_size, record] view on {self.device}")
        shape, stride = t.shape, t.stride()
        if (shape[1] != self.spec["block_size"] or shape[2] < self.spec["kv_record_bytes"]
                or stride[2] != 1):
            raise ValueError(f"{name}: pages of {self.spec['block_size']} records of "
                             f"{self.spec['kv_record_bytes']} contiguous bytes expected, got shape "
                             f"{tuple(shape)}, strides {stride}")
        return t.data_ptr(), stride[0], stride[1], shape[0]

    def attend(self, q, o, positions, row_req, block_table, kv_cache, *, window=0, sinks=0,
               causal=True, scale=None, lse=None, weights=None, stream=None) -> None:
        """Attention of q's rows (bf16 [rows, n_q_heads * head_dim]) over the cached tokens of
        their requests, into o (bf16, like q).  ``window`` 0 is the whole context, else the last
        ``window`` tokens and the first ``sinks``; ``lse`` (f32 [rows, n_q_heads]) gets the
        log-sum-exp of the scores, ``weights`` (f32 [n_req, tokens]) each token's attention weight
        added."""
        dev, i32 = self._dev, torch.int32
        rows, (n_req, max_blocks) = q.shape[0], block_table.shape
        if scale is None:
            scale = 0.0
        elif not _LEAST <= scale <= _MOST:  # (0 is the library's default)
            raise ValueError("scale must be positive, and an f32")
        qp, qs = _mat(q, "q", _BF16, rows, self._width, dev)
        op, os = _mat(o, "o", _BF16, rows, self._width, dev)
        heads = self.spec["n_q_heads"]
        lp = 0
        if lse is not None:
            lp, ls = _mat(lse, "lse", _F32, rows, heads, dev)
            if ls != heads:
                _bad(lse, "lse", _F32, (rows, heads), dev, True)
        wp, ws, wc = (0, 0, 0) if weights is None else _weights(weights, "weights", n_req, dev)
        args = _pack(_ATTEND, qp, op, qs, os, _vec(positions, "positions", i32, rows, dev),
                     _vec(row_req, "row_req", i32, rows, dev),
                     _table(block_table, "block_table", None, dev), max_blocks, n_req, rows,
                     window, sinks, 1 if causal else 0, scale,
                     *self._view(kv_cache, "kv_cache"), lp, wp, ws, wc)
        self._call("mono_cache_attend", args, stream)

    def evict(self, weights, lengths, block_table, kv_cache, kept, new_lengths, *, budget,
              sinks=0, recent=0, weights_out=None, dst_table=None, dst_cache=None,
              stream=None) -> None:
        """Keeps ``budget`` tokens of each request (its first ``sinks``, its last ``recent`` and
        the heaviest of the others by ``weights``, f32 [n_req, tokens]) and moves their records and
        weights, in order, to the front of its pages, or to those of ``dst_table`` (in
        ``dst_cache``).  kept (int32 [n_req, >= budget]) gets the old slots, new_lengths the
        counts."""
        dev, i32 = self._dev, torch.int32
        n_req, max_blocks = block_table.shape
        wp, ws, wc = _weights(weights, "weights", n_req, dev)
        kp, ks = _mat(kept, "kept", (i32,), n_req, None, dev)
        if kept.shape[1] < budget:
            raise ValueError(f"kept holds {kept.shape[1]} slots a request, the budget is {budget}")
        vp, vs, vc = (0, 0, 0) if weights_out is None else _weights(weights_out, "weights_out", n_req, dev)
        tp, tb = (0, 0) if dst_table is None else (_table(dst_table, "dst_table", n_req, dev),
                                                   dst_table.shape[1])
        dst = (0, 0, 0, 0)
        if dst_cache is not None:
            if dst_table is None:
                raise ValueError("dst_cache needs a dst_table")
            dst = self._view(dst_cache, "dst_cache")
        args = _pack(_EVICT, wp, vp, ws, vs, _vec(lengths, "lengths", i32, n_req, dev),
                     _vec(new_lengths, "new_lengths", i32, n_req, dev), kp, ks, budget, sinks,
                     recent, n_req, _table(block_table, "block_table", None, dev), max_blocks,
                     *self._view(kv_cache, "kv_cache"), tp, tb, *dst, wc, vc)
        self._call("mono_cache_evict", args, stream)

    def _call(self, name, args, stream):
        if not self._h:
            raise ValueError("the Cache is closed")
        _call(name, self._dev, stream, self._h, args)

    def status(self, clear: bool = False) -> int:
        """The handle's MONO_STATUS_* bits (waits for the device, all its streams)."""
        if not self._h:
            raise ValueError("the Cache is closed")
        rc = _lib().mono_cache_status(self._h, int(clear))
        if rc < 0:
            raise _m.MonoError(rc, "mono_cache_status")
        return rc

    def close(self) -> None:
        if self._h:
            _lib().mono_cache_free(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def verify_drafts(target, draft, draft_tokens, row_start, u, r, accepted, tokens, *, greedy=None,
                  stream=None) -> None:
    """Verifies drafted tokens: request b's rows are row_start[b] .. row_start[b + 1] - 1, one per
    draft and a last one.  ``target`` and ``draft`` (or None for certain drafts) are probabilities
    [rows, vocab] in f32, bf16 or f16; u [rows] and r [n_req] are uniform random numbers;
    ``greedy`` marks requests that take the target's maximum.  accepted [n_req] gets the number of
    accepted drafts, tokens [rows] the accepted drafts, the drawn token and -1 behind it."""
    dev = target.get_device()
    if dev < 0:
        raise ValueError("target is not a CUDA tensor")
    i32, f32 = torch.int32, torch.float32
    tp, ts = _mat(target, "target", _PROBS, None, None, dev)
    rows, vocab = target.shape
    n_req = row_start.shape[0] - 1
    dp, ds = (0, 0) if draft is None else _mat(draft, "draft", (target.dtype,), rows, vocab, dev)
    args = _pack(_VERIFY, tp, dp, ts, ds, _PROBS[target.dtype], vocab, rows, n_req,
                 _vec(row_start, "row_start", i32, n_req + 1, dev),
                 _vec(draft_tokens, "draft_tokens", i32, rows, dev),
                 _vec(u, "u", f32, rows, dev), _vec(r, "r", f32, n_req, dev),
                 0 if greedy is None else _vec(greedy, "greedy", i32, n_req, dev),
                 _vec(accepted, "accepted", i32, n_req, dev),
                 _vec(tokens, "tokens", i32, rows, dev))
    _call("mono_verify_drafts", dev, stream, args)
