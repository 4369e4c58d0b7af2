"""Python binding of the cache operators' C ABI (include/mono_cache.h): attention over a paged
fp8 cache (also behind prefixes that requests share), eviction by accumulated attention weight,
appending and rotating by position, verification of drafted tokens.

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


class SharedArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("o", C.c_void_p), ("q_stride", C.c_int64),
                ("o_stride", C.c_int64), ("positions", C.c_void_p), ("row_req", C.c_void_p),
                ("block_table", C.c_void_p), ("prefix_table", C.c_void_p),
                ("prefix_lengths", C.c_void_p), ("prefix_of", C.c_void_p),
                ("max_blocks", C.c_int32), ("n_req", C.c_int32), ("prefix_max_blocks", C.c_int32),
                ("n_prefix", C.c_int32), ("rows", C.c_int32), ("causal", C.c_int32),
                ("scale", C.c_float), ("kv_cache", C.c_void_p), ("kv_stride_block", C.c_int64),
                ("kv_stride_tok", C.c_int64), ("kv_num_blocks", C.c_int64), ("lse", C.c_void_p)]


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


class Rope(C.Structure):
    _fields_ = [("table", C.c_void_p), ("stride", C.c_int64), ("positions", C.c_int64),
                ("dim", C.c_int32), ("offset", C.c_int32), ("interleaved", C.c_int32),
                ("inverse", C.c_int32)]


class AppendArgs(C.Structure):
    _fields_ = [("kv", C.c_void_p), ("q", C.c_void_p), ("q_out", C.c_void_p),
                ("kv_stride", C.c_int64), ("q_stride", C.c_int64), ("q_out_stride", C.c_int64),
                ("positions", C.c_void_p), ("rope_positions", C.c_void_p), ("row_req", C.c_void_p),
                ("block_table", C.c_void_p), ("kv_cache", C.c_void_p),
                ("kv_stride_block", C.c_int64), ("kv_stride_tok", C.c_int64),
                ("kv_num_blocks", C.c_int64), ("rope", Rope), ("dtype", C.c_int32),
                ("rows", C.c_int32), ("n_req", C.c_int32), ("max_blocks", C.c_int32)]


class RotateArgs(C.Structure):
    _fields_ = [("x", C.c_void_p), ("out", C.c_void_p), ("x_stride", C.c_int64),
                ("out_stride", C.c_int64), ("positions", C.c_void_p), ("rope", Rope),
                ("dtype", C.c_int32), ("rows", C.c_int32), ("heads", C.c_int32)]


class VerifyArgs(C.Structure):
    _fields_ = [("target", C.c_void_p), ("draft", C.c_void_p), ("target_stride", C.c_int64),
                ("draft_stride", C.c_int64), ("dtype", C.c_int32), ("vocab", C.c_int32),
                ("rows", C.c_int32), ("n_req", C.c_int32), ("row_start", C.c_void_p),
                ("draft_tokens", C.c_void_p), ("u", C.c_void_p), ("r", C.c_void_p),
                ("greedy", C.c_void_p), ("accepted", C.c_void_p), ("tokens", C.c_void_p)]


# The same structures packed at once: setting ctypes fields one by one took most of a call.
_ATTEND = struct.Struct("@PPqqPPPiiiiiifPqqqPPqq")
_SHARED = struct.Struct("@PPqqPPPPPPiiiiiifPqqqP")
_EVICT = struct.Struct("@PPqqPPPqiiiiPiPqqqPiPqqqqq")
_APPEND = struct.Struct("@PPPqqqPPPPPqqqPqqiiiiiiii")
_ROTATE = struct.Struct("@PPqqPPqqiiiiiii4x")
_VERIFY = struct.Struct("@PPqqiiiiPPPPPPP")

CACHE_EXPORTS = ["mono_cache_build", "mono_cache_free", "mono_cache_status", "mono_cache_attend",
                 "mono_cache_attend_shared", "mono_cache_evict", "mono_cache_append",
                 "mono_cache_rotate", "mono_verify_drafts"]


def _lib() -> C.CDLL:
    L = _m.lib()
    if not getattr(L, "_mono_cache_ready", False):
        L.mono_cache_build.argtypes = [C.POINTER(CacheSpec), C.POINTER(C.c_void_p)]
        L.mono_cache_free.argtypes = [C.c_void_p]
        L.mono_cache_free.restype = None
        L.mono_cache_status.argtypes = [C.c_void_p, C.c_int]
        L.mono_cache_attend.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p]
        L.mono_cache_attend_shared.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p]
        L.mono_cache_evict.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p]
        L.mono_cache_append.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p]
        L.mono_cache_rotate.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p]
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
    shape = t.shape
    if (t.dtype not in dtypes or t.get_device() != device or len(shape) != 2
            or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols)):
        _bad(t, name, dtypes, (rows, cols), device, False)
    if shape[1] and t.is_contiguous():  # (most are, and their strides take twice as long to ask for)
        return t.data_ptr(), shape[1]
    stride = t.stride()
    if (shape[1] > 1 and stride[1] != 1) or (shape[0] > 1 and stride[0] < shape[1]):
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


def _pages(t, name, block_size, record, device):
    """(address, strides of pages and of records, pages) of a cache."""
    if t.dim() != 3 or t.dtype is not torch.uint8 or t.get_device() != device:
        raise ValueError(f"{name} is a uint8 [blocks, block_size, record] view on cuda:{device}")
    shape, stride = t.shape, t.stride()
    if shape[1] != block_size or shape[2] < record or stride[2] != 1:
        raise ValueError(f"{name}: pages of {block_size} records of {record} contiguous bytes expected, "
                         f"got shape {tuple(shape)}, strides {stride}")
    return t.data_ptr(), stride[0], stride[1], shape[0]


_IN_PYTHON = _vec, _mat, _table, _pages


def _native():
    """The extension that makes these checks faster, if it is there for this torch."""
    try:
        from . import _args
    except ImportError:
        return None
    if (_args.TORCH, getattr(_args, "INTERFACE", 0)) != (torch.__version__, 2):
        return None
    _args.otherwise(*_IN_PYTHON)
    return _args


_args = _native()
if _args:
    _vec, _mat, _table, _pages = _args.vec, _args.mat, _args.table, _args.pages


def _pack(layout, *values):
    try:
        return layout.pack(*values)
    except struct.error as e:
        raise ValueError(f"an argument is not a 32-bit integer: {e}") from None


_BF16, _F32 = (torch.bfloat16,), (torch.float32,)
_LEAST, _MOST = 2.0 ** -149, (2.0 - 2.0 ** -23) * 2.0 ** 127  # an f32 above 0
_PROBS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_FLOATS = tuple(_PROBS)


# What torch.cuda.current_stream and current_device ask, without their wrappers (2 us of a call); not
# in a torch built without CUDA.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


_functions = {}  # the library's, by name


def _call(name, device, stream, *args):
    """Calls the library with `device` current, on `stream` or torch's current one."""
    if stream is None:
        raw = _raw_stream(device)
    elif stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, not cuda:{device}")
    else:
        raw = stream.cuda_stream
    fn = _functions.get(name) or _functions.setdefault(name, getattr(_lib(), name))
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
        return _pages(t, name, self.spec["block_size"], self.spec["kv_record_bytes"], self._dev)

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

    def attend_shared(self, q, o, positions, row_req, block_table, kv_cache, prefix_table,
                      prefix_lengths, *, prefix_of=None, causal=True, scale=None, lse=None,
                      stream=None) -> None:
        """Attention as ``attend``, where the first prefix_lengths[g] tokens (int32 [prefixes]) of a
        request b with prefix_of[b] = g (int32 [n_req]; -1: none; None: 0 for all) are those of
        row g of ``prefix_table`` (int32 [prefixes, blocks]), read once for all its requests;
        tokens behind them are in ``block_table``, indexed by their place in the whole context.
        Worth it from some 1K shared tokens on; where little is shared and requests of a row or two
        have many tokens of their own, ``attend`` is faster."""
        dev, i32 = self._dev, torch.int32
        rows, (n_req, max_blocks) = q.shape[0], block_table.shape
        n_prefix, prefix_blocks = prefix_table.shape
        if scale is None:
            scale = 0.0
        elif not 2.0 ** -20 <= scale <= 2.0 ** 20:
            raise ValueError("scale must be in [2^-20, 2^20]")
        qp, qs = _mat(q, "q", _BF16, rows, self._width, dev)
        op, os = _mat(o, "o", _BF16, rows, self._width, dev)
        heads = self.spec["n_q_heads"]
        lp = 0
        if lse is not None:
            lp, ls = _mat(lse, "lse", _F32, rows, heads, dev)
            if ls != heads:
                _bad(lse, "lse", _F32, (rows, heads), dev, True)
        args = _pack(_SHARED, qp, op, qs, os, _vec(positions, "positions", i32, rows, dev),
                     _vec(row_req, "row_req", i32, rows, dev),
                     _table(block_table, "block_table", None, dev),
                     _table(prefix_table, "prefix_table", None, dev),
                     _vec(prefix_lengths, "prefix_lengths", i32, n_prefix, dev),
                     0 if prefix_of is None else _vec(prefix_of, "prefix_of", i32, n_req, dev),
                     max_blocks, n_req, prefix_blocks, n_prefix, rows, 1 if causal else 0, scale,
                     *self._view(kv_cache, "kv_cache"), lp)
        self._call("mono_cache_attend_shared", args, stream)

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
        if dst_table is not None and not tp:  # (no address would mean in place)
            raise ValueError("dst_table has no columns")
        dst = (0, 0, 0, 0)
        if dst_cache is not None:
            if dst_table is None:
                raise ValueError("dst_cache needs a dst_table")
            dst = self._view(dst_cache, "dst_cache")
            if not dst[0]:  # (no address would mean kv_cache)
                raise ValueError("dst_cache has no pages")
        args = _pack(_EVICT, wp, vp, ws, vs, _vec(lengths, "lengths", i32, n_req, dev),
                     _vec(new_lengths, "new_lengths", i32, n_req, dev), kp, ks, budget, sinks,
                     recent, n_req, _table(block_table, "block_table", None, dev), max_blocks,
                     *self._view(kv_cache, "kv_cache"), tp, tb, *dst, wc, vc)
        self._call("mono_cache_evict", args, stream)

    def _rope(self, rope, offset, interleaved, inverse):
        """The fields of a rotation: ``rope`` is f32 [positions, dim]."""
        p, stride = _mat(rope, "rope", _F32, None, None, self._dev)
        positions, dim = rope.shape
        if not p:  # (no address would mean no rotation)
            raise ValueError(f"rope has no entries: shape {tuple(rope.shape)}")
        if offset is None:
            offset = self.spec["head_dim"] - dim
        return p, stride, positions, dim, offset, 1 if interleaved else 0, 1 if inverse else 0

    def append(self, kv, positions, row_req, block_table, kv_cache, *, rope=None, rope_offset=None,
               interleaved=False, rope_positions=None, q=None, q_out=None, stream=None) -> None:
        """Stores the rows' latents (kv: f32, bf16 or f16 [rows, kv_dim]) as records of the slots
        ``positions`` (-1: a pad row) of their requests, each latent slice rotated by the row's
        entry of ``rope`` (f32 [positions, dim]: cosines, then sines; None: no rotation) at
        ``rope_positions`` (default: ``positions``).  The rotated dimensions of a head are the
        last ones, or those from ``rope_offset`` on; pairs are halves of them, or neighbours
        (``interleaved``).  ``q`` (like kv, [rows, n_q_heads * head_dim]) is rotated alike, into
        ``q_out`` or in place.  Any number of rows and requests."""
        dev, i32 = self._dev, torch.int32
        rows, dtype = kv.shape[0], kv.dtype
        n_req, max_blocks = block_table.shape
        kp, ks = _mat(kv, "kv", _FLOATS, rows, self.spec["kv_dim"], dev)
        qp, qs, op, os = 0, 0, 0, 0
        if q is not None:
            if rope is None:
                raise ValueError("q needs a rope table")
            qp, qs = _mat(q, "q", (dtype,), rows, self._width, dev)
            op, os = qp, qs
            if q_out is not None:
                op, os = _mat(q_out, "q_out", (dtype,), rows, self._width, dev)
        elif q_out is not None:
            raise ValueError("q_out needs a q")
        if rope is not None:
            turn = self._rope(rope, rope_offset, interleaved, False)
        elif rope_positions is not None or rope_offset is not None:
            raise ValueError("rope_positions and rope_offset need a rope table")
        else:
            turn = (0, 0, 0, 0, 0, 0, 0)
        rp = 0
        if rope_positions is not None:
            rp = _vec(rope_positions, "rope_positions", i32, rows, dev)
        args = _pack(_APPEND, kp, qp, op, ks, qs, os, _vec(positions, "positions", i32, rows, dev),
                     rp, _vec(row_req, "row_req", i32, rows, dev),
                     _table(block_table, "block_table", None, dev),
                     *self._view(kv_cache, "kv_cache"), *turn, _PROBS[dtype], rows, n_req, max_blocks)
        self._call("mono_cache_append", args, stream)

    def rotate(self, x, out, positions, rope, *, rope_offset=None, interleaved=False, inverse=False,
               stream=None) -> None:
        """Rotates the heads of x (f32, bf16 or f16 [rows, heads * head_dim]) by their rows'
        rotary ``positions`` (-1: a pad row, left as it is) into ``out``, which may be x;
        ``inverse`` turns back.  ``rope``, ``rope_offset`` and ``interleaved`` as in append."""
        dev, dh = self._dev, self.spec["head_dim"]
        xp, xs = _mat(x, "x", _FLOATS, None, None, dev)
        rows, width = x.shape
        if width % dh:
            raise ValueError(f"x has rows of {width} elements, not of heads of {dh}")
        op, os = _mat(out, "out", (x.dtype,), rows, width, dev)
        args = _pack(_ROTATE, xp, op, xs, os, _vec(positions, "positions", torch.int32, rows, dev),
                     *self._rope(rope, rope_offset, interleaved, inverse), _PROBS[x.dtype], rows,
                     width // dh)
        self._call("mono_cache_rotate", args, stream)

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
    tp, ts = _mat(target, "target", _FLOATS, None, None, dev)
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
