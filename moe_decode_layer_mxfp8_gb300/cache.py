"""Python binding of the cache operators' C ABI (include/mono_cache.h): attention over a paged
fp8 cache, eviction by accumulated attention weight, verification of drafted tokens.

Argument marshalling and checks only; the operators run in the library's CUDA kernels.  Tensors
must be CUDA tensors of one device and stay valid until the enqueued work has run.  A wrong
dtype, shape, stride or device raises ValueError, what the library refuses raises MonoError.
"""
from __future__ import annotations

import ctypes as C

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
                ("weights_stride", C.c_int64)]


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
                ("dst_num_blocks", C.c_int64)]


class VerifyArgs(C.Structure):
    _fields_ = [("target", C.c_void_p), ("draft", C.c_void_p), ("target_stride", C.c_int64),
                ("draft_stride", C.c_int64), ("dtype", C.c_int32), ("vocab", C.c_int32),
                ("rows", C.c_int32), ("n_req", C.c_int32), ("row_start", C.c_void_p),
                ("draft_tokens", C.c_void_p), ("u", C.c_void_p), ("r", C.c_void_p),
                ("greedy", C.c_void_p), ("accepted", C.c_void_p), ("tokens", C.c_void_p)]


CACHE_EXPORTS = ["mono_cache_build", "mono_cache_free", "mono_cache_status", "mono_cache_attend",
                 "mono_cache_evict", "mono_verify_drafts"]


def _lib() -> C.CDLL:
    L = _m.lib()
    if not getattr(L, "_mono_cache_ready", False):
        L.mono_cache_build.argtypes = [C.POINTER(CacheSpec), C.POINTER(C.c_void_p)]
        L.mono_cache_free.argtypes = [C.c_void_p]
        L.mono_cache_free.restype = None
        L.mono_cache_status.argtypes = [C.c_void_p, C.c_int]
        L.mono_cache_attend.argtypes = [C.c_void_p, C.POINTER(AttendArgs), C.c_void_p]
        L.mono_cache_evict.argtypes = [C.c_void_p, C.POINTER(EvictArgs), C.c_void_p]
        L.mono_verify_drafts.argtypes = [C.POINTER(VerifyArgs), C.c_void_p]
        L._mono_cache_ready = True
    return L


def _check(t, name, dtypes, shape, device, inner=True):
    """A CUDA tensor of one of the dtypes and of the shape (None: any size), its last dimension
    contiguous, on `device`.  Returns its data pointer."""
    names = [str(d).replace("torch.", "") for d in dtypes]
    if t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, not {' or '.join(names)}")
    if t.dim() != len(shape) or any(w is not None and s != w for s, w in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not "
                         f"({', '.join('*' if w is None else str(w) for w in shape)})")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if inner and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} is not contiguous in its last dimension")
    if t.dim() > 1 and any(s > 1 and st <= 0 for s, st in zip(t.shape, t.stride())):
        raise ValueError(f"{name} is broadcast")
    return t.data_ptr()


def _packed(t, name, dtypes, shape, device):
    """_check of a tensor that must be contiguous."""
    p = _check(t, name, dtypes, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return p


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _stream_of(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, not {device}")
    return C.c_void_p(stream.cuda_stream)


class Cache:
    """The operators on one cache layout (``spec``: n_q_heads, head_dim, kv_dim, block_size,
    kv_record_bytes, as in a layer's spec), with a workspace for steps of up to ``max_rows`` rows
    of ``max_requests`` requests on the current device.  Calls on one Cache share the workspace:
    order them on the GPU."""

    def __init__(self, spec: dict, max_rows: int, max_requests: int):
        import torch
        self.spec = {k: int(spec[k]) for k in ("n_q_heads", "head_dim", "kv_dim", "block_size",
                                               "kv_record_bytes")}
        self._h = C.c_void_p()
        self.max_rows, self.max_requests = int(max_rows), int(max_requests)
        s = CacheSpec(**self.spec, max_rows=self.max_rows, max_req=self.max_requests)
        rc = _lib().mono_cache_build(C.byref(s), C.byref(self._h))
        if rc != _m.MONO_OK:
            raise _m.MonoError(rc, "mono_cache_build")
        self.device = torch.device("cuda", torch.cuda.current_device())

    def _view(self, t, name):
        import torch
        if t.dim() != 3 or t.dtype != torch.uint8 or t.device != self.device:
            raise ValueError(f"{name} is a uint8 [blocks, block_size, record] view on {self.device}")
        if t.shape[1] != self.spec["block_size"] or t.shape[2] < self.spec["kv_record_bytes"] \
                or t.stride(2) != 1:
            raise ValueError(f"{name}: pages of {self.spec['block_size']} records of "
                             f"{self.spec['kv_record_bytes']} contiguous bytes expected, got shape "
                             f"{tuple(t.shape)}, strides {t.stride()}")
        return t.data_ptr(), t.stride(0), t.stride(1), t.shape[0]

    def attend(self, q, o, positions, row_req, block_table, kv_cache, *, window=0, sinks=0,
               causal=True, scale=None, lse=None, weights=None, stream=None) -> None:
        """Attention of q's rows (bf16 [rows, n_q_heads * head_dim]) over the cached tokens of
        their requests, into o (bf16, like q).  ``window`` 0 is the whole context, else the last
        ``window`` tokens and the first ``sinks``; ``lse`` (f32 [rows, n_q_heads]) gets the
        log-sum-exp of the scores, ``weights`` (f32 [n_req, tokens]) each token's attention weight
        added."""
        import torch
        s, dev = self.spec, self.device
        rows, n_req, width = q.shape[0], block_table.shape[0], s["n_q_heads"] * s["head_dim"]
        i32 = (torch.int32,)
        a = AttendArgs(
            q=_check(q, "q", (torch.bfloat16,), (rows, width), dev),
            o=_check(o, "o", (torch.bfloat16,), (rows, width), dev),
            q_stride=_row_stride(q), o_stride=_row_stride(o),
            positions=_packed(positions, "positions", i32, (rows,), dev),
            row_req=_packed(row_req, "row_req", i32, (rows,), dev),
            block_table=_packed(block_table, "block_table", i32, (None, None), dev),
            max_blocks=block_table.shape[1], n_req=n_req, rows=rows, window=window, sinks=sinks,
            causal=int(bool(causal)), scale=0.0 if scale is None else float(scale))
        if scale is not None and not scale > 0:
            raise ValueError("scale must be positive")
        a.kv_cache, a.kv_stride_block, a.kv_stride_tok, a.kv_num_blocks = self._view(kv_cache,
                                                                                    "kv_cache")
        if lse is not None:
            a.lse = _packed(lse, "lse", (torch.float32,), (rows, s["n_q_heads"]), dev)
        if weights is not None:
            a.weights = _check(weights, "weights", (torch.float32,), (n_req, None), dev)
            a.weights_stride = _row_stride(weights)
        self._call("mono_cache_attend", a, stream)

    def evict(self, weights, lengths, block_table, kv_cache, kept, new_lengths, *, budget,
              sinks=0, recent=0, weights_out=None, dst_table=None, dst_cache=None,
              stream=None) -> None:
        """Keeps ``budget`` tokens of each request (its first ``sinks``, its last ``recent`` and
        the heaviest of the others by ``weights``, f32 [n_req, tokens]) and moves their records and
        weights, in order, to the front of its pages, or to those of ``dst_table`` (in
        ``dst_cache``).  kept (int32 [n_req, >= budget]) gets the old slots, new_lengths the
        counts."""
        import torch
        dev, f32, i32 = self.device, (torch.float32,), (torch.int32,)
        n_req = block_table.shape[0]
        a = EvictArgs(
            weights=_check(weights, "weights", f32, (n_req, None), dev),
            weights_stride=_row_stride(weights),
            lengths=_packed(lengths, "lengths", i32, (n_req,), dev),
            new_lengths=_packed(new_lengths, "new_lengths", i32, (n_req,), dev),
            kept=_check(kept, "kept", i32, (n_req, None), dev),
            budget=budget, sinks=sinks, recent=recent, n_req=n_req,
            block_table=_packed(block_table, "block_table", i32, (None, None), dev),
            max_blocks=block_table.shape[1])
        if kept.shape[1] < budget:
            raise ValueError(f"kept holds {kept.shape[1]} slots a request, the budget is {budget}")
        a.kept_stride = _row_stride(kept)
        a.kv_cache, a.kv_stride_block, a.kv_stride_tok, a.kv_num_blocks = self._view(kv_cache,
                                                                                    "kv_cache")
        if weights_out is not None:
            a.weights_out = _check(weights_out, "weights_out", f32, (n_req, None), dev)
            a.weights_out_stride = _row_stride(weights_out)
        if dst_table is not None:
            a.dst_table = _packed(dst_table, "dst_table", i32, (n_req, None), dev)
            a.dst_max_blocks = dst_table.shape[1]
        if dst_cache is not None:
            if dst_table is None:
                raise ValueError("dst_cache needs a dst_table")
            a.dst_cache, a.dst_stride_block, a.dst_stride_tok, a.dst_num_blocks = self._view(
                dst_cache, "dst_cache")
        self._call("mono_cache_evict", a, stream)

    def _call(self, name, args, stream):
        import torch
        if not self._h:
            raise ValueError("the Cache is closed")
        with torch.cuda.device(self.device):
            rc = getattr(_lib(), name)(self._h, C.byref(args), _stream_of(stream, self.device))
        if rc != _m.MONO_OK:
            raise _m.MonoError(rc, name)

    def status(self, clear: bool = False) -> int:
        """The handle's MONO_STATUS_* bits (waits for the device)."""
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
    import torch
    dev = target.device
    if dev.type != "cuda":
        raise ValueError("target is not a CUDA tensor")
    dtypes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    i32, f32 = (torch.int32,), (torch.float32,)
    rows, n_req = target.shape[0], row_start.shape[0] - 1
    a = VerifyArgs(
        target=_check(target, "target", tuple(dtypes), (rows, None), dev),
        target_stride=_row_stride(target), dtype=dtypes[target.dtype], vocab=target.shape[1],
        rows=rows, n_req=n_req, row_start=_packed(row_start, "row_start", i32, (None,), dev),
        draft_tokens=_packed(draft_tokens, "draft_tokens", i32, (rows,), dev),
        u=_packed(u, "u", f32, (rows,), dev), r=_packed(r, "r", f32, (n_req,), dev),
        accepted=_packed(accepted, "accepted", i32, (n_req,), dev),
        tokens=_packed(tokens, "tokens", i32, (rows,), dev))
    if draft is not None:
        a.draft = _check(draft, "draft", (target.dtype,), tuple(target.shape), dev)
        a.draft_stride = _row_stride(draft)
    if greedy is not None:
        a.greedy = _packed(greedy, "greedy", i32, (n_req,), dev)
    with torch.cuda.device(dev):
        rc = _lib().mono_verify_drafts(C.byref(a), _stream_of(stream, dev))
    if rc != _m.MONO_OK:
        raise _m.MonoError(rc, "mono_verify_drafts")
