"""What the cache operators' binding hands to the library, on the CPU: the arguments are packed as for
a device, and the call is caught."""
import ctypes as C

import pytest
import torch

import moe_decode_layer_mxfp8_gb300 as m
from moe_decode_layer_mxfp8_gb300 import cache as mc

SPEC = dict(n_q_heads=4, head_dim=64, kv_dim=64, block_size=16, kv_record_bytes=80)


class Caught(m.Cache):
    """A Cache on host tensors whose calls end before the library."""

    def __init__(self):
        self.spec, self.max_rows, self.max_requests = dict(SPEC), 8, 4
        self.device, self._dev, self._width, self._h = torch.device("cpu"), -1, 256, None
        self.args = None

    def _call(self, name, args, stream):
        kind = {"mono_cache_attend": mc.AttendArgs, "mono_cache_evict": mc.EvictArgs}[name]
        assert len(args) == C.sizeof(kind)
        self.args = kind.from_buffer_copy(args)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def attend(**kw):
    h, q = Caught(), torch.zeros((2, 256), dtype=torch.bfloat16)
    d = dict(q=q, o=torch.zeros_like(q), positions=i32(2), row_req=i32(2), block_table=i32(2, 3),
             kv_cache=torch.zeros((4, 16, 80), dtype=torch.uint8))
    h.attend(**dict(d, **kw))
    return h.args


def evict(**kw):
    h = Caught()
    d = dict(weights=torch.zeros((2, 48)), lengths=i32(2), block_table=i32(2, 3),
             kv_cache=torch.zeros((4, 16, 80), dtype=torch.uint8), kept=i32(2, 8), new_lengths=i32(2),
             budget=8)
    h.evict(**dict(d, **kw))
    return h.args


def test_weights_are_as_wide_as_their_view():
    """Not as their rows lie apart: behind a view's columns are another tensor's, or nothing."""
    big = torch.zeros((2, 100))
    a = attend(weights=big[:, 60:])
    assert (a.weights, a.weights_stride, a.weights_cols) == (big.data_ptr() + 240, 100, 40)
    a = attend(weights=big)
    assert (a.weights_stride, a.weights_cols) == (100, 100)
    a = evict(weights=big[:, :48], weights_out=big[:, 90:])
    assert (a.weights_stride, a.weights_cols) == (100, 48)
    assert (a.weights_out_stride, a.weights_out_cols) == (100, 10)
    for call, name in ((attend, "weights"), (evict, "weights"), (evict, "weights_out")):
        with pytest.raises(ValueError):
            call(**{name: big[:, 7:7]})




def test_scales_that_an_f32_does_not_hold_are_refused():
    """A scale that rounds to 0 would be the default one."""
    for scale in (0.0, -1.0, 1e-50, 1e39, float("inf"), float("nan")):
        with pytest.raises(ValueError):
            attend(scale=scale)
    assert attend(scale=2.0 ** -149).scale == 2.0 ** -149
    assert attend().scale == 0.0 and attend(scale=0.25).scale == 0.25


def test_integers_that_32_bits_do_not_hold_are_refused():
    for bad in (2 ** 31, 1.5, None):
        with pytest.raises(ValueError):
            attend(window=bad)
        with pytest.raises(ValueError):
            evict(sinks=bad)
    assert attend(window=2 ** 31 - 1).window == 2 ** 31 - 1
