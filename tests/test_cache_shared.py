"""Attention over shared prefixes: the C structure, and what the binding hands over or refuses, on the CPU;
and the reference against the one of whole contexts."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import moe_decode_layer_mxfp8_gb300 as m
from moe_decode_layer_mxfp8_gb300 import cache as mc
from tests import cache_oracle as co
from tests import shared_oracle as so

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SPEC = dict(n_q_heads=4, head_dim=64, kv_dim=128, block_size=16, kv_record_bytes=144)


def test_struct_layout_matches_header(tmp_path):
    s = mc.SharedArgs
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "mono_cache.h"\nint main(void) {\n'
                   '  printf("%zu\\n", sizeof(mono_shared_args));\n' + "".join(
                       f'  printf("%zu\\n", offsetof(mono_shared_args, {f[0]}));\n' for f in s._fields_)
                   + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [C.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    assert mc._SHARED.size == C.sizeof(s)
    vals = list(range(1, len(s._fields_) + 1))
    a = s.from_buffer_copy(mc._SHARED.pack(*vals))
    assert [getattr(a, f[0]) for f in s._fields_] == vals


class Caught(m.Cache):
    """A Cache on host tensors whose calls end before the library."""

    def __init__(self):
        self.spec, self.max_rows, self.max_requests = dict(SPEC), 8, 4
        self.device, self._dev, self._width, self._h = torch.device("cpu"), -1, 256, None

    def _call(self, name, args, stream):
        assert name == "mono_cache_attend_shared" and len(args) == C.sizeof(mc.SharedArgs)
        self.args = mc.SharedArgs.from_buffer_copy(args)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def call(**kw):
    h, q = Caught(), torch.zeros((3, 256), dtype=torch.bfloat16)
    d = dict(q=q, o=torch.zeros_like(q), positions=i32(3), row_req=i32(3), block_table=i32(2, 5),
             kv_cache=torch.zeros((4, 16, 144), dtype=torch.uint8), prefix_table=i32(3, 7), prefix_lengths=i32(3))
    h.attend_shared(**dict(d, **kw))
    return h.args


def test_it_hands_over_what_it_was_given():
    big, lse, of = torch.zeros((3, 400), dtype=torch.bfloat16), torch.zeros((3, 4)), i32(2)
    a = call(q=big[:, 8:264], lse=lse, prefix_of=of, causal=False, scale=0.5)
    assert (a.q, a.q_stride, a.o_stride, a.lse, a.prefix_of) == (big.data_ptr() + 16, 400, 256, lse.data_ptr(),
                                                                 of.data_ptr())
    assert (a.max_blocks, a.n_req, a.prefix_max_blocks, a.n_prefix, a.rows, a.causal, a.scale) == (5, 2, 7, 3, 3, 0, 0.5)
    a = call()
    assert (a.causal, a.scale, a.prefix_of, a.lse) == (1, 0.0, None, None)


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros((3, 256))), dict(q=torch.zeros((3, 255), dtype=torch.bfloat16)),
    dict(o=torch.zeros((2, 256), dtype=torch.bfloat16)), dict(positions=i32(2)), dict(row_req=i32(4)),
    dict(block_table=torch.zeros((2, 5), dtype=torch.int64)), dict(prefix_table=i32(3, 8)[:, :7]),
    dict(prefix_lengths=i32(2)), dict(prefix_of=i32(3)), dict(prefix_of=torch.zeros(2, dtype=torch.int64)),
    dict(lse=torch.zeros((3, 5))), dict(lse=torch.zeros((3, 8))[:, :4]), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=1e39), dict(scale=2.0 ** 20.1), dict(scale=2.0 ** -20.1), dict(kv_cache=torch.zeros((4, 15, 144), dtype=torch.uint8))])
def test_it_refuses(kw):
    with pytest.raises(ValueError):
        call(**kw)


def test_null_arguments_are_refused():
    from moe_decode_layer_mxfp8_gb300 import build
    build.build()
    assert mc._lib().mono_cache_attend_shared(None, None, None) == -1


def test_reference_is_the_attention_of_whole_contexts():
    rng = np.random.default_rng(1)
    cache = rng.integers(0, 0x70, (9, 16, 144), dtype=np.uint8)
    cache[..., 128:132] = np.frombuffer(np.float32(0.01).tobytes(), np.uint8)
    table = np.array([[3, 1, 4, 0], [3, 1, 5, 2]], np.int32)
    q = rng.standard_normal((4, 256))
    pos, req = [50, 51, 20, 60], [0, 0, 1, 1]
    for causal in (True, False):
        want = co.attend(SPEC, q, pos, req, table, cache, causal=causal)
        for lengths, of in (([32], [0, 0]), ([32], [-1, 0]), ([20, 0], [0, 1])):
            got = so.attend(SPEC, q, pos, req, table, cache, table[[0] * len(lengths)], lengths, of, causal)
            assert np.allclose(got[0], want[0], rtol=1e-12) and np.allclose(got[2], want[2], rtol=1e-12)
