"""Appending and rotating: the C structures, and what the binding hands over or refuses, on the CPU."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import moe_decode_layer_mxfp8_gb300 as m
from moe_decode_layer_mxfp8_gb300 import cache as mc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SPEC = dict(n_q_heads=4, head_dim=64, kv_dim=128, block_size=16, kv_record_bytes=144)


def flat(struct, prefix="", at=0):
    """(name, offset) of every field, those of nested structures one by one."""
    for n, t in struct._fields_:
        o = at + getattr(struct, n).offset
        if issubclass(t, C.Structure):
            yield from flat(t, prefix + n + ".", o)
        else:
            yield prefix + n, o


def test_struct_layout_matches_header(tmp_path):
    structs = [("mono_rope", mc.Rope), ("mono_append_args", mc.AppendArgs), ("mono_rotate_args", mc.RotateArgs)]
    body = "".join(f'  printf("%zu\\n", sizeof({c}));\n' + "".join(
        f'  printf("%zu\\n", offsetof({c}, {n}));\n' for n, _ in flat(s)) for c, s in structs)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "mono_cache.h"\nint main(void) {\n' + body + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    want = []
    for _, s in structs:
        want += [C.sizeof(s)] + [o for _, o in flat(s)]
    assert [int(v) for v in got] == want
    for (_, s), packed in zip(structs[1:], (mc._APPEND, mc._ROTATE)):
        assert packed.size == C.sizeof(s)
        fields = list(flat(s))
        data = packed.pack(*range(1, len(fields) + 1))
        for i, (_, o) in enumerate(fields):
            assert data[o] == i + 1


class Caught(m.Cache):
    """A Cache on host tensors whose calls end before the library."""

    def __init__(self):
        self.spec, self.max_rows, self.max_requests = dict(SPEC), 8, 4
        self.device, self._dev, self._width, self._h = torch.device("cpu"), -1, 256, None

    def _call(self, name, args, stream):
        kind = {"mono_cache_append": mc.AppendArgs, "mono_cache_rotate": mc.RotateArgs}[name]
        assert len(args) == C.sizeof(kind)
        self.args = kind.from_buffer_copy(args)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def append(**kw):
    h = Caught()
    d = dict(kv=torch.zeros((3, 128), dtype=torch.bfloat16), positions=i32(3), row_req=i32(3),
             block_table=i32(2, 5), kv_cache=torch.zeros((4, 16, 144), dtype=torch.uint8))
    h.append(**dict(d, **kw))
    return h.args


def rotate(**kw):
    h = Caught()
    x = torch.zeros((3, 192), dtype=torch.float16)
    h.rotate(**dict(dict(x=x, out=x, positions=i32(3), rope=torch.zeros((9, 32))), **kw))
    return h.args


def test_append_hands_over_what_it_was_given():
    a = append()
    assert (a.rows, a.n_req, a.max_blocks, a.dtype, a.rope.table, a.q, a.q_out) == (3, 2, 5, 1, None, None, None)
    big, q, rope = torch.zeros((3, 400)), torch.zeros((3, 256)), torch.zeros((9, 40))
    a = append(kv=big[:, 16:144], q=q, rope=rope[:, 4:36], rope_positions=i32(3), interleaved=True)
    assert (a.kv, a.kv_stride, a.dtype) == (big.data_ptr() + 64, 400, 0)
    assert (a.q, a.q_out, a.q_stride, a.q_out_stride) == (q.data_ptr(), q.data_ptr(), 256, 256)
    r = a.rope
    assert (r.table, r.stride, r.positions, r.dim, r.offset) == (rope.data_ptr() + 16, 40, 9, 32, 32)
    assert (r.interleaved, r.inverse) == (1, 0) and a.rope_positions
    assert append(rope=rope[:, :16], rope_offset=8).rope.offset == 8


def test_rotate_hands_over_what_it_was_given():
    a = rotate(inverse=True)
    assert (a.rows, a.heads, a.dtype, a.x == a.out) == (3, 3, 2, True)
    assert (a.rope.dim, a.rope.offset, a.rope.interleaved, a.rope.inverse) == (32, 32, 0, 1)


@pytest.mark.parametrize("kw", [
    dict(kv=torch.zeros((3, 128), dtype=torch.float64)), dict(kv=torch.zeros((3, 127))),
    dict(kv=torch.zeros((1, 128)).expand(3, 128)), dict(kv=torch.zeros((128, 3)).T),
    dict(positions=i32(4)), dict(positions=torch.zeros(3, dtype=torch.int64)), dict(row_req=i32(2)),
    dict(block_table=i32(2, 6)[:, :5]), dict(kv_cache=torch.zeros((4, 15, 144), dtype=torch.uint8)),
    dict(kv_cache=torch.zeros((4, 16, 143), dtype=torch.uint8)), dict(q=torch.zeros((3, 256), dtype=torch.bfloat16)),
    dict(q_out=torch.zeros((3, 256), dtype=torch.bfloat16)), dict(rope_positions=i32(3)), dict(rope_offset=0),
    dict(rope=torch.zeros((9, 32)), q=torch.zeros((3, 256))),
    dict(rope=torch.zeros((9, 32)), q=torch.zeros((3, 255), dtype=torch.bfloat16)),
    dict(rope=torch.zeros((9, 32), dtype=torch.bfloat16)), dict(rope=torch.zeros(32)),
    dict(rope=torch.zeros((1, 32)).expand(9, 32)), dict(rope=torch.zeros((9, 32)), rope_positions=i32(2)),
    dict(rope=torch.zeros((9, 32)), rope_offset=2 ** 31)])
def test_append_refuses(kw):
    with pytest.raises(ValueError):
        append(**kw)


@pytest.mark.parametrize("kw", [
    dict(x=torch.zeros((3, 100), dtype=torch.float16)), dict(out=torch.zeros((3, 192))),
    dict(out=torch.zeros((2, 192), dtype=torch.float16)), dict(positions=i32(2)),
    dict(rope=torch.zeros((9, 32)).half()), dict(x=torch.zeros((3, 192), dtype=torch.int16))])
def test_rotate_refuses(kw):
    with pytest.raises(ValueError):
        rotate(**kw)


def test_null_arguments_are_refused():
    from moe_decode_layer_mxfp8_gb300 import build
    build.build()
    lib = mc._lib()
    assert lib.mono_cache_append(None, None, None) == -1
    assert lib.mono_cache_rotate(None, None, None) == -1
