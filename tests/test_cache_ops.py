"""The cache operators' C ABI and their refusals: everything here is decided on the host, before
any device is touched (the addresses are never dereferenced)."""
import ctypes as C
import os
import re
import subprocess

import numpy as np
import pytest

import moe_decode_layer_mxfp8_gb300 as m
from moe_decode_layer_mxfp8_gb300 import cache as mc
from tests import cache_oracle as co

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SPEC = dict(n_q_heads=8, head_dim=64, kv_dim=128, block_size=16, kv_record_bytes=144)


@pytest.fixture(scope="module")
def built():
    from moe_decode_layer_mxfp8_gb300 import build
    build.build()
    return mc._lib()


def test_every_declared_function_is_exported(built):
    text = open(os.path.join(ROOT, "include", "mono_cache.h")).read()
    names = set(re.findall(r"\bint (mono_\w+)\(|\bvoid (mono_\w+)\(", text))
    names = {a or b for a, b in names}
    assert names == set(m.CACHE_EXPORTS)
    for n in names:
        assert hasattr(built, n)


def test_struct_layout_matches_header(tmp_path):
    structs = [("mono_cache_spec", mc.CacheSpec), ("mono_attend_args", mc.AttendArgs),
               ("mono_evict_args", mc.EvictArgs), ("mono_verify_args", mc.VerifyArgs)]
    body = "".join(f'  printf("%zu\\n", sizeof({c}));\n' + "".join(
        f'  printf("%zu\\n", offsetof({c}, {f[0]}));\n' for f in s._fields_) for c, s in structs)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "mono_cache.h"\nint main(void) {\n' + body
                   + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    want = []
    for _, s in structs:
        want += [C.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    assert [int(v) for v in got] == want
    # the binding packs them at once: the same sizes and places
    for (_, s), packed in zip(structs[1:], (mc._ATTEND, mc._EVICT, mc._VERIFY)):
        assert packed.size == C.sizeof(s)
        vals = list(range(1, len(s._fields_) + 1))
        a = s.from_buffer_copy(packed.pack(*vals))
        assert [getattr(a, f[0]) for f in s._fields_] == vals


@pytest.mark.parametrize("change,code", [
    (dict(head_dim=96), -2), (dict(kv_dim=96), -2), (dict(kv_dim=1152), -2),
    (dict(n_q_heads=7), -2), (dict(n_q_heads=34), -2), (dict(n_q_heads=0), -2),
    (dict(block_size=0), -2), (dict(kv_record_bytes=128), -2), (dict(kv_record_bytes=150), -2),
    (dict(max_rows=0), -3), (dict(max_rows=1025), -3), (dict(max_req=0), -3),
    (dict(max_req=513), -3)])
def test_bad_layouts_are_refused(built, change, code):
    s = mc.CacheSpec(**dict(SPEC, max_rows=4, max_req=4, **{}) | change)
    h = C.c_void_p(1)
    assert built.mono_cache_build(C.byref(s), C.byref(h)) == code
    assert not h.value


def test_null_arguments_are_refused(built):
    h = C.c_void_p()
    assert built.mono_cache_build(None, C.byref(h)) == -1
    assert built.mono_cache_status(None, 0) == -1
    assert built.mono_cache_attend(None, None, None) == -1
    assert built.mono_cache_evict(None, None, None) == -1
    assert built.mono_verify_drafts(None, None) == -1
    built.mono_cache_free(None)


def _verify_args(**kw):
    a = 0x10000
    d = dict(target=a, draft=a, target_stride=100, draft_stride=100, dtype=0, vocab=100, rows=4,
             n_req=2, row_start=a, draft_tokens=a, u=a, r=a, greedy=None, accepted=a, tokens=a)
    return mc.VerifyArgs(**dict(d, **kw))


@pytest.mark.parametrize("change,code", [
    (dict(target=None), -1), (dict(row_start=None), -1), (dict(u=None), -1), (dict(r=None), -1),
    (dict(accepted=None), -1), (dict(tokens=None), -1), (dict(draft_tokens=None), -1),
    (dict(vocab=0), -1), (dict(rows=0), -1), (dict(n_req=0), -1), (dict(dtype=3), -1),
    (dict(dtype=-1), -1), (dict(target_stride=99), -1), (dict(draft_stride=99), -1),
    (dict(target=0x10002), -4), (dict(draft=0x10001, dtype=1), -4), (dict(u=0x10002), -4),
    (dict(tokens=0x10001), -4)])
def test_verify_refuses(built, change, code):
    assert built.mono_verify_drafts(C.byref(_verify_args(**change)), None) == code


def test_oracle_e4m3_values():
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, co.E4M3, equal_nan=True)


def test_oracle_verification_follows_the_target():
    """Averaged over drafts from q and a grid of random numbers, the first token has
    distribution p: the grid's error is at most a step of u and one of r per token."""
    p = np.array([[0.5, 0.2, 0.25, 0.05], [0.25] * 4])
    q = np.array([[0.1, 0.6, 0.1, 0.2], [0.25] * 4])
    n = 64
    got = np.zeros(4)
    for x in range(4):
        for i in range(n):
            for k in range(n):
                _, out = co.verify(p, q, [x, 0], [0, 2], [(i + 0.5) / n, 0.5], [(k + 0.5) / n])
                got[out[0]] += q[0, x] / n / n
    assert np.abs(got - p[0]).max() <= 2.0 / n


def test_oracle_eviction_by_hand():
    w = np.array([[9.0, 1, 5, 5, 5, 0, 7, 2]])
    assert co.evict(w, [8], 5, 1, 1) == [[0, 2, 3, 6, 7]]
    assert co.evict(w, [4], 5, 1, 1) == [[0, 1, 2, 3]]
