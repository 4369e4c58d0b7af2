"""Operators that append to and read a cache, on the GPU, where offsets pass 32 bits: pages and rows far from
the first one, and long prefixes."""
import numpy as np
import pytest
import torch

from tests import rope_oracle as ro
from tests import shared_oracle as so
from tests.test_gpu_cache_append import expected, same
from tests.test_gpu_cache_shared import LAYOUTS, _m, check, compare, i32, make_q, make_shared, rows_of, run

pytestmark = pytest.mark.gpu
FAR = 5 << 30


def spread(cache):
    """The same pages, 5 GB from the first to the last one."""
    nb, bs, rec = cache.shape
    stride = FAR // (nb - 1) // 16 * 16
    pool = torch.zeros(FAR + bs * rec, dtype=torch.uint8, device="cuda")
    view = pool.as_strided((nb, bs, rec), (stride, rec, 1))
    view.copy_(torch.from_numpy(cache))
    return view


@pytest.mark.parametrize("layout", ["full", "tiny", "many"])
def test_shared_prefixes_in_far_pages(layout):
    m, spec = _m(), LAYOUTS[layout]
    ptable, table, cache = make_shared(spec, [300], [0, 0], [40, 3], 41)
    pos, req = rows_of([300], [0, 0], [40, 3], [3, 2])
    q = make_q(spec, 5, 41)
    got = run(m, spec, q, pos, req, table, spread(cache), ptable, [300], [0, 0])
    assert got[2] == 0
    compare(got, so.attend(spec, q.double().numpy(), pos, req, table, cache, ptable, [300], [0, 0]))


@pytest.mark.parametrize("layout", ["full", "tiny", "many"])
def test_append_to_far_pages(layout):
    m, spec = _m(), LAYOUTS[layout]
    rng = np.random.default_rng(42)
    bs, kv = spec["block_size"], spec["kv_dim"]
    nb = 12
    cache = rng.integers(0, 256, (nb, bs, spec["kv_record_bytes"]), dtype=np.uint8)
    table = rng.permutation(nb).astype(np.int32)[None]
    pos = [i * bs + j for i in range(nb) for j in {0, bs - 1}]
    tab = ro.table(max(pos) + 1, 64)
    x = torch.from_numpy(rng.standard_normal((len(pos), kv)).astype(np.float32))
    view = spread(cache)
    h = m.Cache(spec, 1, 1)
    h.append(x.cuda(), i32(pos), i32([0] * len(pos)), i32(table), view, rope=torch.from_numpy(tab).cuda())
    assert h.status() == 0
    h.close()
    off = spec["head_dim"] - 64
    assert same(view.cpu().numpy(), expected(spec, cache, x.numpy(), tab, pos, pos, [0] * len(pos), table, off, False), kv)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_rotate_far_rows(dtype):
    m = _m()
    stride = (FAR // 2 // 2) // 64 * 64  # elements: the last row begins 5 GB or more from the first one
    pool = torch.zeros(2 * stride + 256, dtype=dtype, device="cuda")
    x = pool.as_strided((3, 256), (stride, 1))
    v = torch.randn((3, 256), generator=torch.Generator().manual_seed(1)).to(dtype)
    x.copy_(v)
    tab = ro.table(9, 64)
    out = torch.zeros((3, 256), dtype=dtype, device="cuda")
    h = m.Cache(LAYOUTS["tiny"], 1, 1)
    for to in (out, x):
        h.rotate(x, to, i32([8, 1, 5]), torch.from_numpy(tab).cuda())
    assert h.status() == 0
    h.close()
    want = torch.from_numpy(ro.rotate(v.float().numpy(), tab, [8, 1, 5], 64, 0, False, dtype=np.float32)).to(dtype)
    assert torch.equal(out.cpu(), want) and torch.equal(x.cpu(), want)


@pytest.mark.parametrize("layout,P", [("tiny", 400001), ("wide", 150000)])
def test_very_long_prefixes(layout, P):
    check(LAYOUTS[layout], [P], [0, 0], [3, 70], [1, 2], seed=43)
