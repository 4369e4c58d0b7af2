"""Append, rotation and attention over shared prefixes on the GPU for latents of every number of slices, up to
the widest, with few and many heads a slice, and records with bytes behind them."""
import pytest

from tests.test_gpu_cache_append import check_append
from tests.test_gpu_cache_shared import check

pytestmark = pytest.mark.gpu


def spec(head_dim, slices, heads, block_size=16, more=16):
    kv = head_dim * slices
    return dict(n_q_heads=slices * heads, head_dim=head_dim, kv_dim=kv, block_size=block_size, kv_record_bytes=kv + more)


WIDTHS = ([spec(64, n, 1 + n % 3) for n in range(1, 17)] + [spec(128, n, 1 + n % 4, more=48) for n in range(1, 9)]
          + [spec(64, 16, 16, 32), spec(128, 8, 16, 128), spec(64, 3, 16, 5, 64), spec(128, 5, 11, 8)])
NAMES = [f"{s['head_dim']}x{s['kv_dim'] // s['head_dim']}x{s['n_q_heads']}" for s in WIDTHS]


@pytest.mark.parametrize("s", WIDTHS, ids=NAMES)
def test_append(s):
    for dtype, inter in (("bf16", True), ("f32", False)):
        check_append(s, [70, 9, 131], [40, 9, 3], dtype=dtype, dim=32, interleaved=inter, pads=(0, 7), seed=s["kv_dim"])
    check_append(s, [9, 300], [9, 222], dtype="f16", q=None, seed=1)


@pytest.mark.parametrize("s", WIDTHS, ids=NAMES)
def test_shared(s):
    check(s, [333, 40], [0, 0, 1, -1, 0], [5, 140, 1, 90, 33], [2, 3, 1, 1, 33], seed=s["kv_dim"], pads=(2,), shuffle=True)
    check(s, [2900], [0], [70], [1], seed=3)
    check(s, [129], [0] * 40, [1 + i for i in range(40)], [1] * 40, seed=4, causal=False)
