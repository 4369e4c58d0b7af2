"""Attention over the cache on the GPU where scores are far below 0: tokens that are seen, and heads that are NaN
and not 0, however far."""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache_ops import TINY, _m, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 6], ids=["narrow", "wide"])
@pytest.mark.parametrize("L", [200, 40000], ids=["one_piece", "pieces"])
@pytest.mark.parametrize("scale", [2.0 ** 26, 2.0 ** 60, 2.0 ** 100, 1e38])
def test_heads_all_of_whose_scores_are_far_below_0_are_nan(rows, L, scale):
    m, dev = _m(), torch.device("cuda")
    n = -(-L // 16)
    pool = torch.full((n, 16, 80), 0x38, dtype=torch.uint8, device=dev)  # codes of 1.0
    pool[..., 64:68] = torch.tensor([1.0], device=dev).view(torch.uint8)
    q = -torch.ones((rows, 256), dtype=torch.bfloat16)
    q[:, 64:128] = 0.0
    table = np.arange(n, dtype=np.int32)[None]
    o, lse, _, st = run_attend(m, TINY, q, [L - 1] * rows, [0] * rows, table, pool, scale=scale)
    o = o.reshape(rows, 4, 64)
    assert st == 0 and np.isnan(o[:, [0, 2, 3]]).all() and np.isnan(lse[:, [0, 2, 3]]).all()
    # (the second head's scores are zeros)
    assert (o[:, 1] == 1).all() and np.abs(lse[:, 1] - np.log(L)).max() <= 2.0 ** -18
