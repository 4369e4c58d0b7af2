"""Attention over shared prefixes on the GPU where many scores are far below the others, or all are: tokens
whose scores are beyond -2^26 weigh nothing beside ordinary ones, wherever in the context they lie, and a
head that sees no others is NaN.  Against tests/shared_oracle.py without those tokens: a weight of
2^-2^26 is 0 in 64 bits, too."""
import numpy as np
import pytest
import torch

from tests import shared_oracle as so
from tests.test_gpu_cache_shared import LAYOUTS, _m, compare, make_q, make_shared, rows_of, run

pytestmark = pytest.mark.gpu


def lower(spec, cache, tab, b, first, last, power):
    """Tokens [first, last) of a table's row get codes of -1 and scales of 2^power; their pages are left
    out of the table that is returned."""
    bs, kv = spec["block_size"], spec["kv_dim"]
    out = tab.copy()
    assert first % bs == 0 and last % bs == 0
    for i in range(first // bs, last // bs):
        cache[tab[b, i], :, :kv] = 0xB8
        cache[tab[b, i], :, kv:kv + 4] = np.frombuffer(np.float32(2.0 ** power).tobytes(), np.uint8)
        out[b, i] = -1
    return out


def far_below(layout, P, own, ranges, power=26, of=None, rows=None, seed=3):
    """ranges: (first, last) of the prefix's tokens that are far below the others."""
    m, spec = _m(), LAYOUTS[layout]
    of = [0] * len(own) if of is None else of
    ptable, table, cache = make_shared(spec, [P], of, own, seed)
    seen = ptable
    for first, last in ranges:
        seen = np.minimum(seen, lower(spec, cache, ptable, 0, first, last, power))
    pos, req = rows_of([P], of, own, rows or [2] * len(own))
    q = make_q(spec, len(pos), seed).abs() + 1  # (scores of -1 codes: -64 or less, times their scales)
    got = run(m, spec, q, pos, req, table, cache, ptable, [P], of)
    assert got[2] == 0
    o, tol, lse, ltol = so.attend(spec, q.double().numpy(), pos, req, table, cache, seen, [P], of)
    alone = np.isneginf(lse).all(1)  # rows that see none of the others (in their prefix still)
    o[alone] = lse[alone] = np.nan
    compare(got, (o, tol, lse, ltol))


@pytest.mark.parametrize("power", [26, 40, 63])
@pytest.mark.parametrize("layout,ranges", [
    ("tiny", [(0, 32)]), ("many", [(0, 31)]), ("many", [(0, 33)]), ("tiny", [(32, 128)]), ("wide", [(0, 128)]),
    ("full", [(0, 128)]), ("tiny", [(16, 144)]), ("many", [(1, 1000)]), ("full", [(0, 1024)]), ("full", [(256, 512)])])
def test_tokens_of_a_prefix_far_below_the_others(layout, ranges, power):
    far_below(layout, 1100, [9, 150], ranges, power)


@pytest.mark.parametrize("layout", ["full", "wide", "tiny", "three"])
def test_a_whole_prefix_far_below_own_tokens(layout):
    """All pieces of a prefix that every CTA has a part of."""
    for P in (384, 6144):
        far_below(layout, P, [9, 150, 1], [(0, P)])


@pytest.mark.parametrize("layout", ["full", "wide", "tiny"])
def test_every_other_tile_far_below_its_neighbours(layout):
    """One stream of an item sees nothing else, with rows of one block and of two."""
    for phase in (0, 128):
        ranges = [(t, t + 128) for t in range(phase, 2560, 256)]
        far_below(layout, 2700, [3], ranges, rows=[1])
        far_below(layout, 2700, [3, 40, 70], ranges, rows=[1, 40, 70])


def test_own_tokens_far_below_their_prefix():
    m, spec = _m(), LAYOUTS["tiny"]
    ptable, table, cache = make_shared(spec, [160], [0, 0], [400, 64], 5)
    seen = lower(spec, cache, table, 0, 160, 320, 26)
    seen = np.minimum(seen, lower(spec, cache, table, 1, 160, 224, 26))
    pos, req = rows_of([160], [0, 0], [400, 64], [3, 2])
    q = make_q(spec, len(pos), 5).abs() + 1
    got = run(m, spec, q, pos, req, table, cache, ptable, [160], [0, 0])
    assert got[2] == 0
    compare(got, so.attend(spec, q.double().numpy(), pos, req, seen, cache, ptable, [160], [0, 0]))


@pytest.mark.parametrize("layout", ["full", "wide", "tiny", "odd"])
@pytest.mark.parametrize("power,qpower", [(26, 0), (63, 0), (60, 60), (63, 120)])
def test_heads_all_of_whose_scores_are_far_below_0_are_nan(layout, power, qpower):
    """Never 0, however far; other heads of the row are as ever."""
    m, spec = _m(), LAYOUTS[layout]
    dh, nq, kv = spec["head_dim"], spec["n_q_heads"], spec["kv_dim"]
    for P, own in ((300, [5, 140]), (0, [300, 20]), (3000, [1, 1])):
        ptable, table, cache = make_shared(spec, [P], [0, 0], own, 6)
        cache[..., :kv] = 0xB8
        cache[..., kv:kv + 4] = np.frombuffer(np.float32(2.0 ** power).tobytes(), np.uint8)
        pos, req = rows_of([P], [0, 0], own, [2, 1])
        q = torch.ones((3, nq, dh)) * 2.0 ** qpower
        q[:, 1::2] = 0.0  # (these see scores of 0: a mean of the values)
        o, lse, st = run(m, spec, q.reshape(3, -1).to(torch.bfloat16), pos, req, table, cache, ptable, [P], [0, 0])
        o = o.reshape(3, nq, dh)
        assert st == 0 and np.isnan(o[:, 0::2]).all() and np.isnan(lse[:, 0::2]).all()
        # equal weights of equal values: sums of n terms in f32 and one rounding to bf16 of a power of two
        n = np.array(pos)[:, None] + 1
        assert (np.abs(o[:, 1::2] + 2.0 ** power) <= 2.0 ** (power - 8)).all()
        assert (np.abs(lse[:, 1::2] - np.log(n)) <= 2.0 ** -18 + 2.0 ** -22 * np.log(n)).all()


def test_rows_that_see_nothing_are_0_beside_those():
    """No token at all is not the same as tokens far below: o 0 and lse -inf."""
    m, spec = _m(), LAYOUTS["tiny"]
    ptable, table, cache = make_shared(spec, [256], [0, -1], [1, 40], 7)
    ptable[:] = -1
    table[0, 256 // 16] = -1
    cache[..., :64] = 0xB8
    cache[..., 64:68] = np.frombuffer(np.float32(2.0 ** 26).tobytes(), np.uint8)
    q = torch.ones((3, 256)).to(torch.bfloat16)
    o, lse, st = run(m, spec, q, [256, 39, -1], [0, 1, 1], table, cache, ptable, [256], [0, -1])
    assert st == m.STATUS_UNMAPPED_PAGE
    assert not o[[0, 2]].any() and np.isneginf(lse[[0, 2]]).all()
    assert np.isnan(o[1]).all() and np.isnan(lse[1]).all()
