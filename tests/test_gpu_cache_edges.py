"""More of the cache operators on the GPU, against the same 64-bit references: steps whose work goes
round the kernels' rings many times and unevenly, records that no row is to see, views of larger
tensors, other streams."""
import numpy as np
import pytest
import torch

from tests import cache_oracle as co
from tests.test_gpu_cache_ops import (BIG, FULL, ODD, TINY, WIDE, _m, check_attend, make_cache, make_q,
                                      run_attend)

pytestmark = pytest.mark.gpu


def repeats(m, spec, lengths, rows_per, seed, times=40, weights=False, **kw):
    """One call checked against the reference, then the same bits from every other, with whatever else
    in between that changes who is late (another call's records, a cold cache)."""
    dev = torch.device("cuda")
    table, cache = make_cache(spec, lengths, seed)
    pos = [p for L, n in zip(lengths, rows_per) for p in range(L - n, L)]
    req = [b for b, n in enumerate(rows_per) for _ in range(n)]
    q = make_q(spec, len(pos), seed)
    o, tol, lse, ltol, add, wtol = co.attend(spec, q.double().numpy(), pos, req, table, cache,
                                             n_weights=max(lengths) if weights else 0, **kw)
    h = m.Cache(spec, len(pos), len(lengths))
    a = [torch.tensor(x, dtype=torch.int32, device=dev) for x in (pos, req)]
    t, c, q = torch.from_numpy(table).to(dev), torch.from_numpy(cache).to(dev), q.to(dev)
    cold = torch.empty(1 << 28, dtype=torch.uint8, device=dev)
    first = None
    for i in range(times):
        got = [torch.full_like(q, float("nan")),
               torch.full((len(pos), spec["n_q_heads"]), float("nan"), device=dev)]
        w = torch.zeros((len(lengths), max(lengths)), device=dev) if weights else None
        if i % 4 == 1:
            cold.fill_(i)
        h.attend(q, got[0], a[0], a[1], t, c, lse=got[1], weights=w, **kw)
        got += [w] if weights else []
        torch.cuda.synchronize()
        if first is None:
            first = got
            x, y = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
            assert (np.abs(x - o) <= tol).all() and (np.abs(y - lse) <= ltol).all()
            if weights:
                rnd = 2.0 ** -24 * (len(pos) * spec["n_q_heads"] + 2) * add
                assert (np.abs(w.double().cpu().numpy() - add) <= wtol + rnd).all()
        assert all(torch.equal(x, y) for x, y in zip(first, got))
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("rows", [[7, 6, 8, 6], [1, 6, 6, 2, 6], [3, 7, 8, 1, 6, 6]])
def test_attend_groups_of_few_columns_among_wide_ones(rows):
    """Requests of 6 rows (96 columns) with remainders of 16 and 32 columns, many tiles each."""
    repeats(_m(), FULL, [2900 + 777 * i for i in range(len(rows))], rows, seed=sum(rows))


@pytest.mark.parametrize("spec,lengths,rows", [
    (FULL, [3000 + 128 * i for i in range(8)], [1] * 8), (WIDE, [2111, 6400, 900], [5, 1, 3]),
    (BIG, [4700, 1300], [1, 2]), (TINY, [9000] * 12, [2] * 12)], ids=["full", "wide", "big", "tiny"])
def test_attend_weights_over_many_tiles(spec, lengths, rows):
    """One to eight chunks a tile, runs of tiles of every remainder by four."""
    repeats(_m(), spec, lengths, rows, seed=len(lengths), weights=True)
