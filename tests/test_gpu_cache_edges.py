"""More of the cache operators on the GPU, against the same 64-bit references: steps whose work goes
round the kernels' rings many times and unevenly, records that no row is to see, views of larger
tensors, other streams."""
import numpy as np
import pytest
import torch

from tests import cache_oracle as co
from tests.test_gpu_cache_ops import (BIG, FULL, ODD, TINY, WIDE, _m, check_verify, make_cache, make_q,
                                      run_attend, run_verify)

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


def fill_unseen(spec, table, cache, seen, scale, rng):
    """Ordinary codes under a finite scale in every slot that holds no token of `seen` ((b, t) pairs)."""
    kv, bs = spec["kv_dim"], spec["block_size"]
    keep = np.zeros(cache.shape[:2], bool)
    for b, t in seen:
        keep[table[b, t // bs], t % bs] = True
    cache[~keep, :kv] = rng.integers(0, 0x7F, (int((~keep).sum()), kv)) | rng.choice(
        [0, 0x80], (int((~keep).sum()), kv)).astype(np.int64)
    cache[~keep, kv:kv + 4] = np.frombuffer(np.float32(scale).tobytes(), np.uint8)


SCALES = [8.0, -50.0, 1e4, 1e30, 2.9e38]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("spec", [FULL, TINY, ODD], ids=["pages128", "pages16", "pages7"])
@pytest.mark.parametrize("rows", [1, 2, 6])
def test_attend_finite_scales_outside_the_view(spec, rows, scale):
    """Page tails, tokens outside the window and later tokens hold any finite scale: no row is to
    notice."""
    m = _m()
    rng = np.random.default_rng(rows)
    for L, window, sinks in ((rows, 0, 0), (100, 0, 0), (301, 0, 0), (900, 130, 3)):
        table, cache = make_cache(spec, [L + 40], 200 + L)
        pos = list(range(L - rows, L))
        first = max(0, pos[0] - window + 1) if window else 0
        fill_unseen(spec, table, cache, [(0, t) for t in range(L) if t >= first or t < sinks], scale, rng)
        q = make_q(spec, rows, L)
        o, lse, w, st = run_attend(m, spec, q, pos, [0] * rows, table, cache, window=window, sinks=sinks,
                                   weights=torch.zeros((1, L)))
        eo, tol, el, ltol, ew, wtol = co.attend(spec, q.double().numpy(), pos, [0] * rows, table, cache,
                                                window, sinks, n_weights=L)
        assert st == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()
        assert (np.abs(w - ew) <= wtol + 2.0 ** -24 * (rows * spec["n_q_heads"] + 2) * ew).all()


@pytest.mark.parametrize("scale", SCALES[:3])
def test_attend_finite_scales_left_in_shared_memory(scale):
    """Boxes of a tile that are not loaded keep what a call before left there."""
    m = _m()
    dev = torch.device("cuda")
    n = 16 * 10240  # eight tiles and more for every SM
    pool = torch.randint(0, 4, (n // 16, 16, 80), dtype=torch.uint8, device=dev)
    pool[..., 64:68] = torch.tensor([scale], device=dev).view(torch.uint8)
    pages = torch.arange(n // 16, dtype=torch.int32, device=dev)[None].contiguous()
    h = m.Cache(TINY, 1, 1)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    for L in (1, 17, 40, 1000):
        table, cache = make_cache(TINY, [L], 300 + L)
        q = make_q(TINY, 1, L)
        big, out = q.to(dev), torch.empty_like(q, device=dev)
        h.attend(big, out, zero + n - 1, zero, pages, pool)
        o, lse, _, st = run_attend(m, TINY, q, [L - 1], [0], table, cache, handle=h)
        eo, tol, el, ltol, _, _ = co.attend(TINY, q.double().numpy(), [L - 1], [0], table, cache)
        assert st == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()
    h.close()


ONE = dict(n_q_heads=1, head_dim=64, kv_dim=64, block_size=16, kv_record_bytes=80)


@pytest.mark.parametrize("scale", SCALES[:1] + [100.0, 1e4])
def test_attend_blocks_far_below_the_reference(scale):
    """Whole blocks of 32 tokens in view with large scales and scores too low to count: their weights
    are zeros, whatever their values.  (Scores to -10^6: 2^-126 of the largest weight is the least that
    an f32 holds, times at most 448 times the scale: nothing that the bound has not.)"""
    m = _m()
    L, low = 700, {*range(32, 64), *range(192, 256)}
    table, cache = make_cache(ONE, [L], 31)
    q = make_q(ONE, 1, 31)
    away = np.where(q[0].float().numpy() > 0, 0xB8, 0x38).astype(np.uint8)  # -1 and 1
    for t in low:
        rec = cache[table[0, t // 16], t % 16]
        rec[:64] = away
        rec[64:68] = np.frombuffer(np.float32(scale).tobytes(), np.uint8)
    o, lse, _, st = run_attend(m, ONE, q, [L - 1], [0], table, cache)
    seen = [t for t in range(L) if t not in low]
    rec = np.stack([cache[table[0, t // 16], t % 16] for t in seen])
    k = co.E4M3[rec[:, :64]] * np.ascontiguousarray(rec[:, 64:68]).view(np.float32)
    s = k @ q[0].double().numpy() / 8.0
    w = np.exp(s - s.max())
    eo = w / w.sum() @ k
    es = 2.0 ** -16 * (np.abs(k) @ np.abs(q[0].double().numpy()) / 8.0).max()
    tol = 2.0 ** -8 * np.abs(eo) + (2.0 ** -8 + 2 * es + 2.0 ** -12) * (w / w.sum() @ np.abs(k) + np.abs(eo))
    assert st == 0 and (np.abs(o[0] - eo) <= tol).all()
    assert abs(lse[0, 0] - (s.max() + np.log(w.sum()))) <= es + 2.0 ** -18 + 2.0 ** -20


@pytest.mark.parametrize("bad", ["nan", "inf_scale"])
def test_attend_weights_of_tokens_between_windows(bad):
    """Rows of one request far apart, with windows that leave tokens between them to nobody: what
    those hold reaches no weight, also where a pass has fewer rows than it could."""
    m = _m()
    dev = torch.device("cuda")
    table, cache = make_cache(FULL, [1100, 700], 41)
    pos, req = [1099, 10, 699, 650, 40], [0, 0, 1, 1, 1]
    seen = {(b, t) for b, p in zip(req, pos) for t in range(p - 4, p + 1)}
    for b, L in enumerate((1100, 700)):
        for t in range(L):
            if (b, t) not in seen:
                rec = cache[table[b, t // 128], t % 128]
                if bad == "nan":
                    rec[:] = 0x7F
                else:
                    rec[512:516] = np.frombuffer(np.float32(np.inf).tobytes(), np.uint8)
    q = make_q(FULL, 5, 41)
    o, _, w, st = run_attend(m, FULL, q, pos, req, table, cache, window=5, weights=torch.ones((2, 1100)))
    eo, tol, _, _, ew, wtol = co.attend(FULL, q.double().numpy(), pos, req, table, cache, 5,
                                        n_weights=1100)
    assert st == 0 and (np.abs(o - eo) <= tol).all()
    assert (np.abs(w - 1 - ew) <= wtol + 2.0 ** -24 * (1 + (5 * 64 + 2) * ew)).all()
    assert (w[ew == 0] == 1).all()


def test_status_waits_for_every_stream():
    """A call behind long work on a stream of torch's own: its status is there without a wait by the
    caller, and a cleared word stays clear."""
    m = _m()
    dev = torch.device("cuda")
    table, cache = make_cache(TINY, [300], 42)
    table[0, 3] = -1
    i32 = dict(dtype=torch.int32, device=dev)
    q = make_q(TINY, 1, 42).to(dev)
    args = (torch.empty_like(q), torch.tensor([299], **i32), torch.tensor([0], **i32),
            torch.from_numpy(table).to(dev), torch.from_numpy(cache).to(dev))
    h = m.Cache(TINY, 1, 1)
    s, a = torch.cuda.Stream(), torch.randn((8192, 8192), device=dev)
    torch.mm(a, a)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            for _ in range(5):
                torch.mm(a, a)
            h.attend(q, *args)
        assert h.status(clear=True) == 1
        assert h.status() == 0
    h.close()
    with pytest.raises(ValueError):
        h.status()


def test_weights_in_views_of_wider_tensors():
    """Columns before and behind a view of weights, in and out, are left as they were; the last row's
    end is the storage's."""
    m = _m()
    dev = torch.device("cuda")
    lengths = [200, 333]
    table, cache = make_cache(TINY, lengths, 43)
    q = make_q(TINY, 2, 43)
    want, *_ = run_attend(m, TINY, q, [199, 332], [0, 1], table, cache, weights=torch.ones((2, 150)))[2:]
    big = torch.full((2, 300), 7.0, device=dev)
    view = big[:, 150:]
    view.fill_(1.0)
    h = m.Cache(TINY, 2, 2)
    i32 = dict(dtype=torch.int32, device=dev)
    t, c = torch.from_numpy(table).to(dev), torch.from_numpy(cache).to(dev)
    h.attend(q.to(dev), torch.empty_like(q, device=dev), torch.tensor([199, 332], **i32),
             torch.tensor([0, 1], **i32), t, c, weights=view)
    assert h.status() == 0 and (big[:, :150] == 7).all()
    assert np.array_equal(view.double().cpu().numpy(), want)
    # an eviction of 150 columns' tokens into 40, of which 64 cannot be kept
    w = view.cpu().numpy()
    out = torch.full((2, 100), 5.0, device=dev)
    ln, kept = torch.tensor([150, 150], **i32), torch.zeros((2, 64), **i32)
    h.evict(view, ln, t, c, kept, ln, budget=64, sinks=2, recent=9, weights_out=out[:, 60:])
    assert h.status() == 0 and ln.tolist() == [64, 64]
    keep = co.evict(w, [150, 150], 64, 2, 9)
    assert kept.tolist() == keep and (out[:, :60] == 5).all()
    assert np.array_equal(out[:, 60:].cpu().numpy(), np.stack([w[b, k[:40]] for b, k in enumerate(keep)]))
    # lengths beyond a view's columns are cut to them
    ln = torch.tensor([199, 100], **i32)
    h.evict(big[:, :120], ln, t, c, kept, ln, budget=64)
    assert h.status(clear=True) == 1 and ln.tolist() == [64, 64] and kept.max() < 120
    h.close()


# -------------------------------------------------------------------------- verification
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tiny", [2.0 ** -24, 3 * 2.0 ** -24])
def test_verify_small_entries_beside_large_ones(dtype, tiny):
    """Entries that an f32 sum with their neighbours would lose decide where a threshold falls."""
    m = _m()
    V = 4096
    p = torch.zeros((2, V), dtype=torch.float64)
    p[:, ::8] = 1.0
    p[0, :V // 2].view(-1, 8)[:, [2, 4, 6]] = tiny
    p[1, V // 2:].view(-1, 8)[:, [1, 3, 5, 7]] = tiny
    assert torch.equal(p.to(dtype).double(), p)
    rows = p.to(dtype).cuda().repeat_interleave(200, 0)
    r = np.concatenate([np.arange(312, 512), np.arange(0, 200)]).astype(np.float32) / 512
    check_verify(m, rows, None, [0] * 400, list(range(401)), np.zeros(400, np.float32), r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_verify_residuals_of_unlike_sizes(dtype):
    """p - q of a large p and a small q takes more bits than an f32 has."""
    m = _m()
    V, n = 4096, 200
    p, q = torch.zeros((2 * n, V), dtype=torch.float64), torch.zeros((2 * n, V), dtype=torch.float64)
    p[:, ::8] = 16.0
    q[:, V // 2::8] = 2.0 ** -24 * 3  # (an f32 difference loses it)
    tok = [1, 0] * n  # (p is 0 there: refused)
    r = np.arange(312, 512).astype(np.float32) / 512
    check_verify(m, p.to(dtype).cuda(), q.to(dtype).cuda(), tok, list(range(0, 2 * n + 1, 2)),
                 np.full(2 * n, 0.5, np.float32), r)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_verify_infinite_draft_entries(dtype):
    """An infinite q takes all of a finite p; the largest finite p stands against it."""
    m = _m()
    g = torch.Generator().manual_seed(61)
    p, q = torch.rand((60, 999), generator=g), torch.rand((60, 999), generator=g)
    q[:, ::3] = float("inf")
    q[:, 1::5] = float("nan")
    p[:, 4] = -float("inf")
    r = torch.rand(30, generator=g).numpy()
    check_verify(m, p.to(dtype).cuda(), q.to(dtype).cuda(), [0] * 60, list(range(0, 61, 2)),
                 np.full(60, 0.999, np.float32), r)


def test_verify_thresholds_on_a_border():
    """Two copies of some entries with zeros between them, and a threshold at half their sum: the last
    of the first copy or the first of the second, as roundings fall, but one of them.  (Entries span
    30 binades: their sums take more bits than two f32 hold, and differ in their last ones by the order
    of the additions.)"""
    m = _m()
    rng = np.random.default_rng(0)
    n, V = 3000, 1024
    p, ends = np.zeros((n, V), np.float32), []
    for row in p:
        few = rng.integers(3, 10)
        room = rng.integers(few, 13)
        vals = rng.random(few) * 2.0 ** rng.integers(-30, 0, few)
        first = rng.permutation(room)[:few]
        second = room + rng.integers(1, 4) + rng.permutation(16)[:few]
        row[4 * first], row[4 * second] = vals, vals
        ends.append((4 * first.max(), 4 * second.min()))
    acc, out = run_verify(m, torch.from_numpy(p).cuda(), None, [0] * n, list(range(n + 1)),
                          np.zeros(n, np.float32), np.full(n, 0.5, np.float32))
    assert acc == [0] * n
    assert all(x in e for x, e in zip(out, ends)), [(x, e) for x, e in zip(out, ends) if x not in e][:5]


# -------------------------------------------------------------------------------- limits
def test_tables_beyond_the_indices_are_refused():
    m = _m()
    spec = dict(TINY, block_size=65535)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = torch.zeros((1, 65535, 80), dtype=torch.uint8, device="cuda")
    q = torch.zeros((1, 256), dtype=torch.bfloat16, device="cuda")
    zero, w = torch.zeros(1, **i32), torch.zeros((1, 64), device="cuda")
    h = m.Cache(spec, 1, 1)
    table = torch.full((1, 32768), -1, **i32)
    table[0, 0] = 0
    for n, ok in ((32768, False), (32767, True)):  # 2^31 - 2^15; 2^31 - 2^16 - 2^15 + 1 tokens
        t = table[:, :n].contiguous()
        calls = [lambda: h.attend(q, torch.empty_like(q), zero, zero, t, pool),
                 lambda: h.evict(w, zero, t, pool, torch.zeros((1, 8), **i32), zero.clone(), budget=8)]
        for call in calls:
            if ok:
                call()
            else:
                with pytest.raises(m.MonoError) as e:
                    call()
                assert e.value.code == -1
    # the last token that the table could hold lies on no page: nothing is read for it
    o = torch.full_like(q, float("nan"))
    h.attend(q, o, torch.full((1,), 32767 * 65535 - 1, **i32), zero, table[:, :32767].contiguous(), pool,
             window=300)
    assert h.status() == 1 and not o.any()
    h.close()


def test_the_largest_budget():
    """kept is filled up to the budget, with indices that a 32-bit step would pass."""
    m = _m()
    i32 = dict(dtype=torch.int32, device="cuda")
    n = 2 ** 31 - 1
    kept = torch.zeros((1, n), **i32)
    h = m.Cache(TINY, 1, 1)
    h.evict(torch.ones((1, 64), device="cuda"), torch.tensor([50], **i32), torch.arange(4, **i32)[None],
            torch.zeros((4, 16, 80), dtype=torch.uint8, device="cuda"), kept, torch.zeros(1, **i32), budget=n)
    assert h.status() == 0 and kept[0, :50].tolist() == list(range(50))
    assert all(bool((kept[0, i:i + 2 ** 28] == -1).all()) for i in range(50, n, 2 ** 28))
    h.close()


# ------------------------------------------------------------------------- ends of the range
@pytest.mark.parametrize("rows", [1, 6], ids=["narrow", "wide"])
@pytest.mark.parametrize("exponent", [60, 63.9, 70, 100, 126])
def test_attend_largest_scales(rows, exponent):
    """Scales up to 2^64 count as they are; rows that see a larger one are NaN, the others as without
    it (and NaN where their own scores are beyond 2^26)."""
    m = _m()
    L = 300
    table, cache = make_cache(TINY, [L], 51)
    rng = np.random.default_rng(51)
    for t in range(L):
        rec = cache[table[0, t // 16], t % 16]
        s = np.float32(2.0 ** exponent * (1 if t == 294 else rng.uniform(0.5, 1) if exponent < 64 else 2.0 ** -90))
        rec[64:68] = np.frombuffer(s.tobytes(), np.uint8)
    q = make_q(TINY, rows, 51)
    pos = [296 - i for i in range(rows)]
    k = 0.125 * 2.0 ** -exponent if exponent < 64 else 0.125
    args = dict(scale=k, weights=torch.zeros((1, L)))
    o, lse, w, st = run_attend(m, TINY, q, pos, [0] * rows, table, cache, **args)
    eo, tol, el, ltol, _, _ = co.attend(TINY, q.double().numpy(), pos, [0] * rows, table, cache, scale=k)
    sees = np.array([p >= 294 and exponent >= 64 for p in pos])
    far = np.abs(el) > 2.0 ** 26
    assert np.isnan(lse[far]).all() and np.isnan(o.reshape(rows, 4, 64)[far]).all()
    sees |= far.any(1)
    assert st == 0 and np.isnan(o[sees]).all() and np.isnan(lse[sees]).all()
    assert (np.abs(o - eo) <= tol)[~sees].all() and (np.abs(lse - el) <= ltol)[~sees].all()


@pytest.mark.parametrize("rows", [1, 6], ids=["narrow", "wide"])
@pytest.mark.parametrize("L", [200, 40000], ids=["one_piece", "pieces"])
def test_attend_scores_beyond_f32(rows, L):
    """A score that an f32 cannot hold makes its head NaN, not 0."""
    m = _m()
    dev = torch.device("cuda")
    n = -(-L // 16)
    pool = torch.full((n, 16, 80), 0x38, dtype=torch.uint8, device=dev)  # codes of 1.0
    pool[..., 64:68] = torch.tensor([1.0], device=dev).view(torch.uint8)
    q = torch.ones((rows, 256), dtype=torch.bfloat16)
    q[:, 64:128] = 0.0
    pos = [L - 1] * rows
    table = np.arange(n, dtype=np.int32)[None]
    o, lse, _, st = run_attend(m, TINY, q, pos, [0] * rows, table, pool, scale=1e38)
    o = o.reshape(rows, 4, 64)
    assert st == 0 and np.isnan(o[:, [0, 2, 3]]).all() and not np.isfinite(lse[:, [0, 2, 3]]).any()
    # (the second head's scores are zeros)
    assert (o[:, 1] == 1).all() and np.abs(lse[:, 1] - np.log(L)).max() <= 2.0 ** -18


@pytest.mark.parametrize("rows", [1, 6], ids=["narrow", "wide"])
@pytest.mark.parametrize("sign", [1, -1])
def test_attend_scores_near_and_beyond_the_limit(rows, sign):
    """One key's scores, all alike but for one token: at 2^25 the weights of the others are as they
    should be, beyond 2^26 a head is NaN, never 0."""
    m = _m()
    dev = torch.device("cuda")
    L = 900
    n = -(-L // 16)
    pool = torch.full((n, 16, 80), 0x38, dtype=torch.uint8, device=dev)
    pool[..., 64:68] = torch.tensor([1.0], device=dev).view(torch.uint8)
    q = torch.full((rows, 256), float(sign), dtype=torch.bfloat16)
    table = np.arange(n, dtype=np.int32)[None]
    for power, fine in ((10, True), (25, True), (28, False), (40, False), (90, False)):
        o, lse, _, st = run_attend(m, TINY, q, [L - 1] * rows, [0] * rows, table, pool, scale=2.0 ** (power - 6))
        assert st == 0
        if fine:  # (a score is exact; its reference is a multiple of 2 there, o a sum of equal weights)
            assert (o == 1).all() and np.abs(lse - sign * 2.0 ** power - np.log(L)).max() <= 2.0 ** (power - 22)
        else:
            assert np.isnan(o).all() and np.isnan(lse).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_infinite_target_entries(dtype, draft):
    """An infinite entry leaves nothing to draw from, in a residual and in a last row."""
    m = _m()
    g = torch.Generator().manual_seed(62)
    p, q = torch.rand((6, 999), generator=g), torch.rand((6, 999), generator=g)
    p[:, 500] = float("inf")
    q[0, 500] = float("inf")
    tok = [0, 0, 500, 0, 0, 0]  # the first draft falls, the second request's stands
    u = np.array([0.999999, 0, 0.5, 0, 0, 0], np.float32)
    p[0, 0] = 0.0
    acc, out = run_verify(m, p.to(dtype).cuda(), q.to(dtype).cuda() if draft else None, tok, [0, 2, 4, 6], u,
                          np.full(3, 0.5, np.float32))
    assert acc[:2] == [0, 1] and out[:4] == [-1, -1, 500, -1]
