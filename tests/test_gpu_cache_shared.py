"""Attention over shared prefixes on the GPU against tests/shared_oracle.py, whose bounds are derived
there: at the lengths, groups, masks, layouts and values where it can go wrong, captured, on other
streams, beside the attention of whole contexts, and between an append and a rotation back."""
import numpy as np
import pytest
import torch

from tests import rope_oracle as ro
from tests import shared_oracle as so
from tests.test_gpu_cache_ops import FULL, MANY, ODD, THREE, TINY, WIDE, _m, make_q

pytestmark = pytest.mark.gpu
LAYOUTS = dict(full=FULL, wide=WIDE, tiny=TINY, odd=ODD, three=THREE, many=MANY)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def make_shared(spec, prefixes, of, own, seed, std=1.0, scale=None):
    """Random records behind random pages: the requests' tables are those of their whole contexts (a
    prefix's last page, where it is not full, is copied for each).  What no token occupies holds NaN
    codes and NaN scales."""
    rng = np.random.default_rng(seed)
    bs, rec, kv = spec["block_size"], spec["kv_record_bytes"], spec["kv_dim"]
    pages = [max(1, -(-p // bs)) for p in prefixes]
    start = [prefixes[g] if g >= 0 else 0 for g in of]
    end = [max(1, -(-(s + n) // bs)) for s, n in zip(start, own)]
    nb = sum(pages) + sum(e - s // bs for s, e in zip(start, end)) + 2
    perm = rng.permutation(nb)
    ptable = np.full((len(prefixes), max(pages)), -1, np.int32)
    table = np.full((len(of), max(end)), -1, np.int32)
    cache = np.full((nb, bs, rec), 0x7F, np.uint8)
    used = 0

    def fill(page, slots):
        if not len(slots):
            return
        v = torch.from_numpy((rng.standard_normal((len(slots), kv)) * std).astype(np.float32))
        sc = v.abs().amax(-1, keepdim=True) / 448.0
        cache[page, slots, :kv] = (v / sc).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        scb = sc.numpy() if scale is None else np.full((len(slots), 1), scale, np.float32)
        cache[page, slots, kv:kv + 4] = scb.astype(np.float32).view(np.uint8).reshape(-1, 4)

    for g, n in enumerate(pages):
        ptable[g, :n] = perm[used:used + n]
        used += n
        for i in range(n):
            fill(ptable[g, i], np.arange(min(bs, prefixes[g] - i * bs)))
    for b, (s, e) in enumerate(zip(start, end)):
        f = s // bs
        if f:
            table[b, :f] = ptable[of[b], :f]
        table[b, f:e] = perm[used:used + e - f]
        used += e - f
        for i in range(f, e):
            fill(table[b, i], np.arange(max(0, s - i * bs), min(bs, s + own[b] - i * bs)))
            if i == f and s % bs:  # the copy of the prefix's last tokens
                cache[table[b, i], :s % bs] = cache[ptable[of[b], f], :s % bs]
    return ptable, table, cache


def run(m, spec, q, positions, row_req, table, cache, ptable, lengths, of, handle=None, **kw):
    h = handle or m.Cache(spec, max_rows=len(positions), max_requests=table.shape[0])
    o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], spec["n_q_heads"]), float("nan"), device="cuda")
    cd = cache if isinstance(cache, torch.Tensor) else torch.from_numpy(cache).cuda()
    h.attend_shared(q.cuda(), o, i32(positions), i32(row_req), i32(table), cd, i32(ptable), i32(lengths),
                    prefix_of=None if of is None else i32(of), lse=lse, **kw)
    torch.cuda.synchronize()
    st = h.status(clear=True)
    if handle is None:
        h.close()
    return o.double().cpu().numpy(), lse.double().cpu().numpy(), st


def compare(got, want):
    (o, lse, _), (eo, tol, el, ltol) = got, want
    nan = np.isnan(eo)
    assert np.array_equal(np.isnan(o), nan)
    assert (np.abs(o - eo) <= tol)[~nan].all(), np.nanmax(np.abs(o - eo) - tol)
    inf = np.isinf(el)
    assert np.array_equal(lse[inf], el[inf])
    ln = np.isnan(el)
    assert np.array_equal(np.isnan(lse), ln)
    ok = ~inf & ~ln
    assert (np.abs(lse - el) <= ltol)[ok].all(), np.max((np.abs(lse - el) - ltol)[ok])


def rows_of(prefixes, of, own, rows_per):
    """Request b's rows are the last rows_per[b] of its tokens."""
    pos, req = [], []
    for b, (g, n, k) in enumerate(zip(of, own, rows_per)):
        L = (prefixes[g] if g >= 0 else 0) + n
        pos += list(range(max(0, L - k), L))
        req += [b] * (L - max(0, L - k))
    return pos, req


def check(spec, prefixes, of, own, rows_per, seed=0, causal=True, scale=None, pads=(), shuffle=False, q=None,
          status=0, edit=None, handle=None, **kw):
    m = _m()
    ptable, table, cache = make_shared(spec, prefixes, of, own, seed, **kw)
    pos, req = rows_of(prefixes, of, own, rows_per)
    for at in pads:
        pos.insert(at, -1)
        req.insert(at, 0)
    if shuffle:
        order = np.random.default_rng(seed + 1).permutation(len(pos))
        pos, req = [pos[i] for i in order], [req[i] for i in order]
    q = make_q(spec, len(pos), seed) if q is None else q(len(pos))
    if edit is not None:
        edit(cache, ptable, table)
    got = run(m, spec, q, pos, req, table, cache, ptable, prefixes, of, causal=causal, scale=scale, handle=handle)
    assert got[2] == status
    compare(got, so.attend(spec, q.double().numpy(), pos, req, table, cache, ptable, prefixes, of, causal, scale))


@pytest.mark.parametrize("P", [1, 2, 31, 127, 128, 129, 256, 1000])
def test_one_request(P):
    check(FULL, [P], [0], [1], [1], seed=P)
    check(FULL, [P], [0], [130], [3], seed=P)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("causal", [True, False])
def test_layouts(layout, causal):
    check(LAYOUTS[layout], [517], [0, 0, 0, 0], [130, 1, 64, 6], [3, 1, 6, 2], seed=7, causal=causal)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_several_prefixes_and_requests_without_one(layout):
    check(LAYOUTS[layout], [300, 1, 64, 129], [1, 0, -1, 3, 0, -1, 1], [5, 40, 200, 1, 3, 2, 129],
          [5, 2, 6, 1, 3, 1, 4], seed=9, pads=(0, 8), shuffle=True)


@pytest.mark.parametrize("n", [7, 8, 9, 15, 16, 17, 24, 33, 48])
def test_blocks_and_pairs_of_rows(n):
    """16 heads a slice: 8 rows a block; two blocks a pair, an odd one alone."""
    check(FULL, [700], [0] * n, [1 + i % 5 for i in range(n)], [1] * n, seed=n)
    check(FULL, [300], [0], [50], [n], seed=n)


@pytest.mark.parametrize("n", [1, 2, 126, 127, 255, 256, 300])
def test_many_requests_of_few_heads(n):
    check(TINY, [200], [0] * n, [1 + (7 * i) % 90 for i in range(n)], [1] * n, seed=n)
    check(dict(TINY, n_q_heads=1), [77], [0] * n, [1 + i % 3 for i in range(n)], [1] * n, seed=n)


def test_the_largest_step():
    check(dict(WIDE, n_q_heads=4), [150, 40], [i % 3 - 1 for i in range(512)], [2 + i % 9 for i in range(512)],
          [2] * 512, seed=5, shuffle=True)


def test_long_prefix():
    check(FULL, [9000], [0] * 8, [1, 40, 77, 128, 129, 250, 3, 9], [1, 2, 3, 1, 1, 2, 3, 1], seed=11)
    check(WIDE, [20011], [0] * 3, [1, 40, 77], [1, 2, 3], seed=11)


def test_many_steps_of_two_blocks():
    """Some ten tiles a CTA and item: the rings go round."""
    check(dict(TINY, n_q_heads=4), [12000], [0] * 16, [64 + i for i in range(16)], [64] * 16, seed=12)


@pytest.mark.parametrize("layout,P", [("wide", 1500), ("tiny", 3000), ("odd", 1700), ("three", 900)])
def test_many_steps_of_single_blocks(layout, P):
    """Many prefixes with two rows each: two slices at once, or every other tile."""
    n = 128 if layout in ("wide", "tiny") else 60
    check(LAYOUTS[layout], [P - 3 * i for i in range(n)], list(range(n)), [2 + i % 3 for i in range(n)], [2] * n, seed=13)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("P", [14 * 128 + 1, 15 * 128 + 1, 16 * 128 - 1, 17 * 128 + 5])
def test_lone_blocks_of_long_groups(layout, P):
    """About as many tiles as decide how a lone block's slices are taken, of a prefix and of own tokens,
    alone and behind a pair of blocks."""
    spec = LAYOUTS[layout]
    per = 128 // (spec["n_q_heads"] * spec["head_dim"] // spec["kv_dim"])  # rows a block
    check(spec, [P], [0, -1], [3, P], [1, 1], seed=P)
    if per <= 32:
        check(spec, [P], [0], [2 * per + 40], [2 * per + 1], seed=P + 1)


def test_without_any_prefix_and_with_empty_ones():
    check(WIDE, [64], [-1, -1], [300, 20], [3, 2], seed=3)
    check(WIDE, [0, 64], [0, 1], [300, 20], [3, 2], seed=4)
    check(WIDE, [0], [0, 0], [1, 140], [1, 6], seed=4)


def test_rows_inside_their_prefix():
    """A prompt that is still a prefix in part: such rows see that much of it, and nothing of their own."""
    m = _m()
    for causal in (True, False):
        ptable, table, cache = make_shared(WIDE, [400], [0, 0, 0], [10, 1, 1], 6)
        pos, req = [0, 127, 128, 300, 405, 17, 399, 400, 400], [0, 0, 0, 0, 0, 1, 1, 1, 2]
        q = make_q(WIDE, len(pos), 6)
        got = run(m, WIDE, q, pos, req, table, cache, ptable, [400], [0, 0, 0], causal=causal)
        assert got[2] == 0
        compare(got, so.attend(WIDE, q.double().numpy(), pos, req, table, cache, ptable, [400], [0, 0, 0], causal))


def test_pad_rows_alone_and_prefix_of_none():
    m = _m()
    ptable, table, cache = make_shared(TINY, [100], [0, 0], [20, 30], 8)
    q = make_q(TINY, 3, 8)
    o, lse, st = run(m, TINY, q, [-1, -5, -1], [0, 1, 0], table, cache, ptable, [100], None)
    assert st == 0 and not o.any() and np.isneginf(lse).all()
    got = run(m, TINY, q, [119, 129, 128], [0, 1, 1], table, cache, ptable, [100], None)
    assert got[2] == 0
    compare(got, so.attend(TINY, q.double().numpy(), [119, 129, 128], [0, 1, 1], table, cache, ptable, [100], None))


@pytest.mark.parametrize("std,qstd", [(8.0, 4.0), (1e-3, 1.0), (1.0, 1e-6), (1.0, 3e4), (1e4, 1e-5), (1e-20, 1e10)])
def test_sharp_flat_and_scaled_scores(std, qstd):
    check(WIDE, [300], [0, 0], [77, 130], [3, 4], seed=2, std=std, q=lambda n: make_q(WIDE, n, 2, std=qstd))
    check(ODD, [300], [0, 0], [77, 130], [3, 4], seed=2, std=std, q=lambda n: make_q(ODD, n, 2, std=qstd))


@pytest.mark.parametrize("layout", ["full", "tiny"])
def test_scores_that_rise_along_the_context(layout):
    """Every tile's largest weight passes the one before by far: the reference moves again and again."""
    spec = LAYOUTS[layout]
    kv = spec["kv_dim"]

    def rising(cache, ptable, table):
        bs = spec["block_size"]
        cache[..., :kv] = 0x38  # 1.0
        for tab in (ptable, table):
            for b in range(tab.shape[0]):
                for t in range(tab.shape[1] * bs):
                    if 0 <= tab[b, t // bs]:
                        cache[tab[b, t // bs], t % bs, kv:kv + 4] = np.frombuffer(
                            np.float32(t / 16).tobytes(), np.uint8)

    def q(n):
        return torch.full((n, spec["n_q_heads"] * spec["head_dim"]), 0.25).to(torch.bfloat16)

    check(spec, [1200], [0, 0], [300, 20], [2, 3], seed=1, edit=rising, q=q)


def test_zero_and_negative_and_mixed_scales():
    def mixed(cache, ptable, table):
        rng = np.random.default_rng(3)
        kv = WIDE["kv_dim"]
        old = np.ascontiguousarray(cache[..., kv:kv + 4]).view(np.float32)[..., 0]
        f = rng.choice([0.0, -1.0, 1.0, 2.0 ** -30, 2.0 ** 4, -2.0 ** 3, 2.0 ** -126], old.shape)
        new = np.where(np.isnan(old), old, old * f).astype(np.float32)
        cache[..., kv:kv + 4] = new[..., None].view(np.uint8)

    check(WIDE, [300], [0, 0], [77, 130], [3, 4], seed=2, edit=mixed)
    check(WIDE, [300], [0, 0], [77, 130], [3, 4], seed=2, scale=0.01, edit=mixed)


def test_records_that_are_all_zeros():
    """Their keys and values are 0: every weight alike, o 0."""
    def zeros(cache, ptable, table):
        cache[:] = 0

    check(WIDE, [300], [0, 0], [77, 130], [3, 4], seed=2, edit=zeros)


@pytest.mark.parametrize("scale", [2.0 ** -20, 2.0 ** 20])
def test_the_least_and_the_largest_scale(scale):
    """With queries that make the scores ordinary ones."""
    def q(n):
        return (make_q(FULL, n, 3).float() * (2.0 ** -4 / scale)).to(torch.bfloat16)
    check(FULL, [260], [0, 0], [70, 5], [2, 3], seed=8, scale=scale, q=q)


@pytest.mark.parametrize("n", [1, 13, 26, 52, 104])
def test_pieces_joined_by_teams_of_every_size(n):
    """Rows of 64 heads behind a prefix that the whole GPU shares: 8, 4, 2 and 1 warps a query."""
    check(FULL, [9000], [0] * n, [1] * n, [1] * n, seed=n)


def test_nan_codes_and_scales_reach_only_rows_and_heads_that_see_them():
    m = _m()
    kv = WIDE["kv_dim"]
    for what in ("code", "scale", "huge", "inf"):
        for causal in (True, False):
            ptable, table, cache = make_shared(WIDE, [200], [0, 0], [20, 30], 5)
            pos, req = [215, 216, 217, 218, 219, 229], [0] * 5 + [1]
            rec = cache[table[0, 217 // 64], 217 % 64]
            if what == "code":
                rec[70] = 0x7F  # of the second slice
            else:
                rec[kv:kv + 4] = np.frombuffer(np.float32(
                    dict(scale=np.nan, huge=2.0 ** 65, inf=np.inf)[what]).tobytes(), np.uint8)
            q = make_q(WIDE, len(pos), 5)
            o, lse, st = run(m, WIDE, q, pos, req, table, cache, ptable, [200], [0, 0], causal=causal)
            assert st == 0
            sees = np.array([(p >= 217 or not causal) and b == 0 for p, b in zip(pos, req)])
            heads = np.zeros(16, bool)
            heads[8 if what == "code" else 0:] = True
            bad = sees[:, None] & heads[None]
            assert np.array_equal(np.isnan(lse), bad)
            assert np.array_equal(np.isnan(o.reshape(6, 16, 64)).all(-1), bad)
            eo, tol, el, ltol = so.attend(WIDE, q.double().numpy(), pos, req, table, cache, ptable, [200], [0, 0],
                                          causal)
            ok = ~np.repeat(bad, 64, 1).reshape(6, -1)
            assert (np.abs(o - eo) <= tol)[ok].all() and (np.abs(lse - el) <= ltol)[~bad].all()


def test_nan_codes_in_a_prefix():
    """In a tile that every row sees whole, and in one that not every row does."""
    m = _m()
    for at, last in ((5, 290), (290, 280)):
        ptable, table, cache = make_shared(WIDE, [300], [0, 0], [20, 30], 5)
        cache[ptable[0, at // 64], at % 64, 3] = 0xFF  # of the first slice
        pos, req = [last, 319, 329], [0, 0, 1]
        q = make_q(WIDE, 3, 5)
        o, lse, st = run(m, WIDE, q, pos, req, table, cache, ptable, [300], [0, 0])
        bad = np.zeros((3, 16), bool)
        bad[:, :8] = np.array([p >= at for p in pos])[:, None]
        assert st == 0 and np.array_equal(np.isnan(lse), bad)
        eo, tol, el, ltol = so.attend(WIDE, q.double().numpy(), pos, req, table, cache, ptable, [300], [0, 0])
        ok = ~np.repeat(bad, 64, 1).reshape(3, -1)
        assert (np.abs(o - eo) <= tol)[ok].all() and (np.abs(lse - el) <= ltol)[~bad].all()


def test_queries_that_are_not_finite_are_their_own_heads_business():
    m = _m()
    ptable, table, cache = make_shared(ODD, [100], [0], [20], 5)
    q = make_q(ODD, 4, 5)
    q[1, 5] = float("nan")           # row 1, head 0
    q[2, 2 * 128 + 7] = float("inf")  # row 2, head 2
    q[3, 128:256] = 0.0               # row 3, head 1: every weight alike
    q[3, 300] = -float("inf")         # and head 2
    pos = [116, 117, 118, 119]
    o, lse, st = run(m, ODD, q, pos, [0] * 4, table, cache, ptable, [100], [0])
    bad = np.zeros((4, 6), bool)
    bad[1, 0] = bad[2, 2] = bad[3, 2] = True
    assert st == 0 and np.array_equal(np.isnan(lse), bad)
    assert np.array_equal(np.isnan(o.reshape(4, 6, 128)).all(-1), bad)
    qz = torch.where(torch.isfinite(q), q, torch.zeros_like(q))
    eo, tol, el, ltol = so.attend(ODD, qz.double().numpy(), pos, [0] * 4, table, cache, ptable, [100], [0])
    ok = ~np.repeat(bad, 128, 1).reshape(4, -1)
    assert (np.abs(o - eo) <= tol)[ok].all() and (np.abs(lse - el) <= ltol)[~bad].all()


def test_unmapped_pages_bad_requests_and_bad_prefixes():
    m = _m()
    of = [0, 1, 0, -2, 2, -1]
    ptable, table, cache = make_shared(WIDE, [200, 130], [0, 1, 0, 0, 0, -1], [20, 30, 5, 5, 5, 9], 5)
    q = make_q(WIDE, 8, 5)
    pos, req = [219, 150, 204, 203, 203, 8, 9, 4], [0, 1, 2, 3, 4, 5, 6, -1]
    lengths = [200, 130]
    table[0, 3] = 99       # beyond the cache: of request 0's own tokens
    ptable[1, 1] = -7      # the second prefix's second page
    for case in range(3):
        if case == 1:
            lengths = [200, 1000]  # beyond the prefix table, and all that request 1 sees
        if case == 2:
            lengths, pos = [-3, 130], [219, 2 ** 31 - 1, 204, 203, 203, 8, 9, 4]
            of = [0, 1, 0, 7, -9, -1]
        got = run(m, WIDE, q, pos, req, table, cache, ptable, lengths, of)
        assert got[2] == m.STATUS_UNMAPPED_PAGE
        seen = [min(p, 4095) for p in pos]  # (the reference's loop; behind the tables there is nothing)
        compare(got, so.attend(WIDE, q.double().numpy(), seen, req, table, cache, ptable, lengths, of))


def test_strided_queries_results_and_caches():
    m = _m()
    ptable, table, cache = make_shared(WIDE, [200], [0, 0], [20, 30], 5)
    q = make_q(WIDE, 5, 5)
    big = torch.zeros((5, 1400), dtype=torch.bfloat16, device="cuda")
    big[:, 40:1064] = q.cuda()
    out = torch.full((5, 1104), 3.0, dtype=torch.bfloat16, device="cuda")
    pool = torch.full((cache.shape[0], 70, 176), 0x7F, dtype=torch.uint8, device="cuda")
    pool[:, 3:67, 16:160] = torch.from_numpy(cache).cuda()
    pos, req = [218, 219, 227, 228, 229], [0, 0, 1, 1, 1]
    h = m.Cache(WIDE, 5, 2)
    h.attend_shared(big[:, 40:1064], out[:, 16:1040], i32(pos), i32(req), i32(table), pool[:, 3:67, 16:160], i32(ptable),
                    i32([200]))
    torch.cuda.synchronize()
    assert h.status() == 0
    eo, tol, _, _ = so.attend(WIDE, q.double().numpy(), pos, req, table, cache, ptable, [200], [0, 0])
    assert (np.abs(out[:, 16:1040].double().cpu().numpy() - eo) <= tol).all()
    assert (out[:, :16] == 3).all() and (out[:, 1040:] == 3).all()
    h.close()


def test_the_same_as_the_attention_of_whole_contexts():
    """The tables are those of whole contexts: both operators' bounds together."""
    m = _m()
    of, own, per = [0] * 6, [10, 300, 77, 1, 129, 64], [6, 1, 3, 1, 6, 2]
    ptable, table, cache = make_shared(FULL, [1000], of, own, 21)
    pos, req = rows_of([1000], of, own, per)
    q = make_q(FULL, len(pos), 21)
    o, lse, st = run(m, FULL, q, pos, req, table, cache, ptable, [1000], of)
    h = m.Cache(FULL, len(pos), 6)
    o2, lse2 = torch.zeros_like(q).cuda(), torch.zeros((len(pos), 64), device="cuda")
    h.attend(q.cuda(), o2, i32(pos), i32(req), i32(table), torch.from_numpy(cache).cuda(), lse=lse2)
    torch.cuda.synchronize()
    assert st == 0 and h.status() == 0
    h.close()
    from tests import cache_oracle as co
    _, tol2, _, ltol2, _, _ = co.attend(FULL, q.double().numpy(), pos, req, table, cache)
    _, tol, _, ltol = so.attend(FULL, q.double().numpy(), pos, req, table, cache, ptable, [1000], of)
    assert (np.abs(o - o2.double().cpu().numpy()) <= tol + tol2).all()
    assert (np.abs(lse - lse2.double().cpu().numpy()) <= ltol + ltol2).all()


def test_captured_on_other_streams_and_two_handles_at_once():
    m = _m()
    sets = []
    for seed in (1, 2):
        of, own = [0, 0, -1], [30, 200, 150]
        ptable, table, cache = make_shared(FULL, [1500], of, own, seed)
        pos, req = rows_of([1500], of, own, [6, 6, 6])
        q = make_q(FULL, len(pos), seed)
        want = so.attend(FULL, q.double().numpy(), pos, req, table, cache, ptable, [1500], of)
        d = dict(h=m.Cache(FULL, 18, 3), q=q.cuda(), o=torch.zeros_like(q).cuda(), lse=torch.zeros((18, 64), device="cuda"),
                 args=(i32(pos), i32(req), i32(table), torch.from_numpy(cache).cuda(), i32(ptable), i32([1500])),
                 of=i32(of), want=want, stream=torch.cuda.Stream())
        d["call"] = lambda d=d, **kw: d["h"].attend_shared(d["q"], d["o"], *d["args"], prefix_of=d["of"], lse=d["lse"], **kw)
        sets.append(d)
    torch.cuda.synchronize()
    for _ in range(5):
        for d in sets:
            d["call"](stream=d["stream"])
    torch.cuda.synchronize()
    eager = []
    for d in sets:
        assert d["h"].status() == 0
        compare((d["o"].double().cpu().numpy(), d["lse"].double().cpu().numpy(), 0), d["want"])
        eager.append((d["o"].clone(), d["lse"].clone()))
        d["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(d["graph"], stream=d["stream"]):
            d["call"]()
    for _ in range(20):
        for d, e in zip(sets, eager):
            d["o"].zero_(), d["lse"].zero_()
            d["graph"].replay()
            torch.cuda.synchronize()
            # the cut, and so every sum, is that of the step alone
            assert torch.equal(d["o"], e[0]) and torch.equal(d["lse"], e[1])
    # another step in the same graph: rows move on, one becomes a pad row
    d = sets[0]
    d["args"][0][17] = -1
    d["graph"].replay()
    torch.cuda.synchronize()
    assert not d["o"][17].any() and torch.isneginf(d["lse"][17]).all()
    for d in sets:
        assert d["h"].status() == 0
        d["h"].close()


def test_append_attend_and_rotate_back_together():
    """Two decode steps of requests behind one prefix, with rotary positions: latents appended and
    queries rotated, attention over the shared prefix, the output turned back.  Against the same in
    64 bits from the stored records; the rotated queries are the bf16 values that were attended."""
    m = _m()
    spec, P, of, own = WIDE, 150, [0, 0, 0], [1, 60, 127]
    dh, kv, width, dim = 64, 128, 1024, 32
    rng = np.random.default_rng(4)
    tab = ro.table(600, dim)
    ptable, table, cache = make_shared(spec, [P], of, [n + 4 for n in own], 4)
    for b, n in enumerate(own):  # the tokens to come are not there yet
        for t in range(P + n, P + n + 4):
            cache[table[b, t // 64], t % 64] = 0x7F
    h = m.Cache(spec, 6, 3)
    pool, rope = torch.from_numpy(cache).cuda(), torch.from_numpy(tab).cuda()
    o, back = torch.zeros((6, width), dtype=torch.bfloat16, device="cuda"), torch.zeros((6, width), dtype=torch.bfloat16, device="cuda")
    for step in range(2):
        pos = [P + n + 2 * step + j for n in own for j in range(2)]
        req = [0, 0, 1, 1, 2, 2]
        x = torch.from_numpy(rng.standard_normal((6, kv)).astype(np.float32)).to(torch.bfloat16)
        q = torch.from_numpy(rng.standard_normal((6, width)).astype(np.float32)).to(torch.bfloat16)
        qd = q.cuda()
        h.append(x.cuda(), i32(pos), i32(req), i32(table), pool, rope=rope, q=qd)
        h.attend_shared(qd, o, i32(pos), i32(req), i32(table), pool, i32(ptable), i32([P]), prefix_of=i32(of))
        h.rotate(o, back, i32(pos), rope, inverse=True)
        torch.cuda.synchronize()
        assert h.status() == 0
        stored = pool.cpu().numpy()
        y = ro.rotate(x.double().numpy(), tab, pos, dh, dh - dim, False)
        for r, p in enumerate(pos):  # a code is off by half a step: 2^-4 relative, 2^-10 of the scale
            rec = stored[table[req[r], p // 64], p % 64]
            s = float(np.frombuffer(rec[kv:kv + 4].tobytes(), np.float32)[0])
            assert (np.abs(so.E4M3[rec[:kv]] * s - y[r]) <= (2.0 ** -4 * np.abs(y[r]) + 2.0 ** -10 * s) * (1 + 2.0 ** -10)).all()
        qr = ro.rotate(q.double().numpy(), tab, pos, dh, dh - dim, False)
        assert (np.abs(qd.double().cpu().numpy() - qr) <= 2.0 ** -8 * np.abs(qr) + 2.0 ** -20).all()
        eo, tol, _, _ = so.attend(spec, qd.double().cpu().numpy(), pos, req, table, stored, ptable, [P], of)
        eb = ro.rotate(eo, tab, pos, dh, dh - dim, False, inverse=True)
        # a turn moves at most the sum of a pair's errors, and is rounded to bf16
        one, two = ro.pairs(dim, dh - dim, False)
        t2 = tol.reshape(6, -1, dh).copy()
        t2[..., one] = t2[..., two] = t2[..., one] + t2[..., two]
        t2 = t2.reshape(6, -1) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(eb) + 2.0 ** -20
        assert (np.abs(back.double().cpu().numpy() - eb) <= t2).all()
    h.close()


def test_the_library_refuses():
    """Decided on the host: the addresses are never used."""
    import ctypes as C
    m = _m()
    from moe_decode_layer_mxfp8_gb300 import cache as mc
    h = m.Cache(WIDE, 8, 4)
    a = 0x10000
    good = dict(q=a, o=a, positions=a, row_req=a, block_table=a, prefix_table=a, prefix_lengths=a, max_blocks=5, n_req=2,
                prefix_max_blocks=3, n_prefix=1, rows=3, causal=1, kv_cache=a, kv_stride_block=64 * 144,
                kv_stride_tok=144, kv_num_blocks=4)
    for change, code in [
            (dict(q=None), -1), (dict(o=None), -1), (dict(positions=None), -1), (dict(row_req=None), -1),
            (dict(block_table=None), -1), (dict(prefix_table=None), -1), (dict(prefix_lengths=None), -1),
            (dict(kv_cache=None), -1), (dict(rows=0), -1), (dict(rows=9), -3), (dict(n_req=0), -1), (dict(n_req=5), -3),
            (dict(n_prefix=0), -1), (dict(n_prefix=129), -3), (dict(q=a + 8), -4), (dict(o=a + 2), -4),
            (dict(q_stride=1023), -1), (dict(o_stride=1028), -4), (dict(positions=a + 2), -4), (dict(lse=a + 2), -4),
            (dict(prefix_of=a + 1), -4), (dict(prefix_lengths=a + 2), -4), (dict(scale=-1.0), -1),
            (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(scale=2.0 ** 21), -1),
            (dict(scale=2.0 ** -21), -1), (dict(max_blocks=0), -1),
            (dict(prefix_max_blocks=0), -1), (dict(max_blocks=2 ** 26), -1), (dict(prefix_max_blocks=2 ** 26), -1),
            (dict(kv_stride_tok=128), -5), (dict(kv_num_blocks=0), -1)]:
        args = mc.SharedArgs(**dict(good, **change))
        assert mc._lib().mono_cache_attend_shared(h._h, C.byref(args), None) == code, change
    h.close()
    # work that 32 bits do not count: 2 rows' blocks x 2 slices x 2^23 tiles
    h = m.Cache(WIDE, 1024, 4)
    args = mc.SharedArgs(**dict(good, rows=1024, max_blocks=2 ** 24))
    assert mc._lib().mono_cache_attend_shared(h._h, C.byref(args), None) == -1
    torch.cuda.synchronize()
    assert h.status() == 0
    h.close()
