"""The cache operators on the GPU against 64-bit references (tests/cache_oracle.py): at the
lengths, masks, layouts and page sizes where they can go wrong, captured, on other streams, and
run together on a layer's own cache.  Whole numbers have to be equal; the bounds of the
attention's results are derived with the reference."""
import numpy as np
import pytest
import torch

from tests import cache_oracle as co

pytestmark = pytest.mark.gpu

FULL = dict(n_q_heads=64, head_dim=128, kv_dim=512, block_size=128, kv_record_bytes=528)
WIDE = dict(n_q_heads=16, head_dim=64, kv_dim=128, block_size=64, kv_record_bytes=144)
TINY = dict(n_q_heads=4, head_dim=64, kv_dim=64, block_size=16, kv_record_bytes=80)
ODD = dict(n_q_heads=6, head_dim=128, kv_dim=128, block_size=7, kv_record_bytes=160)
THREE = dict(n_q_heads=9, head_dim=64, kv_dim=192, block_size=24, kv_record_bytes=208)
MANY = dict(n_q_heads=32, head_dim=64, kv_dim=128, block_size=1, kv_record_bytes=144)


def _m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import moe_decode_layer_mxfp8_gb300 as m
    from moe_decode_layer_mxfp8_gb300 import build
    build.build()
    return m


def make_cache(spec, lengths, seed, poison=True, std=1.0):
    """Random records behind random pages.  Everything that no request's tokens occupy (page
    tails, spare pages, record padding) holds NaN codes and NaN scales."""
    rng = np.random.default_rng(seed)
    bs, rec, kv = spec["block_size"], spec["kv_record_bytes"], spec["kv_dim"]
    per = [max(1, -(-n // bs)) for n in lengths]
    nb = sum(per) + 2
    perm = rng.permutation(nb)
    table = np.full((len(per), max(per)), -1, np.int32)
    cache = np.full((nb, bs, rec), 0x7F if poison else 0, np.uint8)
    o = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[o:o + n]
        o += n
        L = lengths[b]
        v = torch.from_numpy((rng.standard_normal((L, kv)) * std).astype(np.float32))
        sc = (v.abs().amax(-1, keepdim=True) / 448.0 if L else v[:, :1])
        codes = (v / sc).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        scb = sc.numpy().astype(np.float32).view(np.uint8).reshape(L, 4)
        for t in range(L):
            cache[table[b, t // bs], t % bs, :kv] = codes[t]
            cache[table[b, t // bs], t % bs, kv:kv + 4] = scb[t]
    return table, cache


def make_q(spec, rows, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, spec["n_q_heads"] * spec["head_dim"]), generator=g) * std).to(
        torch.bfloat16)


def run_attend(m, spec, q, positions, row_req, table, cache, weights=None, handle=None, **kw):
    dev = torch.device("cuda")
    h = handle or m.Cache(spec, max_rows=len(positions), max_requests=table.shape[0])
    qd = q.to(dev)
    o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
    lse = torch.full((q.shape[0], spec["n_q_heads"]), float("nan"), device=dev)
    w = None if weights is None else weights.to(dev)
    cd = cache if isinstance(cache, torch.Tensor) else torch.from_numpy(cache).to(dev)
    h.attend(qd, o, torch.tensor(positions, dtype=torch.int32, device=dev),
             torch.tensor(row_req, dtype=torch.int32, device=dev),
             torch.from_numpy(table).to(dev), cd, lse=lse, weights=w, **kw)
    torch.cuda.synchronize()
    st = h.status()
    if handle is None:
        h.close()
    return o.double().cpu().numpy(), lse.double().cpu().numpy(), \
        None if w is None else w.double().cpu().numpy(), st


def check_attend(m, spec, lengths, rows_per, seed, window=0, sinks=0, causal=True, pads=(),
                 shuffle=False, scale=None, n_weights=None, **cache_kw):
    """Request b's rows are the last rows_per[b] of its lengths[b] tokens."""
    table, cache = make_cache(spec, lengths, seed, **cache_kw)
    positions, row_req = [], []
    for b, (L, n) in enumerate(zip(lengths, rows_per)):
        positions += list(range(L - n, L))
        row_req += [b] * n
    for at in pads:
        positions.insert(at, -1)
        row_req.insert(at, 0)
    if shuffle:
        order = np.random.default_rng(seed + 1).permutation(len(positions))
        positions = [positions[i] for i in order]
        row_req = [row_req[i] for i in order]
    q = make_q(spec, len(positions), seed)
    cap = max(lengths) if n_weights is None else n_weights
    w0 = torch.rand((len(lengths), cap), generator=torch.Generator().manual_seed(seed))
    o, lse, w, st = run_attend(m, spec, q, positions, row_req, table, cache, weights=w0,
                               window=window, sinks=sinks, causal=causal, scale=scale)
    assert st == 0
    eo, tol, el, ltol, ew, wtol = co.attend(spec, q.double().numpy(), positions, row_req, table,
                                            cache, window, sinks, causal, scale, cap)
    assert not np.isnan(o).any() and (np.abs(o - eo) <= tol).all(), np.max(np.abs(o - eo) - tol)
    inf = np.isinf(el)
    assert np.array_equal(lse[inf], el[inf])
    assert (np.abs(lse - el)[~inf] <= ltol[~inf]).all()
    start = w0.double().numpy()
    # the sum of the old weight and up to rows x heads new ones, in f32
    rnd = 2.0 ** -24 * (np.abs(start) + (len(positions) * spec["n_q_heads"] + 2) * ew)
    assert (np.abs(w - start - ew) <= wtol + rnd).all(), np.max(np.abs(w - start - ew) - wtol - rnd)


@pytest.mark.parametrize("L", [1, 2, 31, 127, 128, 129, 256, 1000])
def test_attend_one_row(L):
    check_attend(_m(), FULL, [L], [1], seed=L)


@pytest.mark.parametrize("spec", [WIDE, TINY, ODD, THREE, MANY], ids=["wide", "tiny", "odd",
                                                                     "three", "many"])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_layouts(spec, causal):
    check_attend(_m(), spec, [130, 1, 517, 64], [3, 1, 6, 2], seed=7, causal=causal)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (100, 0), (128, 4), (129, 1), (300, 200),
                                          (5000, 7), (1000, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_window_and_sinks(window, sinks, causal):
    check_attend(_m(), WIDE, [700, 90, 1301, 3], [6, 4, 5, 3], seed=window, window=window,
                 sinks=sinks, causal=causal)


def test_attend_full_layout_window():
    check_attend(_m(), FULL, [1200, 333], [6, 6], seed=3, window=500, sinks=4)


def test_attend_sinks_without_window_change_nothing():
    check_attend(_m(), WIDE, [300], [2], seed=4, window=0, sinks=9)


def test_attend_pad_rows_and_rows_in_any_order():
    check_attend(_m(), WIDE, [200, 40, 333], [5, 3, 4], seed=5, pads=(0, 4, 12), shuffle=True)


@pytest.mark.parametrize("n", [7, 16, 17, 48])
def test_attend_many_rows_of_one_request(n):
    check_attend(_m(), FULL, [300], [n], seed=n)
    check_attend(_m(), TINY, [300], [n], seed=n)


def test_attend_many_requests():
    lengths = [1 + (i * 37) % 400 for i in range(60)]
    check_attend(_m(), TINY, lengths, [min(2, n) for n in lengths], seed=6)


@pytest.mark.parametrize("spec,lengths,rows", [
    (FULL, [9000], [42]), (FULL, [6000, 200, 5000], [12, 6, 11]),
    (FULL, [4100 + 97 * i for i in range(12)], [1] * 12), (THREE, [20000, 9000], [16, 7]),
    (ODD, [15000, 15001], [13, 16])], ids=["groups", "mixed", "single", "three", "odd"])
def test_attend_many_tiles_per_block(spec, lengths, rows):
    """Every block goes round its rings of buffers several times, over several items."""
    check_attend(_m(), spec, lengths, rows, seed=lengths[0])


def test_attend_scale_and_short_weight_rows():
    check_attend(_m(), WIDE, [300, 20], [2, 2], seed=8, scale=0.31, n_weights=150)


def test_attend_sharp_scores():
    """Scores spread over hundreds: every weight but a few underflows."""
    check_attend(_m(), WIDE, [700], [3], seed=9, scale=4.0, std=2.0)


def test_attend_rows_between_tokens():
    """A row below its request's last cached token sees nothing beyond its own position, whatever
    the later records hold."""
    m = _m()
    table, cache = make_cache(WIDE, [400], 11)
    for t in range(250, 400):
        cache[table[0, t // 64], t % 64] = 0x7F  # NaN codes and scale
    q = make_q(WIDE, 2, 11)
    o, lse, _, st = run_attend(m, WIDE, q, [249, 100], [0, 0], table, cache)
    eo, tol, el, ltol, _, _ = co.attend(WIDE, q.double().numpy(), [249, 100], [0, 0], table, cache)
    assert st == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()


@pytest.mark.parametrize("bits", [0x7F, 0x00], ids=["nan", "inf"])
def test_attend_masked_values_do_not_reach_a_row(bits):
    """Draft rows: the last token's record is NaN codes (and an infinite or NaN scale); rows before
    it are exact, the row that sees it is NaN where codes are."""
    m = _m()
    table, cache = make_cache(FULL, [200], 12)
    pg, sl = table[0, 199 // 128], 199 % 128
    cache[pg, sl, :512] = bits or 0x38
    cache[pg, sl, 512:516] = np.frombuffer(np.float32(np.inf).tobytes(), np.uint8)
    pos, req = [197, 198, 199], [0, 0, 0]
    q = make_q(FULL, 3, 12)
    w0 = torch.zeros((1, 200))
    o, lse, w, st = run_attend(m, FULL, q, pos, req, table, cache, weights=w0)
    eo, tol, el, ltol, _, _ = co.attend(FULL, q.double().numpy()[:2], pos[:2], req[:2], table, cache)
    assert (np.abs(o[:2] - eo) <= tol).all() and (np.abs(lse[:2] - el) <= ltol).all()
    if bits:
        assert np.isnan(o[2]).all()


def test_attend_zero_scales_and_zero_codes():
    """A token of zeros scores 0 and still takes its share."""
    m = _m()
    table, cache = make_cache(WIDE, [300], 13)
    for t in (0, 17, 130, 299):
        cache[table[0, t // 64], t % 64, :128] = 0
    for t in (5, 131, 298):
        cache[table[0, t // 64], t % 64, 128:132] = 0
    q = make_q(WIDE, 1, 13)
    o, lse, _, st = run_attend(m, WIDE, q, [299], [0], table, cache)
    eo, tol, el, ltol, _, _ = co.attend(WIDE, q.double().numpy(), [299], [0], table, cache)
    assert st == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()


def test_attend_codes_below_the_normal_range():
    """Records of subnormal codes only: o keeps 8 bits of them (weights to 2^-8 each, o's rounding
    2^-8, and 2^-12 for the scores' and sums' roundings)."""
    m = _m()
    table, cache = make_cache(WIDE, [300], 21)
    rng = np.random.default_rng(21)
    for t in range(300):
        cache[table[0, t // 64], t % 64, :128] = rng.integers(1, 8, 128)
        cache[table[0, t // 64], t % 64, 128:132] = np.frombuffer(np.float32(0.37).tobytes(), np.uint8)
    q = make_q(WIDE, 2, 21)
    o, _, _, st = run_attend(m, WIDE, q, [150, 299], [0, 0], table, cache)
    eo, *_ = co.attend(WIDE, q.double().numpy(), [150, 299], [0, 0], table, cache)
    assert st == 0 and (np.abs(o - eo) <= (2.0 ** -7 + 2.0 ** -12) * np.abs(eo)).all()


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 30])
def test_attend_scales_far_from_one(scale):
    """Records of tiny and of huge values (the queries and the score factor make up for it)."""
    m = _m()
    table, cache = make_cache(WIDE, [200], 22)
    f = np.float32(scale)
    for t in range(200):
        r = cache[table[0, t // 64], t % 64]
        r[128:132] = np.frombuffer((r[128:132].copy().view(np.float32) * f).tobytes(), np.uint8)
    q = make_q(WIDE, 1, 22)
    k = 0.125 / scale
    o, lse, _, st = run_attend(m, WIDE, q, [199], [0], table, cache, scale=k)
    eo, tol, el, ltol, _, _ = co.attend(WIDE, q.double().numpy(), [199], [0], table, cache, scale=k)
    assert st == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()


@pytest.mark.parametrize("first", [True, False])
def test_attend_one_heavy_token_and_a_long_tail(first):
    """One token of weight 2^15 times the others' (an attention sink): the tail carries as much."""
    m = _m()
    L = 9000
    rng = np.random.default_rng(14)
    table, cache = make_cache(TINY, [L], 14, std=0.05)
    at = 0 if first else L - 1
    q = make_q(TINY, 1, 14)
    v = q.float().numpy().reshape(4, 64)[0] * 4
    sc = np.abs(v).max() / 448
    cache[table[0, at // 16], at % 16, :64] = torch.from_numpy(v / sc).to(
        torch.float8_e4m3fn).view(torch.uint8).numpy()
    cache[table[0, at // 16], at % 16, 64:68] = np.frombuffer(np.float32(sc).tobytes(), np.uint8)
    want = np.log(L / 2.0)
    scale = want / float((v * q.float().numpy().reshape(4, 64)[0]).sum())
    o, lse, _, st = run_attend(m, TINY, q, [L - 1], [0], table, cache, scale=scale)
    eo, tol, el, ltol, _, _ = co.attend(TINY, q.double().numpy(), [L - 1], [0], table, cache,
                                        scale=scale)
    assert st == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()
    del rng


def test_attend_unmapped_pages_are_left_out():
    m = _m()
    table, cache = make_cache(TINY, [300, 40], 15)
    table[0, 3] = -1
    table[0, 10] = cache.shape[0]
    q = make_q(TINY, 4, 15)
    pos, req = [299, 39, 30, 5], [0, 1, 2, -1]  # the last two: no such request
    o, lse, _, st = run_attend(m, TINY, q, pos, req, table, cache)
    eo, tol, el, ltol, _, _ = co.attend(TINY, q.double().numpy(), pos, req, table, cache)
    assert st == 1
    assert (np.abs(o - eo) <= tol).all() and not o[2:].any() and np.isneginf(lse[2:]).all()
    assert (np.abs(lse - el)[:2] <= ltol[:2]).all()
    # nothing visible at all: every page unmapped; a position beyond the table
    table[:] = -1
    o, lse, _, st = run_attend(m, TINY, q[:1], [40], [0], table, cache)
    assert st == 1 and not o.any() and np.isneginf(lse).all()


def test_attend_position_beyond_the_table():
    m = _m()
    table, cache = make_cache(TINY, [64], 16)
    q = make_q(TINY, 1, 16)
    o, lse, _, st = run_attend(m, TINY, q, [70], [0], table, cache)
    eo, tol, el, ltol, _, _ = co.attend(TINY, q.double().numpy(), [70], [0], table, cache)
    assert st == 1 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()


def test_attend_strided_rows_records_and_pages():
    m = _m()
    table, cache = make_cache(WIDE, [333], 17)
    dev = torch.device("cuda")
    big = torch.full((cache.shape[0], 64 + 3, 176), 0x7F, dtype=torch.uint8, device=dev)
    big[:, :64, :144] = torch.from_numpy(cache).to(dev)
    view = big[:, :64, :144]
    q = make_q(WIDE, 3, 17)
    W = q.shape[1]
    qd = torch.full((3, W + 24), float("nan"), dtype=torch.bfloat16, device=dev)
    od = torch.full((3, W + 8), 5.0, dtype=torch.bfloat16, device=dev)
    qd[:, :W] = q.to(dev)
    h = m.Cache(WIDE, 3, 1)
    pos = torch.tensor([330, 331, 332], dtype=torch.int32, device=dev)
    h.attend(qd[:, :W], od[:, :W], pos, torch.zeros_like(pos), torch.from_numpy(table).to(dev), view)
    torch.cuda.synchronize()
    eo, tol, _, _, _, _ = co.attend(WIDE, q.double().numpy(), [330, 331, 332], [0] * 3, table, cache)
    assert (np.abs(od[:, :W].double().cpu().numpy() - eo) <= tol).all()
    assert (od[:, W:] == 5.0).all()  # behind the rows: as it was
    h.close()


def test_attend_offsets_beyond_32_bits():
    """Pages more than 4 GiB apart."""
    m = _m()
    dev = torch.device("cuda")
    table, cache = make_cache(WIDE, [190], 18)
    far = 5 << 30
    pool = torch.zeros(far + 64 * 144 * 8, dtype=torch.uint8, device=dev)
    nb = cache.shape[0]
    stride = (far // (nb - 1)) // 16 * 16
    view = torch.as_strided(pool, (nb, 64, 144), (stride, 144, 1))
    view.copy_(torch.from_numpy(cache).to(dev))
    q = make_q(WIDE, 1, 18)
    o, _, _, st = run_attend(m, WIDE, q, [189], [0], table, view)
    eo, tol, _, _, _, _ = co.attend(WIDE, q.double().numpy(), [189], [0], table, cache)
    assert st == 0 and (np.abs(o - eo) <= tol).all()


def test_attend_same_bits_every_time_on_streams_and_in_a_graph():
    m = _m()
    dev = torch.device("cuda")
    lengths = [3000, 129, 1700]
    table, cache = make_cache(WIDE, lengths, 19)
    pos = [L - 1 - i for L in lengths for i in range(3)]
    req = [b for b in range(3) for _ in range(3)]
    q = make_q(WIDE, 9, 19).to(dev)
    args = (torch.tensor(pos, dtype=torch.int32, device=dev),
            torch.tensor(req, dtype=torch.int32, device=dev), torch.from_numpy(table).to(dev),
            torch.from_numpy(cache).to(dev))
    h, h2 = m.Cache(WIDE, 9, 3), m.Cache(WIDE, 9, 3)

    def outs():
        return (torch.empty_like(q), torch.empty((9, 16), device=dev),
                torch.zeros((3, 3000), device=dev))

    def call(h, out, stream=None):
        h.attend(q, out[0], *args, lse=out[1], weights=out[2], stream=stream)

    ref = outs()
    call(h, ref)
    a, b = outs(), outs()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):  # two handles at once
        a[2].zero_()
        b[2].zero_()
        torch.cuda.synchronize()
        call(h, a, s1)
        call(h2, b, s2)
        torch.cuda.synchronize()
        for x, y, z in zip(ref, a, b):
            assert torch.equal(x, y) and torch.equal(x, z)
    c = outs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s1):
        c[2].zero_()
        call(h, c, s1)
    for _ in range(4):
        c[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(ref, c):
            assert torch.equal(x, y)
    h.close(), h2.close()


def test_attend_refusals():
    m = _m()
    dev = torch.device("cuda")
    table, cache = make_cache(TINY, [40], 20)
    h = m.Cache(TINY, 2, 1)
    q = make_q(TINY, 1, 20).to(dev)
    o = torch.empty_like(q)
    i32 = dict(dtype=torch.int32, device=dev)
    pos, req = torch.tensor([39], **i32), torch.tensor([0], **i32)
    t, c = torch.from_numpy(table).to(dev), torch.from_numpy(cache).to(dev)

    def refused(*a, code=None, **kw):
        with pytest.raises(m.MonoError if code else ValueError) as e:
            h.attend(*a, **kw)
        if code:
            assert e.value.code == code

    refused(q.float(), o, pos, req, t, c)
    refused(q[:, :-64], o, pos, req, t, c)
    refused(q, o[:, ::2], pos, req, t, c)
    refused(q, o, pos.long(), req, t, c)
    refused(q, o, pos.cpu(), req, t, c)
    refused(q, o, pos, req, t.t().contiguous().t()[:, :1].expand(1, 3), c)
    refused(q, o, pos, req, t, c[:, :8])
    refused(q, o, pos, req, t, c, scale=-1.0)
    refused(q, o, pos, req, t, c, lse=torch.empty((1, 3), device=dev))
    refused(q, o, pos, req, t, c, weights=torch.empty((2, 40), device=dev))
    refused(q, o, pos, req, t, c, window=-1, code=-1)
    refused(q, o, pos, req, t, c, sinks=-1, code=-1)
    three = make_q(TINY, 3, 20).to(dev)
    refused(three, torch.empty_like(three), torch.zeros(3, **i32), torch.zeros(3, **i32), t, c,
            code=-3)
    two = t.repeat(2, 1)
    refused(q, o, pos, req, two, c, code=-3)
    wide = torch.empty((2, q.shape[1] + 4), dtype=torch.bfloat16, device=dev)
    refused(wide[:, :q.shape[1]], wide.clone()[:, :q.shape[1]], torch.zeros(2, **i32),
            torch.zeros(2, **i32), t, c, code=-4)
    off = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device=dev)[1:1 + q.numel()].view(1, -1)
    refused(off, o, pos, req, t, c, code=-4)
    lap = torch.as_strided(c, c.shape, (c.stride(0), 64, 1))
    refused(q, o, pos, req, t, lap, code=-5)
    h.close()
    with pytest.raises(ValueError):
        h.attend(q, o, pos, req, t, c)


# ------------------------------------------------------------------------------ eviction
def run_evict(m, spec, weights, lengths, table, cache, budget, sinks, recent, dst=None,
              in_place_weights=True, alias_lengths=False, out_cols=None):
    dev = torch.device("cuda")
    n = len(lengths)
    h = m.Cache(spec, 1, n)
    w = torch.from_numpy(weights).to(dev)
    ln = torch.tensor(lengths, dtype=torch.int32, device=dev)
    nl = ln if alias_lengths else torch.full((n,), -9, dtype=torch.int32, device=dev)
    kept = torch.full((n, budget + 2), -7, dtype=torch.int32, device=dev)
    c = torch.from_numpy(cache).to(dev)
    wo = None if in_place_weights else torch.full((n, out_cols or weights.shape[1]), 77.0, device=dev)
    kw = {}
    if dst is not None:
        kw = dict(dst_table=torch.from_numpy(dst[0]).to(dev))
        if dst[1] is not None:
            kw["dst_cache"] = torch.from_numpy(dst[1]).to(dev)
    h.evict(w, ln, torch.from_numpy(table).to(dev), c, kept, nl, budget=budget, sinks=sinks,
            recent=recent, weights_out=wo, **kw)
    torch.cuda.synchronize()
    st = h.status()
    h.close()
    d = kw.get("dst_cache", c)
    return (kept.cpu().numpy(), nl.cpu().numpy(), (w if wo is None else wo).cpu().numpy(),
            c.cpu().numpy(), d.cpu().numpy(), st)


def check_evict(m, spec, lengths, budget, sinks, recent, seed, weights=None, where="in_place",
                in_place_weights=True, alias_lengths=False, out_cols=None):
    rng = np.random.default_rng(seed)
    table, cache = make_cache(spec, lengths, seed)
    cols = max(max(lengths), 1) + 3
    if weights is None:
        weights = np.exp(rng.standard_normal((len(lengths), cols)) * 2).astype(np.float32)
    bs, nbytes = spec["block_size"], spec["kv_dim"] + 4
    keep = co.evict(weights, lengths, budget, sinks, recent)
    dst = None
    if where != "in_place":
        per = [-(-len(k) // bs) for k in keep]
        dt = np.full((len(keep), max(max(per), 1)), -1, np.int32)
        nb = sum(per)
        pages = rng.permutation(nb)
        if where == "same_pool":
            cache = np.concatenate([cache, np.full((nb, *cache.shape[1:]), 0x55, np.uint8)])
            pages = pages + cache.shape[0] - nb
        o = 0
        for b, n in enumerate(per):
            dt[b, :n] = pages[o:o + n]
            o += n
        other = np.full((max(nb, 1), *cache.shape[1:]), 0x55, np.uint8)
        dst = (dt, None if where == "same_pool" else other)
    kept, nl, w, c, d, st = run_evict(m, spec, weights, lengths, table, cache, budget, sinks, recent,
                                      dst, in_place_weights, alias_lengths, out_cols)
    assert st == 0
    want_c = cache.copy()
    want_d = want_c if dst is None or dst[1] is None else dst[1].copy()
    want_w = weights.copy() if in_place_weights else np.full(w.shape, 77.0, np.float32)
    for b, k in enumerate(keep):
        assert nl[b] == len(k)
        assert kept[b, :len(k)].tolist() == k
        assert (kept[b, len(k):budget] == -1).all() and (kept[b, budget:] == -7).all()
        n, cols_out = len(k), want_w.shape[1]
        row = np.zeros(max(lengths[b], n), np.float32)
        row[:n] = weights[b, k]
        want_w[b, :min(len(row), cols_out)] = row[:cols_out]
        tab = table if dst is None else dst[0]
        for i, t in enumerate(k):
            want_d[tab[b, i // bs], i % bs, :nbytes] = cache[table[b, t // bs], t % bs, :nbytes]
    assert np.array_equal(w, want_w, equal_nan=True)
    # record padding is not compared: it may move along
    assert np.array_equal(d[..., :nbytes], want_d[..., :nbytes])
    if dst is not None and dst[1] is not None:
        assert np.array_equal(c, want_c)
    if dst is not None:
        used = np.zeros(d.shape[:2], bool)
        for b, k in enumerate(keep):
            for i in range(len(k)):
                used[dst[0][b, i // bs], i % bs] = True
        assert np.array_equal(d[~used], (cache if dst[1] is None else dst[1])[~used])


@pytest.mark.parametrize("where", ["in_place", "same_pool", "other_pool"])
@pytest.mark.parametrize("spec", [FULL, WIDE, ODD, MANY], ids=["full", "wide", "odd", "many"])
def test_evict(spec, where):
    check_evict(_m(), spec, [700, 0, 130, 1, 99, 100, 101], 100, 3, 20, seed=31, where=where,
                in_place_weights=where == "in_place")


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 0, 0),
                                                 (64, 64, 0), (64, 0, 64), (64, 32, 32), (999, 5, 5),
                                                 (1000, 0, 0), (2000, 4, 4)])
def test_evict_budgets(budget, sinks, recent):
    check_evict(_m(), TINY, [1000, 500, 1], budget, sinks, recent, seed=budget)


@pytest.mark.parametrize("kind", ["equal", "zero", "few", "nan", "inf", "negative", "signed_zero"])
def test_evict_ties_and_special_weights(kind):
    rng = np.random.default_rng(33)
    w = np.exp(rng.standard_normal((2, 600))).astype(np.float32)
    if kind == "equal":
        w[:] = 0.25
    elif kind == "zero":
        w[:] = 0.0
    elif kind == "few":
        w = rng.integers(0, 3, w.shape).astype(np.float32)
    elif kind == "nan":
        w[:, ::3] = np.nan
        w[:, 1::3] = -np.inf
    elif kind == "inf":
        w[:, ::2] = np.inf
    elif kind == "negative":
        w = -w
    else:
        w = np.where(rng.random(w.shape) < 0.5, 0.0, -0.0).astype(np.float32)
    for budget in (100, 350):
        check_evict(_m(), TINY, [597, 410], budget, 2, 30, seed=34, weights=w)


def test_evict_long_and_ragged():
    rng = np.random.default_rng(35)
    lengths = [20000, 3, 9001, 1024, 16385]
    check_evict(_m(), TINY, lengths, 8000, 4, 100, seed=35)
    check_evict(_m(), TINY, lengths, 8000, 4, 100, seed=36, where="other_pool")
    del rng


def test_evict_aliased_lengths_and_short_weight_rows_out():
    check_evict(_m(), TINY, [300, 80], 120, 1, 8, seed=37, alias_lengths=True)
    check_evict(_m(), TINY, [300, 80], 120, 1, 8, seed=38, in_place_weights=False, out_cols=50)


def test_evict_repeats_in_a_graph():
    """Out of place, so that every replay finds the same inputs."""
    m = _m()
    dev = torch.device("cuda")
    lengths = [5000, 1300]
    table, cache = make_cache(TINY, lengths, 39)
    w = torch.rand((2, 5000), device=dev)
    dt = torch.arange(126, dtype=torch.int32, device=dev).view(2, 63)
    h = m.Cache(TINY, 1, 2)
    c, t = torch.from_numpy(cache).to(dev), torch.from_numpy(table).to(dev)
    ln = torch.tensor(lengths, dtype=torch.int32, device=dev)

    def outs():
        return [torch.zeros((2, 1000), dtype=torch.int32, device=dev),
                torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros((2, 1000), device=dev),
                torch.zeros((126, 16, 80), dtype=torch.uint8, device=dev)]

    def call(o, s):
        h.evict(w, ln, t, c, o[0], o[1], budget=1000, sinks=2, recent=50, weights_out=o[2],
                dst_table=dt, dst_cache=o[3], stream=s)

    s = torch.cuda.Stream()
    ref, got = outs(), outs()
    torch.cuda.synchronize()
    call(ref, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(got, s)
    for _ in range(5):
        for o in got:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            assert torch.equal(a, b)
    h.close()


def test_evict_lengths_beyond_the_table_and_unmapped_pages():
    m = _m()
    table, cache = make_cache(TINY, [64], 40)
    w = np.ones((1, 64), np.float32)
    kept, nl, _, c, _, st = run_evict(m, TINY, w, [1000], table, cache, 10, 2, 2)
    assert st == 1 and nl[0] == 10 and kept[0, :10].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 62, 63]
    table[0, 3] = -1
    kept, nl, _, c2, _, st = run_evict(m, TINY, w, [64], table, cache, 10, 2, 2)
    assert st == 1 and nl[0] == 10
    pg = table[0, 0]
    assert np.array_equal(c2[pg, :8], cache[pg, :8])  # the mapped ones are in place already


def test_evict_refusals():
    m = _m()
    dev = torch.device("cuda")
    h = m.Cache(TINY, 1, 1)
    i32 = dict(dtype=torch.int32, device=dev)
    w, ln, t = torch.zeros((1, 64), device=dev), torch.zeros(1, **i32), torch.zeros((1, 4), **i32)
    c = torch.zeros((4, 16, 80), dtype=torch.uint8, device=dev)
    kept, nl = torch.zeros((1, 8), **i32), torch.zeros(1, **i32)

    def refused(code=None, **kw):
        d = dict(weights=w, lengths=ln, block_table=t, kv_cache=c, kept=kept, new_lengths=nl, budget=8)
        with pytest.raises(m.MonoError if code else ValueError) as e:
            h.evict(**dict(d, **kw))
        if code:
            assert e.value.code == code

    refused(weights=w.double())
    refused(budget=9)
    refused(kept=kept.long())
    refused(lengths=ln.cpu())
    refused(dst_cache=c)
    refused(weights_out=torch.zeros((2, 64), device=dev))
    refused(code=-1, budget=0)
    refused(code=-1, sinks=5, recent=4)
    refused(code=-1, sinks=-1)
    refused(code=-1, recent=-1)
    refused(code=-3, weights=torch.zeros((2, 64), device=dev), lengths=torch.zeros(2, **i32),
            block_table=torch.zeros((2, 4), **i32), kept=torch.zeros((2, 8), **i32),
            new_lengths=torch.zeros(2, **i32))
    h.close()


# -------------------------------------------------------------------------- verification
def run_verify(m, target, draft, tokens_in, row_start, u, r, greedy=None, stream=None):
    dev = torch.device("cuda")
    rows, n = target.shape[0], len(row_start) - 1
    i32 = dict(dtype=torch.int32, device=dev)
    acc = torch.full((n,), -9, **i32)
    out = torch.full((rows,), -9, **i32)
    m.verify_drafts(target, draft, torch.tensor(tokens_in, **i32), torch.tensor(row_start, **i32),
                    torch.tensor(u, device=dev), torch.tensor(r, device=dev), acc, out,
                    greedy=None if greedy is None else torch.tensor(greedy, **i32), stream=stream)
    torch.cuda.synchronize()
    return acc.tolist(), out.tolist()


def check_verify(m, target, draft, tokens_in, row_start, u, r, greedy=None):
    acc, out = run_verify(m, target, draft, tokens_in, row_start, u, r, greedy)
    ea, eo = co.verify(target.double().cpu().numpy(),
                       None if draft is None else draft.double().cpu().numpy(), tokens_in,
                       row_start, u, r, greedy)
    assert acc == ea
    assert out == [-9 if x is None else x for x in eo]


def make_verify(counts, V, dtype, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    starts = np.concatenate([[0], np.cumsum([c + 1 for c in counts])]).tolist()
    rows = starts[-1]
    logits = torch.randn((rows, V), generator=g) * std
    dl = logits + torch.randn((rows, V), generator=g) * 0.7
    target, q = torch.softmax(logits, -1), torch.softmax(dl, -1)
    tok = torch.multinomial(q, 1, generator=g)[:, 0].tolist()
    u = torch.rand(rows, generator=g).numpy()
    r = torch.rand(len(counts), generator=g).numpy()
    return target.to(dtype).cuda(), q.to(dtype).cuda(), tok, starts, u, r


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1, 2, 17, 1000, 8191, 32000, 100003])
def test_verify(V, dtype):
    m = _m()
    counts = [5, 0, 3, 1, 7, 2]
    target, draft, tok, starts, u, r = make_verify(counts, V, dtype, seed=V)
    check_verify(m, target, draft, tok, starts, u, r)
    check_verify(m, target, None, tok, starts, u, r)
    check_verify(m, target, draft, tok, starts, u, r, greedy=[0, 1, 1, 0, 1, 0])


@pytest.mark.parametrize("n", [1, 30, 200, 700])
def test_verify_many_requests(n):
    m = _m()
    counts = [i % 6 for i in range(n)]
    target, draft, tok, starts, u, r = make_verify(counts, 1501, torch.float32, seed=n)
    check_verify(m, target, draft, tok, starts, u, r, greedy=[int(i % 5 == 4) for i in range(n)])


def test_verify_every_draft_stands_or_falls():
    m = _m()
    target, draft, tok, starts, u, r = make_verify([4, 4], 333, torch.float32, seed=51)
    check_verify(m, target, target, tok, starts, u, r)  # q = p: all stand
    acc, _ = run_verify(m, target, target, tok, starts, u, r)
    assert acc == [4, 4]
    for j in range(len(tok)):
        target[j, tok[j]] = 0.0
    check_verify(m, target, draft, tok, starts, u, r)  # p(x) = 0: the first falls
    acc, _ = run_verify(m, target, draft, tok, starts, u, r)
    assert acc == [0, 0]


def test_verify_random_numbers_at_the_ends():
    m = _m()
    target, draft, tok, starts, u, r = make_verify([2] * 6, 777, torch.float32, seed=52)
    top = np.float32(1.0) - np.float32(2.0 ** -24)
    u[:9] = [0.0, top, 0.5] * 3
    r = np.array([0.0, top, 0.0, top, 0.5, 2.0 ** -30], np.float32)
    check_verify(m, target, draft, tok, starts, u, r)


def test_verify_strides_and_unaligned_rows():
    m = _m()
    for dtype in (torch.float32, torch.bfloat16):
        target, draft, tok, starts, u, r = make_verify([3, 2, 4], 1003, dtype, seed=53)
        big = torch.full((target.shape[0], 1100), float("nan"), dtype=dtype, device="cuda")
        for off in (0, 1, 3):
            view = big[:, off:off + 1003]
            view.copy_(target)
            dv = torch.full((target.shape[0], 1031), float("nan"), dtype=dtype,
                            device="cuda")[:, 5:5 + 1003]
            dv.copy_(draft)
            check_verify(m, view, dv, tok, starts, u, r, greedy=[0, 1, 0])


def test_verify_rows_outside_requests_and_bad_tokens():
    m = _m()
    target, draft, tok, starts, u, r = make_verify([2, 2, 2], 100, torch.float32, seed=54)
    tok[0], tok[3], tok[4] = -1, 100, 2 ** 31 - 1
    check_verify(m, target, draft, tok, [1, 3, 3, 7], u, r)   # row 0, 7, 8 belong to nobody
    check_verify(m, target, draft, tok, [-5, 3, 6, 99], u, r)  # cut to the rows
    check_verify(m, target, None, tok, starts, u, r, greedy=[1, 0, 1])


def test_verify_zero_and_nan_entries():
    m = _m()
    target, draft, tok, starts, u, r = make_verify([2, 2, 2, 2], 500, torch.float32, seed=55)
    target[0] = 0.0                 # nothing to draw from
    target[3, 100:200] = float("nan")
    target[3, 200:300] = -1.0
    draft[3, :50] = float("nan")
    target[6] = 0.0
    target[6, 7] = 1.0              # a certain token that the draft also has
    draft[6] = target[6] * 2
    tok[6] = 8
    check_verify(m, target, draft, tok, starts, u, r)
    target[9, :] = float("nan")
    check_verify(m, target, draft, tok, starts, u, r, greedy=[1, 1, 1, 1])


def test_verify_greedy_ties_take_the_first():
    m = _m()
    V = 4099
    t = torch.zeros((4, V), device="cuda")
    t[:, [77, 1000, 4098]] = 3.0
    t[1] -= 5.0  # logits may be negative
    check_verify(m, t, None, [77, 77, 1000, 0], [0, 4], np.zeros(4, np.float32),
                 np.zeros(1, np.float32), greedy=[1])
    acc, out = run_verify(m, t, None, [77, 77, 1000, 0], [0, 4], np.zeros(4, np.float32),
                          np.zeros(1, np.float32), greedy=[1])
    assert acc == [2] and out == [77, 77, 77, -1]


def test_verify_follows_the_target():
    """Over a grid of random numbers and drafts weighted by q, the token at the first row has
    the target's distribution (to a step of each grid)."""
    m = _m()
    V, n = 5, 48
    p = torch.tensor([0.4, 0.3, 0.15, 0.1, 0.05])
    q = torch.tensor([0.1, 0.2, 0.3, 0.35, 0.05])
    got = np.zeros(V)
    grid = (np.arange(n, dtype=np.float32) + 0.5) / n
    rows = 2 * n * n
    for x in range(V):
        u = np.repeat(np.repeat(grid, n), 2).astype(np.float32)
        r = np.tile(grid, n).astype(np.float32)
        tok = [x] * rows
        _, out = run_verify(m, p.repeat(rows, 1).cuda(), q.repeat(rows, 1).cuda(), tok,
                            list(range(0, rows + 1, 2)), u, r)
        first = np.array(out[::2])
        for v in range(V):
            got[v] += float(q[x]) * (first == v).mean()
    assert np.abs(got - p.numpy()).max() <= 2.0 / n


def test_verify_in_a_graph_and_on_a_stream():
    m = _m()
    dev = torch.device("cuda")
    target, draft, tok, starts, u, r = make_verify([3] * 20, 5000, torch.bfloat16, seed=57)
    i32 = dict(dtype=torch.int32, device=dev)
    t_in, t_st = torch.tensor(tok, **i32), torch.tensor(starts, **i32)
    ud, rd = torch.tensor(u, device=dev), torch.tensor(r, device=dev)
    acc, out = torch.zeros(20, **i32), torch.zeros(80, **i32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        m.verify_drafts(target, draft, t_in, t_st, ud, rd, acc, out, stream=s)
    ea, eo = co.verify(target.double().cpu().numpy(), draft.double().cpu().numpy(), tok, starts, u, r)
    for _ in range(3):
        acc.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert acc.tolist() == ea and out.tolist() == eo


def test_verify_refusals():
    m = _m()
    t = torch.zeros((2, 10), device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    a = dict(target=t, draft=t, draft_tokens=torch.zeros(2, **i32),
             row_start=torch.tensor([0, 2], **i32), u=torch.zeros(2, device="cuda"),
             r=torch.zeros(1, device="cuda"), accepted=torch.zeros(1, **i32),
             tokens=torch.zeros(2, **i32))
    for bad in (dict(target=t.double()), dict(draft=t.half()), dict(draft=t[:, :9]),
                dict(target=t.cpu()), dict(draft_tokens=torch.zeros(3, **i32)),
                dict(u=torch.zeros(2)), dict(r=torch.zeros(2, device="cuda")),
                dict(row_start=torch.zeros(2, device="cuda")), dict(greedy=torch.zeros(3, **i32)),
                dict(target=t[:1].expand(2, 10)), dict(target=t.t().contiguous().t()),
                dict(accepted=torch.zeros(2, **i32)), dict(tokens=torch.zeros((1, 2), **i32))):
        with pytest.raises(ValueError):
            m.verify_drafts(**dict(a, **bad))


# ------------------------------------------------------------------------- run together
def test_a_serving_step_end_to_end():
    """On a layer's own cache: steps insert records, the attention reads what they left (and
    equals the layer's window attention where the window is the same), an eviction halves the
    caches, the attention reads the compacted ones, the layer goes on at the new lengths, and the
    step's drafts are verified."""
    m = _m()
    import gen
    from tests.gpu_harness import f16_to_bf16_bits, to_device
    from tests.helpers import bf16_f64
    dev = torch.device("cuda")
    spec, w, st = gen.make_workload("wide_r9")
    st = gen.make_step(spec, gen.WORKLOADS["wide_r9"], prefill_tokens=1 << 20)
    wd, sd = to_device(w, st, dev)
    layer = m.Layer(spec, wd)
    rows, W = st["rows"], spec["n_q_heads"] * spec["head_dim"]
    cache = sd["kv_cache"].clone()
    out = torch.empty_like(sd["x"])
    layer.step(sd["x"], out, sd["positions"], sd["row_req"], sd["block_table"], cache)
    torch.cuda.synchronize()
    q = torch.from_numpy(layer.read("q", rows * W * 2).view(np.int16).reshape(rows, W)).view(
        torch.bfloat16)
    o_step = bf16_f64(f16_to_bf16_bits(layer.read("o", rows * W * 2).view(np.float16).reshape(rows, W)))
    pos, req = st["positions"].tolist(), st["row_req"].tolist()
    table = st["block_table"].numpy()
    h = m.Cache(spec, rows, len(st["contexts"]))
    # the layer's own window: the same result within both sides' bounds
    o, _, _, s = run_attend(m, spec, q, pos, req, table, cache, handle=h, window=spec["window"])
    eo, tol, *_ = co.attend(spec, q.double().numpy(), pos, req, table, cache.cpu().numpy(),
                            window=spec["window"])
    assert s == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(o - o_step) <= 2 * tol).all()
    # the whole context, with the weights
    lengths = [c + n for c, n in zip(st["contexts"], st["rows_per_req"])]
    w0 = torch.zeros((len(lengths), max(lengths)))
    host = cache.cpu().numpy()
    o, _, acc, s = run_attend(m, spec, q, pos, req, table, cache, handle=h, weights=w0)
    eo, tol, _, _, ew, wtol = co.attend(spec, q.double().numpy(), pos, req, table, host,
                                        n_weights=max(lengths))
    assert s == 0 and (np.abs(o - eo) <= tol).all()
    assert (np.abs(acc - ew) <= wtol + 2.0 ** -24 * 200 * ew).all()
    # evict in place, weights and lengths with it
    budget = 200
    wt = torch.from_numpy(acc).float().to(dev)
    keep = co.evict(acc.astype(np.float32), lengths, budget, 4, 32)
    ln = torch.tensor(lengths, dtype=torch.int32, device=dev)
    kept = torch.empty((len(lengths), budget), dtype=torch.int32, device=dev)
    h.evict(wt, ln, sd["block_table"], cache, kept, ln, budget=budget, sinks=4, recent=32)
    torch.cuda.synchronize()
    assert h.status() == 0 and ln.tolist() == [len(k) for k in keep]
    bs, nb = spec["block_size"], spec["kv_dim"] + 4
    now = cache.cpu().numpy()
    for b, k in enumerate(keep):
        assert kept[b, :len(k)].tolist() == k
        for i, t in enumerate(k):
            assert np.array_equal(now[table[b, i // bs], i % bs, :nb], host[table[b, t // bs], t % bs, :nb])
    # the next step continues at the new lengths, and the attention over it
    pos2 = [len(keep[b]) + sum(1 for i in range(r) if req[i] == b and pos[i] >= 0) if pos[r] >= 0 else -1
            for r, b in enumerate(req)]
    p2 = torch.tensor(pos2, dtype=torch.int32, device=dev)
    layer.step(sd["x"], out, p2, sd["row_req"], sd["block_table"], cache)
    torch.cuda.synchronize()
    assert layer.status() == 0
    o, _, _, s = run_attend(m, spec, q, pos2, req, table, cache, handle=h, window=100, sinks=4)
    eo, tol, *_ = co.attend(spec, q.double().numpy(), pos2, req, table, cache.cpu().numpy(),
                            window=100, sinks=4)
    assert s == 0 and (np.abs(o - eo) <= tol).all()
    # which of the step's drafts stand (each request's rows but the pad row)
    counts = [n - 1 for n in st["rows_per_req"]]
    target, draft, tok, starts, u, r = make_verify(counts, 2000, torch.float32, seed=60)
    check_verify(m, target, draft, tok, starts, u, r)
    layer.close(), h.close()


def test_attend_work_limit():
    """The work of a step is counted in 32 bits: (tiles of 128 tokens + 16) * rows < 2^31."""
    m = _m()
    rows, blocks = 1024, (2 ** 21 - 17) * 8  # of 16 tokens
    table = torch.full((1, blocks + 8), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    pool = torch.zeros((1, 16, 80), dtype=torch.uint8, device="cuda")
    h = m.Cache(TINY, max_rows=rows, max_requests=1)
    q = torch.zeros((rows, 256), dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, float("nan"))
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    with pytest.raises(m.MonoError):
        h.attend(q, o, pos, pos, table, pool)
    h.attend(q, o, pos, pos, table[:, :blocks].contiguous(), pool)
    torch.cuda.synchronize()
    assert h.status() == 0 and not o.any()
    h.close()


@pytest.mark.parametrize("rows", [1, 6], ids=["narrow", "wide"])
def test_attend_negative_token_scales(rows):
    """A record is its codes times its scale, whatever the scale's sign."""
    m = _m()
    L = 700
    table, cache = make_cache(FULL, [L], seed=rows)
    rng = np.random.default_rng(3)
    for t in rng.choice(L, 300, replace=False):
        rec = cache[table[0, t // 128], t % 128]
        rec[512:516] = (-rec[512:516].view(np.float32)).view(np.uint8)
    q = make_q(FULL, rows, 4)
    pos = list(range(L - rows, L))
    w0 = torch.zeros((1, L))
    o, lse, w, st = run_attend(m, FULL, q, pos, [0] * rows, table, cache, weights=w0)
    eo, tol, el, ltol, ew, wtol = co.attend(FULL, q.double().numpy(), pos, [0] * rows, table, cache,
                                            n_weights=L)
    assert st == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()
    assert (np.abs(w - ew) <= wtol + 2.0 ** -24 * (rows * 64 + 2) * ew).all()


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("window", [0, 200])
def test_attend_rows_per_request(n, window):
    """Every number of query columns: 16 heads a slice times n rows, as one group or two."""
    check_attend(_m(), FULL, [700, 130], [n, n], seed=70 + n, window=window, sinks=2 * (window > 0))


BIG = dict(n_q_heads=256, head_dim=64, kv_dim=1024, block_size=32, kv_record_bytes=1040)


@pytest.mark.parametrize("rows", [1, 2, 3, 4])
def test_attend_widest_records(rows):
    check_attend(_m(), BIG, [300, 45], [rows, 1], seed=80 + rows)


@pytest.mark.parametrize("rows", [1, 2, 6], ids=["narrow", "narrow2", "wide"])
@pytest.mark.parametrize("down", [False, True], ids=["rising", "falling"])
def test_attend_scores_that_rise_by_orders(rows, down):
    """Values, and with them scores, that grow along the context: the running reference has to move
    many times, and by more than an exponential can hold."""
    m = _m()
    L = 2000
    table, cache = make_cache(FULL, [L], seed=90 + rows)
    for t in range(L):
        rec = cache[table[0, t // 128], t % 128]
        x = (L - 1 - t if down else t) / L
        rec[512:516] = (rec[512:516].view(np.float32) * np.float32(0.02 * 3000.0 ** x)).view(np.uint8)
    q = make_q(FULL, rows, 5)
    pos = list(range(L - rows, L))
    o, lse, w, st = run_attend(m, FULL, q, pos, [0] * rows, table, cache, weights=torch.zeros((1, L)))
    eo, tol, el, ltol, ew, wtol = co.attend(FULL, q.double().numpy(), pos, [0] * rows, table, cache,
                                            n_weights=L)
    assert st == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()
    # (each of the rows * 64 weights that a token's sum is of is an f32: below 2^-126 it may be 0)
    assert (np.abs(w - ew) <= wtol + 2.0 ** -24 * (rows * 64 + 2) * ew + rows * 64 * 2.0 ** -126).all()


@pytest.mark.parametrize("rows", [1, 6], ids=["narrow", "wide"])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_nan_records_outside_the_view(rows, causal):
    """NaN codes and scales in every token that no row sees, and behind the rows that are ahead of
    them: window, first tokens, later rows' tokens."""
    m = _m()
    L, W, S = 900, 300, 3
    table, cache = make_cache(FULL, [L], seed=95)
    pos = list(range(L - 30, L - 30 + rows))
    hi = pos[-1]
    first = (pos[0] if causal else hi) - W + 1
    for t in range(L):
        if not (t <= hi and (t >= first or t < S)):
            cache[table[0, t // 128], t % 128] = 0x7F
    q = make_q(FULL, rows, 6)
    kw = dict(window=W, sinks=S, causal=causal)
    o, lse, w, st = run_attend(m, FULL, q, pos, [0] * rows, table, cache, weights=torch.zeros((1, L)),
                               **kw)
    eo, tol, el, ltol, ew, wtol = co.attend(FULL, q.double().numpy(), pos, [0] * rows, table, cache, W,
                                            S, causal, n_weights=L)
    assert st == 0 and (np.abs(o - eo) <= tol).all() and (np.abs(lse - el) <= ltol).all()
    assert (np.abs(w - ew) <= wtol + 2.0 ** -24 * (rows * 64 + 2) * ew).all()
    # a later row's token that holds NaN reaches the rows that see it, and no other
    if rows > 1 and causal:
        t = pos[3]
        cache[table[0, t // 128], t % 128, :512] = 0x7F
        o, _, _, st = run_attend(m, FULL, q, pos, [0] * rows, table, cache, **kw)
        assert st == 0 and np.isnan(o[3:]).all() and (np.abs(o[:3] - eo[:3]) <= tol[:3]).all()


def test_attend_largest_step():
    """1024 rows of 512 requests, in any order, some of them pad rows."""
    rng = np.random.default_rng(7)
    lengths = rng.integers(2, 40, 512).tolist()
    check_attend(_m(), TINY, lengths, [2] * 511 + [1], seed=97, pads=(5,), shuffle=True)


def test_two_caches_at_once():
    """Two handles on two streams give what each gives alone."""
    m = _m()
    dev = torch.device("cuda")
    sets = []
    for k, (spec, n) in enumerate([(FULL, 1), (FULL, 6), (WIDE, 3)]):
        lengths = [3000 + 501 * k, 700]
        table, cache = make_cache(spec, lengths, seed=98 + k)
        pos = [p for L in lengths for p in range(L - n, L)]
        req = [b for b in range(2) for _ in range(n)]
        q = make_q(spec, 2 * n, 98 + k).to(dev)
        args = (torch.tensor(pos, dtype=torch.int32, device=dev),
                torch.tensor(req, dtype=torch.int32, device=dev),
                torch.from_numpy(table).to(dev), torch.from_numpy(cache).to(dev))
        h = m.Cache(spec, max_rows=2 * n, max_requests=2)
        alone = torch.empty_like(q)
        h.attend(q, alone, *args)
        sets.append((h, q, args, alone, torch.cuda.Stream(), [torch.empty_like(q) for _ in range(20)]))
    torch.cuda.synchronize()
    for i in range(20):
        for h, q, args, _, s, outs in sets:
            h.attend(q, outs[i], *args, stream=s)
    torch.cuda.synchronize()
    for h, _, _, alone, _, outs in sets:
        assert h.status() == 0 and all(torch.equal(alone, x) for x in outs)
        h.close()
