"""Appending to the cache and rotating heads on the GPU against tests/rope_oracle.py.  The interface
states every rounding, so records and 32-bit results are compared bit for bit with the formulas
evaluated in 32 bits; against 64 bits, with u = 2^-24, a rotated value is off by at most
2 u (|x1 cos| + |x2 sin|) before its rounding to 16 bits (half a step), if any."""
import numpy as np
import pytest
import torch

from tests import rope_oracle as ro
from tests.test_gpu_cache_ops import FULL, MANY, ODD, THREE, TINY, WIDE, _m

pytestmark = pytest.mark.gpu
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LAYOUTS = dict(full=FULL, wide=WIDE, tiny=TINY, odd=ODD, three=THREE, many=MANY)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def pages(spec, lengths, seed):
    """A block table over random pages, and their number."""
    rng = np.random.default_rng(seed)
    bs = spec["block_size"]
    per = [max(1, -(-n // bs)) for n in lengths]
    perm = rng.permutation(sum(per) + 2)
    t = np.full((len(per), max(per)), -1, np.int32)
    o = 0
    for b, n in enumerate(per):
        t[b, :n] = perm[o:o + n]
        o += n
    return t, o + 2


def codes_of(vals):
    return torch.from_numpy(vals).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def expected(spec, cache, kv32, tab, positions, rope_positions, row_req, table, offset, interleaved):
    """The cache's bytes after an append of kv32 (the stored values, f32)."""
    out, kv, bs = cache.copy(), spec["kv_dim"], spec["block_size"]
    live = [p if 0 <= p else -1 for p in rope_positions]
    y = kv32 if tab is None else ro.rotate(kv32, tab, live, spec["head_dim"], offset, interleaved,
                                           dtype=np.float32)
    for r, p in enumerate(positions):
        b = row_req[r]
        if p < 0 or not 0 <= b < table.shape[0] or p // bs >= table.shape[1]:
            continue
        pg = table[b, p // bs]
        if not 0 <= pg < cache.shape[0]:
            continue
        vals, s = ro.record(y[r])
        rec = out[pg, p % bs]
        rec[:kv] = codes_of(vals)
        rec[kv:kv + 4] = np.frombuffer(np.float32(s).tobytes(), np.uint8)
    return out


def same(got, want, kv):
    """Equal bytes, but that a NaN code may have either sign."""
    nan = (got & 0x7F == 0x7F) & (want & 0x7F == 0x7F)
    nan[..., kv:] = False
    return np.array_equal(np.where(nan, 0, got), np.where(nan, 0, want))


def check_append(spec, lengths, rows_per, dtype="bf16", dim=None, offset=None, interleaved=False,
                 shift=0, q="out", pads=(), seed=0, shuffle=True):
    m = _m()
    dh, kv = spec["head_dim"], spec["kv_dim"]
    dim = dh if dim is None else dim
    at = dh - dim if offset is None else offset
    rng = np.random.default_rng(seed)
    pos = [p for L, n in zip(lengths, rows_per) for p in range(L - n, L)]
    req = [b for b, n in enumerate(rows_per) for _ in range(n)]
    for i in pads:
        pos.insert(i, -1)
        req.insert(i, 0)
    if shuffle:
        o = rng.permutation(len(pos))
        pos, req = [pos[i] for i in o], [req[i] for i in o]
    rp = [p if p < 0 else p + shift for p in pos]
    tab = ro.table(max(rp) + 1, dim)
    table, nb = pages(spec, lengths, seed)
    cache = rng.integers(0, 256, (nb, spec["block_size"], spec["kv_record_bytes"]), dtype=np.uint8)
    x = torch.from_numpy(rng.standard_normal((len(pos), kv)).astype(np.float32)).to(DTYPES[dtype])
    qx = torch.from_numpy(rng.standard_normal((len(pos), spec["n_q_heads"] * dh)).astype(np.float32)).to(DTYPES[dtype])
    h = m.Cache(spec, max_rows=1, max_requests=1)  # (no limits of an append)
    cd, qd = torch.from_numpy(cache).cuda(), qx.cuda()
    qo = qd if q == "place" else torch.full_like(qd, 7.0)
    h.append(x.cuda(), i32(pos), i32(req), i32(table), cd, rope=torch.from_numpy(tab).cuda(),
             rope_offset=offset, interleaved=interleaved, rope_positions=i32(rp) if shift else None,
             q=None if q is None else qd, q_out=None if q != "out" else qo)
    torch.cuda.synchronize()
    assert h.status() == 0
    h.close()
    want = expected(spec, cache, x.float().numpy(), tab, pos, rp, req, table, at, interleaved)
    assert same(cd.cpu().numpy(), want, kv)
    if q is None:
        return
    f32 = ro.rotate(qx.float().numpy(), tab, rp, dh, at, interleaved, dtype=np.float32)
    f32 = torch.from_numpy(f32).to(DTYPES[dtype])
    if q == "out":
        f32[torch.tensor(pos) < 0] = 7.0
    assert torch.equal(qo.cpu(), f32)
    # and against 64 bits
    ex = ro.rotate(qx.double().numpy(), tab, rp, dh, at, interleaved)
    mag = np.abs(ro.rotate(np.abs(qx.double().numpy()), np.abs(tab) * np.repeat([1, 1], dim // 2), rp,
                           dh, at, interleaved, inverse=True))
    mag += np.abs(ro.rotate(np.abs(qx.double().numpy()), np.abs(tab), rp, dh, at, interleaved))
    half = torch.finfo(DTYPES[dtype]).eps / 2
    live = np.array(pos) >= 0
    off = np.abs(qo.cpu().double().numpy() - ex)
    bound = half * np.abs(ex) + 2.1 * 2.0 ** -24 * mag + (2.0 ** -25 if dtype == "f16" else 0)
    assert (off <= bound)[live].all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_layouts(layout, dtype, interleaved):
    check_append(LAYOUTS[layout], [37, 1, 130, 16], [5, 1, 6, 16], dtype=dtype, interleaved=interleaved,
                 pads=(0, 9))


@pytest.mark.parametrize("dim,offset", [(16, 0), (16, 48), (16, 40), (32, 8), (48, 16), (48, 0), (64, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotated_dimensions(dim, offset, interleaved):
    check_append(THREE, [50, 3], [7, 3], dim=dim, offset=offset, interleaved=interleaved, seed=dim + offset)
    check_append(ODD, [50, 3], [7, 3], dim=2 * dim, offset=offset, interleaved=interleaved, seed=dim, q="place")


def test_append_far_positions_and_shifted_slots():
    check_append(WIDE, [300, 9], [4, 4], shift=150000, dim=32)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 255, 3001])
def test_append_many_rows(rows):
    check_append(TINY, [rows + 5], [rows], dim=32, seed=rows, q="place" if rows % 2 else "out")


def test_append_without_queries():
    check_append(FULL, [400], [300], dim=64, q=None, dtype="f32")


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_without_rotation_stores_what_is_given(dtype):
    m = _m()
    x = torch.randn((9, 128), generator=torch.Generator().manual_seed(3)).to(DTYPES[dtype])
    x[2] = 0.0
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    x[5] = 1e-39 if dtype != "f16" else 6e-8  # subnormal
    x[6] = 2.0 ** -148 if dtype == "f32" else 0.0
    table, nb = pages(WIDE, [20], 1)
    cache = np.zeros((nb, 64, 144), np.uint8)
    h = m.Cache(WIDE, 1, 1)
    cd = torch.from_numpy(cache).cuda()
    pos, req = list(range(11, 20)), [0] * 9
    h.append(x.cuda(), i32(pos), i32(req), i32(table), cd)
    torch.cuda.synchronize()
    assert h.status() == 0
    want = expected(WIDE, cache, x.float().numpy(), None, pos, pos, req, table, 0, False)
    assert same(cd.cpu().numpy(), want, 128)
    h.close()


def test_append_stores_a_records_as_the_layers_step_does():
    import gen
    m = _m()
    spec, w, st = gen.make_workload("small_r11")
    dev = torch.device("cuda")
    wd = {k: v.to(dev) for k, v in w.items()}
    sd = {k: (v.to(dev) if isinstance(v, torch.Tensor) else v) for k, v in st.items()}
    layer = m.Layer(spec, wd)
    before = sd["kv_cache"].clone()
    out = torch.empty_like(sd["x"])
    layer.step(sd["x"], out, sd["positions"], sd["row_req"], sd["block_table"], sd["kv_cache"])
    torch.cuda.synchronize()
    rows = st["rows"]
    kvn = torch.from_numpy(layer.read("kvn").view(np.int16).copy()).view(torch.bfloat16)
    kvn = kvn[:rows * spec["kv_dim"]].view(rows, -1).cuda()
    h = m.Cache(spec, max_rows=1, max_requests=1)
    h.append(kvn, sd["positions"], sd["row_req"], sd["block_table"], before)
    torch.cuda.synchronize()
    assert h.status() == 0 and torch.equal(before, sd["kv_cache"])
    h.close()
    layer.close()


def test_append_bad_rows_are_left_out_and_reported():
    m = _m()
    table = np.array([[0, -1, 7], [1, 2, 99]], np.int32)
    cache = np.full((8, 64, 144), 0x5A, np.uint8)
    x = torch.randn((8, 128), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    q = torch.randn((8, 1024), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    tab = ro.table(200, 64)
    h = m.Cache(WIDE, 1, 1)
    for pos, req, rp, bits in (
            ([3, 70, 130, 190, 192, 5, 6, -1], [0, 0, 0, 1, 0, 2, -1, 0], None, m.STATUS_UNMAPPED_PAGE),
            ([3, 4, 5, 6, 7, 8, -1, 9], [0] * 8, [0, 199, 200, -1, 2 ** 31 - 1, -2 ** 31, 5, 3],
             m.STATUS_POSITION)):
        cd, qo = torch.from_numpy(cache).cuda(), torch.full((8, 1024), 7.0, dtype=torch.bfloat16, device="cuda")
        h.append(x.cuda(), i32(pos), i32(req), i32(table), cd, rope=torch.from_numpy(tab).cuda(),
                 rope_positions=None if rp is None else i32(rp), q=q.cuda(), q_out=qo)
        torch.cuda.synchronize()
        assert h.status(clear=True) == bits
        eff = [p if p < 0 else t for p, t in zip(pos, pos if rp is None else rp)]
        live = [p >= 0 and 0 <= t < 200 for p, t in zip(pos, eff)]
        p2 = [p if ok else -1 for p, ok in zip(pos, live)]
        t2 = [t if ok else -1 for t, ok in zip(eff, live)]
        want = expected(WIDE, cache, x.float().numpy(), tab, p2, t2, req, table, 0, False)
        assert same(cd.cpu().numpy(), want, 128)
        f32 = torch.from_numpy(ro.rotate(q.float().numpy(), tab, t2, 64, 0, False, dtype=np.float32)).to(torch.bfloat16)
        f32[~torch.tensor(live)] = 7.0
        assert torch.equal(qo.cpu(), f32)
    assert h.status() == 0
    h.close()


def test_append_strided_rows_tables_and_caches():
    m = _m()
    g = torch.Generator().manual_seed(8)
    big = torch.randn((6, 400), generator=g).to(torch.bfloat16).cuda()
    kv, q = big[:, 8:136], torch.randn((6, 2048), generator=g).to(torch.bfloat16).cuda()[:, 512:1536]
    tab = ro.table(50, 32)
    wide = torch.full((50, 64), float("nan"), device="cuda")
    wide[:, 12:44] = torch.from_numpy(tab).cuda()
    pool = torch.full((4, 70, 176), 0x11, dtype=torch.uint8, device="cuda")
    view = pool[:, 3:67, 16:160]  # pages and records further apart than they are long
    qo = torch.zeros((6, 1040), dtype=torch.bfloat16, device="cuda")
    table, pos, req = np.array([[2, 0], [3, 1]], np.int32), [0, 63, 64, 30, 31, 100], [0, 0, 0, 1, 1, 1]
    rp = [0, 49, 7, 8, 9, 10]
    before = pool.cpu().numpy().copy()
    h = m.Cache(WIDE, 1, 1)
    h.append(kv, i32(pos), i32(req), i32(table), view, rope=wide[:, 12:44], rope_positions=i32(rp),
             rope_offset=16, q=q, q_out=qo[:, 8:1032])
    torch.cuda.synchronize()
    assert h.status() == 0
    h.close()
    want = before.copy()
    want[:, 3:67, 16:160] = expected(WIDE, before[:, 3:67, 16:160], kv.float().cpu().numpy(), tab, pos, rp, req,
                                     table, 16, False)
    assert np.array_equal(pool.cpu().numpy(), want)
    f32 = torch.from_numpy(ro.rotate(q.float().cpu().numpy(), tab, rp, 64, 16, False, dtype=np.float32))
    assert torch.equal(qo[:, 8:1032].cpu(), f32.to(torch.bfloat16))
    assert not qo[:, :8].any() and not qo[:, 1032:].any()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("heads", [1, 3, 17, 64, 131])
def test_rotate_there_and_back(layout, heads):
    m = _m()
    spec = LAYOUTS[layout]
    dh, rows = spec["head_dim"], 13
    h = m.Cache(spec, 1, 1)
    rng = np.random.default_rng(heads)
    pos = rng.integers(0, 4000, rows)
    pos[[2, 7]] = -1
    for dtype, dim, off, inter in (("f32", 16, 8, True), ("bf16", 64, 0, False), ("f16", 48, 16, False),
                                   ("f32", 64, 0, False)):
        tab = ro.table(4000, dim)
        x = torch.from_numpy(rng.standard_normal((rows, heads * dh)).astype(np.float32)).to(DTYPES[dtype])
        for inverse in (False, True):
            xd, out = x.cuda(), torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
            td = torch.from_numpy(tab).cuda()
            h.rotate(xd, out, i32(pos), td, rope_offset=off, interleaved=inter, inverse=inverse)
            h.rotate(xd, xd, i32(pos), td, rope_offset=off, interleaved=inter, inverse=inverse)
            want = torch.from_numpy(ro.rotate(x.float().numpy(), tab, pos, dh, off, inter, inverse,
                                              dtype=np.float32)).to(x.dtype)
            assert torch.equal(xd.cpu(), want)
            want[torch.from_numpy(pos) < 0] = 7.0
            assert torch.equal(out.cpu(), want)
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("layout,heads,rows", [("full", 5, 4001), ("full", 64, 1500), ("wide", 16, 1250),
                                               ("wide", 7, 2777), ("wide", 131, 1300)])
@pytest.mark.parametrize("inter", [False, True])
def test_rotate_many_rows(layout, heads, rows, inter):
    """So many that a thread takes several heads, and a CTA several rows."""
    m = _m()
    spec = LAYOUTS[layout]
    h = m.Cache(spec, 1, 1)
    rng = np.random.default_rng(heads)
    pos = rng.integers(-1, 300, rows)
    tab = ro.table(300, 32)
    x = torch.from_numpy(rng.standard_normal((rows, heads * spec["head_dim"])).astype(np.float32)).to(torch.float16)
    xd, out = x.cuda(), torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
    h.rotate(xd, out, i32(pos), torch.from_numpy(tab).cuda(), rope_offset=16, interleaved=inter)
    want = torch.from_numpy(ro.rotate(x.float().numpy(), tab, pos, spec["head_dim"], 16, inter, False,
                                      dtype=np.float32)).to(x.dtype)
    want[torch.from_numpy(pos) < 0] = 7.0
    assert torch.equal(out.cpu(), want)
    assert h.status() == 0
    h.close()


def test_rotate_positions_outside_the_table():
    m = _m()
    h = m.Cache(TINY, 1, 1)
    x = torch.randn((3, 128), device="cuda")
    out = torch.zeros_like(x)
    h.rotate(x, out, i32([10, 9, -1]), torch.ones((10, 32), device="cuda"))
    assert h.status(clear=True) == m.STATUS_POSITION
    assert not out[0].any() and out[1].any() and not out[2].any()
    h.close()


def test_append_and_rotate_captured_and_on_another_stream():
    m = _m()
    h = m.Cache(WIDE, 1, 1)
    g = torch.Generator().manual_seed(4)
    kv = torch.randn((5, 128), generator=g).to(torch.bfloat16).cuda()
    q = torch.randn((5, 1024), generator=g).to(torch.bfloat16).cuda()
    tab = torch.from_numpy(ro.table(300, 64)).cuda()
    pos, req, table = i32([1, 2, 3, 70, 71]), i32([0] * 5), i32([[1, 0]])
    pool, qo, back = torch.zeros((2, 64, 144), dtype=torch.uint8, device="cuda"), torch.zeros_like(q), torch.zeros_like(q)
    stream = torch.cuda.Stream()

    def step(**kw):
        h.append(kv, pos, req, table, pool, rope=tab, q=q, q_out=qo, **kw)
        h.rotate(qo, back, pos, tab, inverse=True, **kw)

    torch.cuda.synchronize()
    step(stream=stream)
    torch.cuda.synchronize()
    eager = [t.clone() for t in (pool, qo, back)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for shift in (0, 100):
        for t in (pool, qo, back):
            t.zero_()
        pos.copy_(i32([1, 2, 3, 70, 71]))
        if shift:
            pos[4] = 127
        graph.replay()
        torch.cuda.synchronize()
        if not shift:
            assert all(torch.equal(a, b) for a, b in zip(eager, (pool, qo, back)))
        else:
            want = ro.rotate(q[4:].float().cpu().numpy(), tab.cpu().numpy(), [127], 64, 0, False, dtype=np.float32)
            assert torch.equal(qo[4:].cpu(), torch.from_numpy(want).to(torch.bfloat16))
            assert pool[0, 63].any() and not pool[0, 7].any()
    h.close()


def test_the_library_refuses():
    """Decided on the host: the addresses are never used."""
    import ctypes as C
    m = _m()
    from moe_decode_layer_mxfp8_gb300 import cache as mc
    h = m.Cache(WIDE, 1, 1)
    lib, a = mc._lib(), 0x10000
    rope = dict(table=a, stride=0, positions=9, dim=32, offset=32, interleaved=0, inverse=0)
    app = dict(kv=a, q=a, q_out=a, positions=a, row_req=a, block_table=a, kv_cache=a, kv_stride_block=64 * 144,
               kv_stride_tok=144, kv_num_blocks=4, dtype=1, rows=3, n_req=2, max_blocks=5)
    rot = dict(x=a, out=a, positions=a, dtype=1, rows=3, heads=2)
    bad_rope = [(dict(dim=0), -2), (dict(dim=24), -2), (dict(dim=80), -2), (dict(offset=4), -2),
                (dict(offset=-8), -2), (dict(offset=40), -2), (dict(stride=16), -1), (dict(stride=34), -4),
                (dict(table=a + 8), -4), (dict(positions=0), -1), (dict(positions=2 ** 31), -1)]
    for change, code in [
            (dict(kv=None), -1), (dict(positions=None), -1), (dict(row_req=None), -1), (dict(block_table=None), -1),
            (dict(kv_cache=None), -1), (dict(q_out=None), -1), (dict(q=None), -1), (dict(rows=0), -1),
            (dict(n_req=0), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(rows=2 ** 30 + 1), -3),
            (dict(kv=a + 8), -4), (dict(kv_stride=127), -1), (dict(kv_stride=132), -4), (dict(q=a + 2), -4),
            (dict(q_stride=1032), -1), (dict(q_out_stride=1028), -4), (dict(positions=a + 2), -4),
            (dict(rope_positions=a + 1), -4), (dict(kv_cache=a + 8), -4), (dict(kv_stride_tok=128), -5),
            (dict(kv_stride_block=63 * 144), -5), (dict(kv_num_blocks=0), -1), (dict(max_blocks=0), -1),
            (dict(max_blocks=2 ** 25), -1)]:
        args = mc.AppendArgs(**dict(app, **change), rope=mc.Rope(**rope))
        assert lib.mono_cache_append(h._h, C.byref(args), None) == code, change
    for change, code in [
            (dict(x=None), -1), (dict(out=None), -1), (dict(positions=None), -1), (dict(rows=0), -1), (dict(heads=0), -1),
            (dict(heads=2 ** 20 + 1), -2), (dict(dtype=4), -1), (dict(x=a + 8), -4), (dict(out=a + 4), -4),
            (dict(x_stride=136), -1), (dict(x_stride=127), -1), (dict(out_stride=132), -4), (dict(positions=a + 2), -4)]:
        args = mc.RotateArgs(**dict(rot, **change), rope=mc.Rope(**rope))
        assert lib.mono_cache_rotate(h._h, C.byref(args), None) == code, change
    for change, code in bad_rope:
        args = mc.RotateArgs(**rot, rope=mc.Rope(**dict(rope, **change)))
        assert lib.mono_cache_rotate(h._h, C.byref(args), None) == code, change
        args = mc.AppendArgs(**app, rope=mc.Rope(**dict(rope, **change)))
        assert lib.mono_cache_append(h._h, C.byref(args), None) == code, change
    args = mc.AppendArgs(**app, rope=mc.Rope())  # queries without a rotation
    assert lib.mono_cache_append(h._h, C.byref(args), None) == -1
    args = mc.RotateArgs(**rot, rope=mc.Rope())
    assert lib.mono_cache_rotate(h._h, C.byref(args), None) == -1
    torch.cuda.synchronize()
    assert h.status() == 0
    h.close()
    with pytest.raises(ValueError):
        h.rotate(torch.zeros((1, 64), device="cuda"), torch.zeros((1, 64), device="cuda"), i32([0]),
                 torch.zeros((1, 32), device="cuda"))
