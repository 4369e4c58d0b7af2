"""Operators that fill a layer's paged cache and read a prefix in common, as cases to be measured.

They stand next to the decode layer's own insert and to the attention over its cache (records of
kv_dim e4m3 codes and one f32 scale, the latent being key and value at once):

* ``append``   rotating the rows' latents by their positions and storing them as records; the
               rows' queries may be rotated in the same call;
* ``rotate``   rotating heads by their rows' positions, forwards (queries) or back (an attention's
               output, since the values carry the rotation too);
* ``shared``   attention of the rows over a prefix that many requests share, and their own tokens.

With ``own`` false, ``run`` is the plain form: elementary torch operations in 32 bits.  With
``own`` true it calls the framework.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

# Cache layouts: the full-size layer, the narrow 64-wide one, small 16-token pages, one latent.
LAYOUTS = {
    "full": dict(n_q_heads=64, head_dim=128, kv_dim=512, block_size=128, kv_record_bytes=528),
    "wide": dict(n_q_heads=16, head_dim=64, kv_dim=128, block_size=64, kv_record_bytes=144),
    "small": dict(n_q_heads=8, head_dim=64, kv_dim=128, block_size=16, kv_record_bytes=144),
    "tiny": dict(n_q_heads=4, head_dim=64, kv_dim=64, block_size=16, kv_record_bytes=80),
}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token: latent and queries rotated, one record; pure latency
        dict(name="append_one", op="append", layout="full", n_req=1, rows_lo=1, rows_hi=1,
             ctx_hi=8192, shift=0, pad=0, rope=64, last=True, interleaved=True, dtype="bf16",
             queries=True),
        # the largest decode step: eight requests with five drafts each, some padding, caches that
        # an eviction has shortened (their rotary positions run ahead of their slots)
        dict(name="append_step", op="append", layout="full", n_req=8, rows_lo=6, rows_hi=6,
             ctx_hi=32768, shift=20000, pad=3, rope=64, last=True, interleaved=True, dtype="bf16",
             queries=True),
        # prompts of several requests at once, from a few tokens to many thousand
        dict(name="append_prompts", op="append", layout="full", n_req=5, rows_lo=17, rows_hi=8192,
             ctx_hi=1024, shift=0, pad=0, rope=64, last=True, interleaved=False, dtype="bf16",
             queries=True),
        # a narrow model's prompts in 32 bits, whole heads rotated, ragged, no queries
        dict(name="append_narrow", op="append", layout="wide", n_req=7, rows_lo=301, rows_hi=4099,
             ctx_hi=1, shift=0, pad=5, rope=64, last=True, interleaved=False, dtype="f32",
             queries=False),
        # a step's attention output turned back by the rows' positions
        dict(name="rotate_back", op="rotate", layout="full", heads=64, rows=48, pos_hi=65536, pad=2,
             rope=64, last=True, interleaved=True, dtype="bf16", inverse=True),
        # a long prompt's queries of a narrow model
        dict(name="rotate_prompt", op="rotate", layout="wide", heads=16, rows=20001, pos_hi=20001,
             pad=0, rope=32, last=False, interleaved=False, dtype="f16", inverse=False),
        # one question to a short instruction
        dict(name="shared_one", op="shared", layout="full", n_req=1, rows=1, prefixes=1, solo=0,
             prefix=777, own_lo=50, own_hi=50, causal=True),
        # eight requests decoding behind one long document
        dict(name="shared_decode", op="shared", layout="full", n_req=8, rows=1, prefixes=1, solo=0,
             prefix=32768, own_lo=64, own_hi=2048, causal=True),
        # the same with five drafts each: the largest step
        dict(name="shared_drafts", op="shared", layout="full", n_req=8, rows=6, prefixes=1, solo=0,
             prefix=32768, own_lo=64, own_hi=2048, causal=True),
        # a large server behind one instruction that ends inside a page
        dict(name="shared_batch", op="shared", layout="full", n_req=256, rows=1, prefixes=1, solo=0,
             prefix=8001, own_lo=1, own_hi=1024, causal=True),
        # a narrow model, three instructions and requests without one, odd lengths
        dict(name="shared_narrow", op="shared", layout="wide", n_req=33, rows=3, prefixes=3, solo=4,
             prefix=4099, own_lo=1, own_hi=1500, causal=True),
        # small pages, draft rows that all see up to the last one
        dict(name="shared_small", op="shared", layout="small", n_req=5, rows=5, prefixes=1, solo=0,
             prefix=3001, own_lo=1, own_hi=333, causal=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rotate", "shared", "shared"])
    layout = rng.choice(["full", "full", "wide", "small", "tiny"])
    lay = LAYOUTS[layout]
    rot = dict(rope=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= lay["head_dim"]]),
               last=rng.random() < 0.7, interleaved=rng.random() < 0.5,
               dtype=rng.choice(sorted(DTYPES)))
    if op == "append":
        n_req = _log_int(rng, 1, 16)
        queries = rng.random() < 0.6
        hi = _log_int(rng, 1, (8192 if rot["dtype"] != "f32" else 4096) // n_req)
        return dict(op=op, layout=layout, n_req=n_req, rows_lo=rng.randint(1, hi), rows_hi=hi,
                    ctx_hi=_log_int(rng, 1, 16384), shift=rng.choice([0, 0, rng.randint(1, 30000)]),
                    pad=rng.randint(0, 5), **rot, queries=queries)
    if op == "rotate":
        rows = _log_int(rng, 1, 20000)
        return dict(op=op, layout=layout, rows=rows,
                    heads=lay["n_q_heads"] if rows < 4000 else rng.randint(1, 16), pos_hi=_log_int(rng, rows, 65536), pad=rng.randint(0, min(3, rows - 1)), **rot,
                    inverse=rng.random() < 0.5)
    n_req = _log_int(rng, 1, 128)
    rows = rng.randint(1, 6 if n_req <= 40 else 2)
    hi = _log_int(rng, 1, 1500 if n_req <= 40 else 700)
    return dict(op=op, layout=layout, n_req=n_req, rows=rows, prefixes=rng.randint(1, min(3, n_req)),
                solo=rng.randint(0, n_req // 4), prefix=_log_int(rng, 1, min(32768, 1500000 // (n_req * rows))),
                own_lo=rng.randint(1, hi), own_hi=hi, causal=rng.random() < 0.7)


def _spread(n, lo, hi):
    """n whole numbers of lo..hi: both ends and a spread between them."""
    if n == 1:
        return [hi]
    frac = [0.0, 1.0] + [((i * 0.6180339887498949) % 1.0) for i in range(1, n - 1)]
    return [lo + int(round(f * (hi - lo))) for f in frac]


def _counts(case):
    """Rows that each request of an append brings, and the tokens it holds before."""
    return (_spread(case["n_req"], case["rows_lo"], case["rows_hi"]),
            _spread(case["n_req"], case["ctx_hi"] // 8, case["ctx_hi"]))


def _lengths(case):
    """Of a shared attention: each prefix's tokens, each request's prefix (-1: none), and the
    tokens of its own, the step's rows among them."""
    pre = _spread(case["prefixes"], max(1, case["prefix"] // 3), case["prefix"])
    of = [-1 if i < case["solo"] else i % case["prefixes"] for i in range(case["n_req"])]
    return pre, of, [o + case["rows"] for o in _spread(case["n_req"], case["own_lo"], case["own_hi"])]


# ------------------------------------------------------------------------------- work
def work(case):
    """Bytes and operations that the operator cannot do without."""
    lay = LAYOUTS[case["layout"]]
    if case["op"] == "rotate":
        live, es = case["rows"] - case["pad"], BYTES[case["dtype"]]
        n = live * case["heads"]
        return {"bytes": 2 * n * lay["head_dim"] * es + min(live, case["pos_hi"]) * case["rope"] * 4,
                "flops": 3 * n * case["rope"]}
    kv, qw = lay["kv_dim"], lay["n_q_heads"] * lay["head_dim"]
    if case["op"] == "append":
        rows, ctx = _counts(case)
        at = set()
        for n, c in zip(rows, ctx):
            at.update(range(c, c + n))
        es, live = BYTES[case["dtype"]], sum(rows)
        heads = kv // lay["head_dim"] + (lay["n_q_heads"] if case["queries"] else 0)
        return {"bytes": live * (kv * es + kv + 4) + len(at) * case["rope"] * 4
                + (2 * live * qw * es if case["queries"] else 0),
                "flops": live * (3 * heads * case["rope"] + 2 * kv)}
    pre, of, mine = _lengths(case)
    n = case["rows"]
    used = {g for g in of if g >= 0}
    tokens = sum(pre[g] for g in used) + sum(mine)
    seen = 0
    for g, m in zip(of, mine):
        seen += n * ((pre[g] if g >= 0 else 0) + m) - (n * (n - 1) // 2 if case["causal"] else 0)
    rows = case["n_req"] * n
    return {"bytes": tokens * (kv + 4) + rows * (4 * qw + 4 * lay["n_q_heads"]), "flops": 4 * seen * qw}


# ---------------------------------------------------------------------------- inputs
def _table(positions, rope, base=10000.0):
    """cos and sin of every position's angles, [positions, rope]: cosines, then sines."""
    f = base ** (-torch.arange(0, rope, 2, dtype=torch.float64, device="cuda") / rope)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).to(torch.float32)


def _records(blocks, lay, gen):
    """A pool of cache records: normed latents quantised to e4m3 under a scale of amax / 448."""
    kv, rec, bs = lay["kv_dim"], lay["kv_record_bytes"], lay["block_size"]
    pool = torch.zeros((blocks, bs, rec), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 18) // bs)
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        v = torch.randn((n, bs, kv), generator=gen, device="cuda")
        sc = v.abs().amax(-1, keepdim=True) / 448.0
        pool[b:b + n, :, :kv] = (v / sc).to(torch.float8_e4m3fn).view(torch.uint8)
        pool[b:b + n, :, kv:kv + 4] = sc.view(torch.uint8)
    return pool


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 29)
    st = dict(case=case, handle=None)
    {"append": _prepare_append, "rotate": _prepare_rotate, "shared": _prepare_shared}[case["op"]](
        case, gen, st)
    torch.cuda.synchronize()
    return st


def _prepare_append(case, gen, st):
    lay, dt = LAYOUTS[case["layout"]], DTYPES[case["dtype"]]
    bs = lay["block_size"]
    rows, ctx = _counts(case)
    per = [(c + n + bs - 1) // bs for n, c in zip(rows, ctx)]
    perm = torch.randperm(sum(per) + 2, generator=gen, device="cuda").to(torch.int32)
    # pages that the rows reach; the tokens before them lie elsewhere and are not touched
    first = [c // bs for c in ctx]
    table = torch.full((case["n_req"], max(per)), -1, dtype=torch.int32, device="cuda")
    used = 0
    for i, (f, n) in enumerate(zip(first, per)):
        table[i, f:n] = perm[used:used + n - f]
        used += n - f
    order = perm[:used].sort().indices.to(torch.int32)  # numbered 0..used - 1, at random
    back = torch.empty_like(order)
    back[order.long()] = torch.arange(used, dtype=torch.int32, device="cuda")
    used = 0
    for i, (f, n) in enumerate(zip(first, per)):
        table[i, f:n] = back[used:used + n - f]
        used += n - f
    live, pad = sum(rows), case["pad"]
    pos = np.concatenate([np.arange(c, c + n) for n, c in zip(rows, ctx)] + [np.full(pad, -1)])
    req = np.concatenate([np.full(n, i) for i, n in enumerate(rows)] + [np.zeros(pad)])
    st.update(layout=lay, live=live, table=table, positions=_i32(pos.astype(np.int32)),
              row_req=_i32(req.astype(np.int32)),
              rope_positions=_i32((pos + case["shift"] * (pos >= 0)).astype(np.int32)),
              rope=_table(int(pos.max()) + 1 + case["shift"], case["rope"]),
              offset=lay["head_dim"] - case["rope"] if case["last"] else 0,
              pool=torch.zeros((used, bs, lay["kv_record_bytes"]), dtype=torch.uint8, device="cuda"),
              kv=torch.randn((live + pad, lay["kv_dim"]), generator=gen, device="cuda").to(dt),
              q=None, q_out=None)
    if case["queries"]:
        qw = lay["n_q_heads"] * lay["head_dim"]
        st["q"] = torch.empty((live + pad, qw), dtype=dt, device="cuda")
        for i in range(0, live + pad, 4096):
            n = min(4096, live + pad - i)
            st["q"][i:i + n] = torch.randn((n, qw), generator=gen, device="cuda").to(dt)
        st["q_out"] = torch.zeros_like(st["q"])
    # what a pass leaves: the records as what their bits stand for (codes, and scales), the queries
    kv = lay["kv_dim"]
    st["left"] = [st["pool"][..., :kv].view(torch.float8_e4m3fn), st["pool"][..., kv:kv + 4].view(torch.float32)]
    if case["queries"]:
        st["left"].append(st["q_out"])
    if own:
        import moe_decode_layer_mxfp8_gb300 as m
        st["handle"] = m.Cache(lay, max_rows=48, max_requests=max(8, case["n_req"]))


def _prepare_rotate(case, gen, st):
    rows, pad = case["rows"], case["pad"]
    pos = torch.randint(0, case["pos_hi"], (rows,), generator=gen, device="cuda").to(torch.int32)
    if rows > 1000:  # a prompt: one position after another
        pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    pos[rows - pad:] = -1
    lay = LAYOUTS[case["layout"]]
    x = torch.randn((rows, case["heads"] * lay["head_dim"]), generator=gen, device="cuda")
    st.update(layout=lay, positions=pos, live=rows - pad, rope=_table(case["pos_hi"], case["rope"]),
              offset=lay["head_dim"] - case["rope"] if case["last"] else 0,
              x=x.to(DTYPES[case["dtype"]]))
    st["out"] = torch.zeros_like(st["x"])
    if own:
        import moe_decode_layer_mxfp8_gb300 as m
        st["handle"] = m.Cache(lay, max_rows=48, max_requests=8)


def _prepare_shared(case, gen, st):
    lay = LAYOUTS[case["layout"]]
    bs, n, n_req = lay["block_size"], case["rows"], case["n_req"]
    pre, of, mine = _lengths(case)
    pages = [(p + bs - 1) // bs for p in pre]
    start = [pre[g] if g >= 0 else 0 for g in of]
    end = [(s + m + bs - 1) // bs for s, m in zip(start, mine)]
    total = sum(pages) + sum(e - s // bs for s, e in zip(start, end)) + 2
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    prefix_table = torch.zeros((len(pre), max(pages)), dtype=torch.int32, device="cuda")
    table = torch.zeros((n_req, max(end)), dtype=torch.int32, device="cuda")
    used = 0
    for g, k in enumerate(pages):
        prefix_table[g, :k] = perm[used:used + k]
        used += k
    # every request's table is that of its whole context: the prefix's whole pages, then its own
    for i, (s, e) in enumerate(zip(start, end)):
        f = s // bs
        if f:
            table[i, :f] = prefix_table[of[i], :f]
        table[i, f:e] = perm[used:used + e - f]
        used += e - f
    qw = lay["n_q_heads"] * lay["head_dim"]
    # queries that pick some tokens out: scores spread by about 1.5
    q = torch.randn((n_req * n, qw), generator=gen, device="cuda").mul_(1.5).to(torch.bfloat16)
    st.update(layout=lay, pre=pre, prefix_table=prefix_table, table=table,
              members=[torch.tensor([i for i in range(n_req) if of[i] == g], device="cuda")
                       for g in range(len(pre))],
              longest=max(mine), start=torch.tensor(start, device="cuda"), prefix_of=_i32(of),
              prefix_lengths=_i32(pre), pool=_records(total, lay, gen), q=q,
              positions=_i32([s + m - n + j for s, m in zip(start, mine) for j in range(n)]),
              row_req=torch.arange(n_req, dtype=torch.int32, device="cuda").repeat_interleave(n),
              o=torch.zeros_like(q), lse=torch.zeros((n_req * n, lay["n_q_heads"]), device="cuda"))
    if own:
        import moe_decode_layer_mxfp8_gb300 as m
        st["handle"] = m.Cache(lay, max_rows=n_req * n, max_requests=n_req)


# ------------------------------------------------------------------------------- run
def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _append_own, "rotate": _rotate_own, "shared": _shared_own}[op](st)
    return {"append": _append_plain, "rotate": _rotate_plain, "shared": _shared_plain}[op](st)


def _append_own(st):
    case = st["case"]
    st["handle"].append(st["kv"], st["positions"], st["row_req"], st["table"], st["pool"],
                        rope=st["rope"], rope_offset=st["offset"], interleaved=case["interleaved"],
                        rope_positions=st["rope_positions"], q=st["q"], q_out=st["q_out"])
    return st["left"]


def _rotate_own(st):
    case = st["case"]
    st["handle"].rotate(st["x"], st["out"], st["positions"], st["rope"], rope_offset=st["offset"],
                        interleaved=case["interleaved"], inverse=case["inverse"])
    return [st["out"]]


def _shared_own(st):
    st["handle"].attend_shared(st["q"], st["o"], st["positions"], st["row_req"], st["table"],
                               st["pool"], st["prefix_table"], st["prefix_lengths"],
                               prefix_of=st["prefix_of"], causal=st["case"]["causal"], lse=st["lse"])
    return [st["o"], st["lse"]]


# ------------------------------------------------------------------- the plain forms
def _turn(x, table, positions, head_dim, offset, interleaved, inverse):
    """x (rows of heads) rotated by its rows' positions, in 32 bits."""
    rope = table.shape[1]
    y = x.to(torch.float32).view(x.shape[0], -1, head_dim).clone()
    cs = table[positions.long()][:, None, :]
    c, s = cs[..., :rope // 2], cs[..., rope // 2:]
    if inverse:
        s = -s
    part = y[..., offset:offset + rope]
    if interleaved:
        a, b = part[..., 0::2].clone(), part[..., 1::2].clone()
        part[..., 0::2] = a * c - b * s
        part[..., 1::2] = b * c + a * s
    else:
        a, b = part[..., :rope // 2].clone(), part[..., rope // 2:].clone()
        part[..., :rope // 2] = a * c - b * s
        part[..., rope // 2:] = b * c + a * s
    return y.view(x.shape)


def _append_plain(st):
    case, lay, live = st["case"], st["layout"], st["live"]
    kv, bs = lay["kv_dim"], lay["block_size"]
    at = st["rope_positions"][:live]
    y = _turn(st["kv"][:live], st["rope"], at, lay["head_dim"], st["offset"], case["interleaved"], False)
    amax = y.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (y / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    p = st["positions"][:live].long()
    page = st["table"][st["row_req"][:live].long(), p // bs].long()
    st["pool"][page, p % bs, :kv] = codes.view(torch.uint8)
    st["pool"][page, p % bs, kv:kv + 4] = scale.view(torch.uint8)
    if st["q"] is not None:
        q = _turn(st["q"][:live], st["rope"], at, lay["head_dim"], st["offset"], case["interleaved"], False)
        st["q_out"][:live] = q.to(st["q"].dtype)
    return st["left"]


def _rotate_plain(st):
    case, live = st["case"], st["live"]
    y = _turn(st["x"][:live], st["rope"], st["positions"][:live],
              st["layout"]["head_dim"], st["offset"], case["interleaved"], case["inverse"])
    st["out"][:live] = y.to(st["x"].dtype)
    return [st["out"]]


def _keys(rec, lay):
    """Records (any leading sizes) as f32 [..., slices, head_dim]."""
    kv = lay["kv_dim"]
    k = rec[..., :kv].view(torch.float8_e4m3fn).to(torch.float32)
    k = k * rec[..., kv:kv + 4].contiguous().view(torch.float32)
    return k.view(*k.shape[:-1], kv // lay["head_dim"], lay["head_dim"])


def _part(s, v, pattern):
    """A part of a softmax over the last axis: its maximum, its sum and its weighted values."""
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(s - m)
    return m, p.sum(-1, keepdim=True), torch.einsum(pattern, p, v)


def _shared_plain(st):
    case, lay = st["case"], st["layout"]
    bs, dh, nq = lay["block_size"], lay["head_dim"], lay["n_q_heads"]
    g, n, n_req = lay["kv_dim"] // dh, case["rows"], case["n_req"]
    q = st["q"].to(torch.float32).view(n_req, n, g, nq // g, dh) * (1.0 / math.sqrt(dh))
    hi = st["positions"].long().view(n_req, n, 1)
    if not case["causal"]:
        hi = hi.amax(1, keepdim=True).expand(n_req, n, 1)
    # their own tokens, padded to the longest
    t = st["start"][:, None] + torch.arange(st["longest"], device="cuda")
    page = torch.gather(st["table"].long(), 1, (t // bs).clamp_max(st["table"].shape[1] - 1))
    keys = _keys(st["pool"][page, t % bs], lay)
    s = torch.einsum("bnghd,btgd->bnght", q, keys)
    s = torch.where((t[:, None, :] <= hi)[:, :, None, None, :], s, torch.full_like(s, float("-inf")))
    m, l, o = _part(s, keys, "bnght,btgd->bnghd")
    for i, who in enumerate(st["members"]):  # each prefix once, for all of its requests
        if not who.numel():
            continue
        t = torch.arange(st["pre"][i], device="cuda")
        keys = _keys(st["pool"][st["prefix_table"][i, t // bs].long(), t % bs], lay)
        m1, l1, o1 = _part(torch.einsum("bnghd,tgd->bnght", q[who], keys), keys, "bnght,tgd->bnghd")
        top = torch.maximum(m[who], m1)
        a, b = torch.exp(m[who] - top), torch.exp(m1 - top)
        m[who], l[who], o[who] = top, l[who] * a + l1 * b, o[who] * a + o1 * b
    st["o"].copy_((o / l).reshape(n_req * n, nq * dh))
    st["lse"].copy_((m + torch.log(l)).reshape(n_req * n, nq))
    return [st["o"], st["lse"]]


# ------------------------------------------------------------------------------ exact
def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _append_exact, "rotate": _rotate_exact, "shared": _shared_exact}[case["op"]](st)


def _complex(x, st, positions, head_dim, inverse):
    """Rotation as a product of complex numbers, in 64 bits, from the table's entries."""
    case, rope, off = st["case"], st["rope"].shape[1], st["offset"]
    y = x.double().reshape(x.shape[0], -1, head_dim)
    e = st["rope"][positions.long()].double()
    turn = torch.complex(e[:, :rope // 2], e[:, rope // 2:] * (-1.0 if inverse else 1.0))[:, None, :]
    idx = torch.arange(rope // 2, device="cuda")
    one = off + (2 * idx if case["interleaved"] else idx)
    two = one + (1 if case["interleaved"] else rope // 2)
    z = torch.complex(y[..., one], y[..., two]) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y.reshape(x.shape)


def _append_exact(st):
    lay, live = st["layout"], st["live"]
    bs, at = lay["block_size"], st["rope_positions"][:live]
    y = _complex(st["kv"][:live], st, at, lay["head_dim"], False)
    scale = y.abs().max(-1).values / 448.0
    scale[scale == 0] = 1.0
    shape = tuple(st["pool"].shape[:2])
    codes = torch.zeros((shape[0] * shape[1], lay["kv_dim"]), dtype=torch.float64, device="cuda")
    scales = torch.zeros((shape[0] * shape[1], 1), dtype=torch.float64, device="cuda")
    p, b = st["positions"][:live].long(), st["row_req"][:live].long()
    slot = st["table"][b, torch.div(p, bs, rounding_mode="floor")].long() * bs + p % bs
    codes[slot] = y / scale[:, None]  # (before they are rounded to what 8 bits hold)
    scales[slot] = scale[:, None]
    out = [codes.view(*shape, -1), scales.view(*shape, 1)]
    if st["q"] is not None:
        rot = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        for i in range(0, live, 4096):
            j = min(live, i + 4096)
            rot[i:j] = _complex(st["q"][i:j], st, at[i:j], lay["head_dim"], False)
        out.append(rot)
    return out


def _rotate_exact(st):
    out = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
    live = st["live"]
    out[:live] = _complex(st["x"][:live], st, st["positions"][:live],
                          st["layout"]["head_dim"], st["case"]["inverse"])
    return [out]


def _e4m3_table():
    """The 256 values of e4m3 (bias 7, no infinities; 0x7F and 0xFF are NaN)."""
    out = []
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        if (b & 127) == 127:
            v = float("nan")
        out.append(-v if b & 128 else v)
    return out


def _shared_exact(st):
    """Request by request over its whole context in 64 bits, from the stored bits."""
    case, lay = st["case"], st["layout"]
    kv, bs, dh, nq = lay["kv_dim"], lay["block_size"], lay["head_dim"], lay["n_q_heads"]
    per, n = nq // (kv // dh), case["rows"]
    lut = torch.tensor(_e4m3_table(), dtype=torch.float64, device="cuda")
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    pre, of, mine = _lengths(case)
    for i in range(case["n_req"]):
        first = pre[of[i]] if of[i] >= 0 else 0
        t = torch.arange(first + mine[i], device="cuda")
        page = st["table"][i, torch.div(t, bs, rounding_mode="floor")].long()
        if first:
            u = t[:first]
            page[:first] = st["prefix_table"][of[i], torch.div(u, bs, rounding_mode="floor")].long()
        rec = st["pool"][page, t % bs]
        scale = rec[:, kv:kv + 4].contiguous().view(torch.float32).double()
        last = first + mine[i] - 1
        sees = torch.tensor([last if not case["causal"] else last - n + 1 + j for j in range(n)],
                            device="cuda")
        late = (t[None, :] > sees[:, None]).repeat_interleave(per, 0)
        rows = slice(i * n, (i + 1) * n)
        for sl in range(kv // dh):
            z = lut[rec[:, sl * dh:(sl + 1) * dh].long()] * scale
            heads = slice(sl * per, (sl + 1) * per)
            q = st["q"][rows].double().view(n, nq, dh)[:, heads].reshape(n * per, dh)
            s = (q @ z.T / math.sqrt(dh)).masked_fill(late, float("-inf"))
            norm = torch.logsumexp(s, -1)
            o[rows].view(n, nq, dh)[:, heads] = (torch.exp(s - norm[:, None]) @ z).view(n, per, dh)
            lse[rows, heads] = norm.view(n, per)
    return [o, lse]
