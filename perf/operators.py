"""The cache and draft operators of a serving loop, as cases to be measured.

Four operators that stand next to the decode layer, on its own paged cache (records of kv_dim
e4m3 codes and one f32 scale, the latent being key and value at once):

* ``attend``   attention of the step's rows over their requests' whole cached context;
* ``window``   the same with a sliding window and a few first tokens that stay visible;
* ``evict``    keeping the cached tokens that gathered most attention weight (which the
               attention adds up where a case says ``weigh``);
* ``verify``   verification of drafted tokens against the target's probabilities.

With ``own`` false, ``run`` is the plain form: elementary torch operations in 32 bits (64 for
running sums and comparisons next to a border).  With ``own`` true it calls the framework.
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


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # one request, one new token, a short conversation: the latency of a single user
        dict(name="attend_one_short", op="attend", layout="full", n_req=1, rows=1, ctx_lo=777,
             ctx_hi=777, window=0, sinks=0, causal=True, weigh=False),
        # eight requests decoding one token each over contexts from short to long
        dict(name="attend_decode", op="attend", layout="full", n_req=8, rows=1, ctx_lo=1024,
             ctx_hi=65536, window=0, sinks=0, causal=True, weigh=False),
        # the largest step: eight requests with five speculative drafts each, long contexts
        dict(name="attend_drafts", op="attend", layout="full", n_req=8, rows=6, ctx_lo=1024,
             ctx_hi=65536, window=0, sinks=0, causal=True, weigh=False),
        # a full server of short contexts on the narrow layer, odd lengths, ragged pages
        dict(name="attend_many_narrow", op="attend", layout="wide", n_req=33, rows=3, ctx_lo=1,
             ctx_hi=4099, window=0, sinks=0, causal=True, weigh=False),
        # a streaming layer: 4096-token window with four first tokens, drafts in flight
        dict(name="window_drafts", op="window", layout="full", n_req=8, rows=6, ctx_lo=1024,
             ctx_hi=65536, window=4096, sinks=4, causal=True, weigh=False),
        # one streaming user on small pages, a window that starts inside a page; draft rows that
        # all see up to the last one
        dict(name="window_one", op="window", layout="small", n_req=1, rows=5, ctx_lo=3001,
             ctx_hi=3001, window=1000, sinks=3, causal=False, weigh=False),
        # a step that also gathers each token's weight, ahead of an eviction
        dict(name="attend_weigh", op="attend", layout="full", n_req=8, rows=1, ctx_lo=1024,
             ctx_hi=32768, window=0, sinks=0, causal=True, weigh=True),
        # halving the caches of a full batch of long contexts
        dict(name="evict_long", op="evict", layout="full", n_req=8, ctx_lo=33000, ctx_hi=65536,
             budget=32768, sinks=4, recent=512),
        # trimming a few mid-length caches; one is already below the budget
        dict(name="evict_short", op="evict", layout="wide", n_req=3, ctx_lo=500, ctx_hi=5003,
             budget=1021, sinks=1, recent=64),
        # the step's verification: eight requests, five drafts, float32 probabilities
        dict(name="verify_step", op="verify", n_req=8, drafts=5, vocab=131072, dtype="f32",
             probs=True, greedy=False),
        # a large batch, bf16 probabilities, an odd vocabulary, some greedy requests
        dict(name="verify_batch", op="verify", n_req=192, drafts=3, vocab=100003, dtype="bf16",
             probs=True, greedy=True),
        # drafts from a table (no draft probabilities), small vocabulary: pure latency
        dict(name="verify_table", op="verify", n_req=4, drafts=2, vocab=32000, dtype="f16",
             probs=False, greedy=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "window", "evict", "verify"])
    if op == "verify":
        n_req = _log_int(rng, 1, 192)
        return dict(op=op, n_req=n_req, drafts=rng.randint(1, 8),
                    vocab=_log_int(rng, 1000, 131072 if n_req <= 64 else 100003),
                    dtype=rng.choice(sorted(DTYPES)), probs=rng.random() < 0.7,
                    greedy=rng.random() < 0.4)
    layout = rng.choice(["full", "full", "wide", "small", "tiny"])
    if op == "evict":
        n_req = _log_int(rng, 1, 8 if layout == "full" else 32)
        hi = _log_int(rng, 64, 65536)
        budget = rng.randint(max(1, hi // 8), max(1, hi - hi // 8))
        sinks = rng.randint(0, min(8, budget))
        return dict(op=op, layout=layout, n_req=n_req, ctx_lo=rng.randint(1, hi), ctx_hi=hi,
                    budget=budget, sinks=sinks, recent=rng.randint(0, (budget - sinks) // 2))
    n_req = _log_int(rng, 1, 8 if layout == "full" else 40)
    hi = _log_int(rng, 1, 65536 if n_req <= 8 else 16384)
    window = _log_int(rng, 1, 8192) if op == "window" else 0
    return dict(op=op, layout=layout, n_req=n_req, rows=rng.randint(1, 6),
                ctx_lo=rng.randint(1, hi), ctx_hi=hi, window=window,
                sinks=rng.randint(0, 8) if op == "window" else 0, causal=rng.random() < 0.7,
                weigh=rng.random() < 0.4)


def _contexts(case):
    """Tokens cached per request before the step: the two ends of the range and a spread."""
    n, lo, hi = case["n_req"], case["ctx_lo"], case["ctx_hi"]
    if n == 1:
        return [hi]
    frac = [0.0, 1.0] + [((i * 0.6180339887498949) % 1.0) for i in range(1, n - 1)]
    return [lo + int(round(f * (hi - lo))) for f in frac]


# ------------------------------------------------------------------------------- work
def _spans(case):
    """Per request: (tokens some row sees, tokens summed over its rows)."""
    n, w, s = case["rows"], case["window"], case["sinks"]
    out = []
    for c in _contexts(case):
        last = c + n - 1
        union = set_sum = 0
        for i in range(n):
            hi = c + i if case["causal"] else last
            seen = hi + 1 if w == 0 else min(hi + 1, w) + max(0, min(s, hi + 1 - w))
            set_sum += seen
        lo_first = 0 if w == 0 else max(0, (c if case["causal"] else last) - w + 1)
        union = last + 1 - lo_first + min(s, lo_first)
        out.append((union, set_sum))
    return out


def work(case):
    """Bytes and operations that the operator cannot do without."""
    if case["op"] == "verify":
        es = 4 if case["dtype"] == "f32" else 2
        rows = case["n_req"] * (2 if case["probs"] else 1)  # the row(s) the token is drawn from
        return {"bytes": rows * case["vocab"] * es + case["n_req"] * case["drafts"] * 20,
                "flops": 2 * rows * case["vocab"]}
    lay = LAYOUTS[case["layout"]]
    rec = lay["kv_dim"] + 4
    if case["op"] == "evict":
        ctx = _contexts(case)
        kept = sum(min(c, case["budget"]) for c in ctx)
        return {"bytes": 4 * sum(ctx) + kept * (2 * rec + 8), "flops": sum(ctx)}
    spans = _spans(case)
    qw = lay["n_q_heads"] * lay["head_dim"]
    rows = case["n_req"] * case["rows"]
    b = sum(u for u, _ in spans) * rec + rows * (qw * 4 + lay["n_q_heads"] * 4)
    if case["weigh"]:
        b += 8 * sum(u for u, _ in spans)
    return {"bytes": b, "flops": 4 * sum(t for _, t in spans) * qw}


# ---------------------------------------------------------------------------- inputs
def _pages(lengths, bs, gen, extra=2):
    """A block table over a random permutation of physical pages, and their number."""
    per = [(n + bs - 1) // bs for n in lengths]
    total = sum(per) + extra
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(per), max(per)), dtype=torch.int32, device="cuda")
    o = 0
    for i, n in enumerate(per):
        table[i, :n] = perm[o:o + n]
        o += n
    return table, total


def _records(blocks, lay, gen):
    """A pool of cache records as the layer's insert stores them: normed latents quantised to
    e4m3 under a scale of amax / 448."""
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    st = dict(case=case, handle=None)
    if case["op"] == "verify":
        _prepare_verify(case, gen, st)
        return st
    lay = LAYOUTS[case["layout"]]
    ctx = _contexts(case)
    n_req = case["n_req"]
    st["layout"] = lay
    if case["op"] == "evict":
        st["table"], blocks = _pages(ctx, lay["block_size"], gen)
        st["pool"] = _records(blocks, lay, gen)
        st["dst_table"], dblocks = _pages([min(c, case["budget"]) for c in ctx],
                                          lay["block_size"], gen)
        st["dst_pool"] = torch.zeros((dblocks, *st["pool"].shape[1:]), dtype=torch.uint8,
                                     device="cuda")
        # weights as attention gathers them: mostly small, a long tail of heavy tokens
        acc = torch.randn((n_req, max(ctx)), generator=gen, device="cuda").mul_(2.0).exp_()
        st["acc"] = acc
        st["lengths"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        st["kept"] = torch.full((n_req, case["budget"]), -1, dtype=torch.int32, device="cuda")
        st["new_lengths"] = torch.zeros(n_req, dtype=torch.int32, device="cuda")
        st["acc_out"] = torch.zeros((n_req, case["budget"]), device="cuda")
        rows = 1
    else:
        rows = case["rows"]
        total = [c + rows for c in ctx]
        st["table"], blocks = _pages(total, lay["block_size"], gen)
        st["pool"] = _records(blocks, lay, gen)
        qw = lay["n_q_heads"] * lay["head_dim"]
        # queries that pick some tokens out: scores spread by about 1.5
        q = torch.randn((n_req * rows, qw), generator=gen, device="cuda").mul_(1.5)
        st["q"] = q.to(torch.bfloat16)
        st["positions"] = torch.tensor([c + i for c in ctx for i in range(rows)],
                                       dtype=torch.int32, device="cuda")
        st["row_req"] = torch.arange(n_req, dtype=torch.int32,
                                     device="cuda").repeat_interleave(rows)
        st["o"] = torch.zeros((n_req * rows, qw), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros((n_req * rows, lay["n_q_heads"]), device="cuda")
        if case["weigh"]:  # what earlier steps have gathered
            st["acc"] = torch.rand((n_req, max(total)), generator=gen, device="cuda")
    if own:
        import moe_decode_layer_mxfp8_gb300 as m
        st["handle"] = m.Cache(lay, max_rows=n_req * rows, max_requests=n_req)
    torch.cuda.synchronize()
    return st


def _prepare_verify(case, gen, st):
    n, k, v = case["n_req"], case["drafts"], case["vocab"]
    # ragged: request i brings 0..k drafts (at least one request brings all of them)
    counts = [k if i % 3 == 0 else (k - i % (k + 1)) for i in range(n)]
    starts = np.concatenate([[0], np.cumsum([c + 1 for c in counts])])
    rows = int(starts[-1])
    dt = DTYPES[case["dtype"]]
    target = torch.empty((rows, v), dtype=dt, device="cuda")
    draft = torch.empty((rows, v), dtype=dt, device="cuda") if case["probs"] else None
    tokens = torch.empty(rows, dtype=torch.int32, device="cuda")
    for r in range(rows):  # a draft model that mostly agrees with the target
        logits = torch.randn(v, generator=gen, device="cuda").mul_(2.0)
        peak = torch.randint(0, v, (8,), generator=gen, device="cuda")
        logits[peak] += 12.0
        target[r] = torch.softmax(logits, 0).to(dt)
        logits += torch.randn(v, generator=gen, device="cuda").mul_(0.3)
        d = torch.softmax(logits, 0)
        tokens[r] = torch.multinomial(d, 1, generator=gen)[0].to(torch.int32)
        if draft is not None:
            draft[r] = d.to(dt)
    st.update(target=target, draft=draft, tokens_in=tokens,
              row_start=torch.tensor(starts, dtype=torch.int32, device="cuda"),
              u=torch.rand(rows, generator=gen, device="cuda"),
              r=torch.rand(n, generator=gen, device="cuda"),
              greedy=(torch.arange(n, device="cuda") % 4 == 1).to(torch.int32)
              if case["greedy"] else None,
              accepted=torch.zeros(n, dtype=torch.int32, device="cuda"),
              tokens=torch.zeros(rows, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------------------- run
def run(st):
    case = st["case"]
    if case["op"] == "verify":
        return _verify_own(st) if own else _verify_plain(st)
    if case["op"] == "evict":
        return _evict_own(st) if own else _evict_plain(st)
    return _attend_own(st) if own else _attend_plain(st)


def _attend_own(st):
    case = st["case"]
    acc = st["acc"].clone() if case["weigh"] else None
    st["handle"].attend(st["q"], st["o"], st["positions"], st["row_req"], st["table"], st["pool"],
                        window=case["window"], sinks=case["sinks"], causal=case["causal"],
                        lse=st["lse"], weights=acc)
    out = [st["o"], st["lse"]]
    return out if acc is None else out + [acc]


def _evict_own(st):
    case = st["case"]
    st["handle"].evict(st["acc"], st["lengths"], st["table"], st["pool"], st["kept"],
                       st["new_lengths"], budget=case["budget"], sinks=case["sinks"],
                       recent=case["recent"], weights_out=st["acc_out"],
                       dst_table=st["dst_table"], dst_cache=st["dst_pool"])
    return [st["kept"], st["new_lengths"], st["acc_out"], st["dst_pool"]]


def _verify_own(st):
    import moe_decode_layer_mxfp8_gb300 as m
    m.verify_drafts(st["target"], st["draft"], st["tokens_in"], st["row_start"], st["u"], st["r"],
                    st["accepted"], st["tokens"], greedy=st["greedy"])
    return [st["accepted"], st["tokens"]]


# ------------------------------------------------------------------- the plain forms
def _attend_plain(st):
    case, lay = st["case"], st["layout"]
    kv, bs, dh, nq = lay["kv_dim"], lay["block_size"], lay["head_dim"], lay["n_q_heads"]
    g, n = kv // dh, case["rows"]
    acc = st["acc"].clone() if case["weigh"] else None
    for i, c in enumerate(_contexts(case)):
        last = c + n - 1
        first = 0
        if case["window"]:
            first = max(0, (c if case["causal"] else last) - case["window"] + 1)
        t = torch.arange(first, last + 1, device="cuda")
        if case["sinks"] and first:
            t = torch.cat([torch.arange(0, min(case["sinks"], first), device="cuda"), t])
        rec = st["pool"][st["table"][i, t // bs].long(), t % bs]
        keys = rec[:, :kv].view(torch.float8_e4m3fn).to(torch.float32)
        keys = keys * rec[:, kv:kv + 4].contiguous().view(torch.float32)
        keys = keys.view(-1, g, dh)
        q = st["q"][i * n:(i + 1) * n].to(torch.float32).view(n, g, nq // g, dh)
        s = torch.einsum("nghd,tgd->nght", q, keys) * (1.0 / math.sqrt(dh))
        hi = st["positions"][i * n:(i + 1) * n].long().view(n, 1)
        if not case["causal"]:
            hi = hi.amax().expand(n, 1)
        seen = t <= hi
        if case["window"]:
            seen = seen & ((t > hi - case["window"]) | (t < case["sinks"]))
        s = torch.where(seen[:, None, None, :], s, torch.full_like(s, float("-inf")))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        p = p / l
        o = torch.einsum("nght,tgd->nghd", p, keys)
        st["o"][i * n:(i + 1) * n] = o.reshape(n, nq * dh).to(torch.bfloat16)
        st["lse"][i * n:(i + 1) * n] = (m + torch.log(l)).view(n, nq)
        if acc is not None:
            acc[i, t] += p.sum((0, 1, 2))
    out = [st["o"], st["lse"]]
    return out if acc is None else out + [acc]


def _evict_plain(st):
    case, bs = st["case"], st["layout"]["block_size"]
    budget, sinks, recent = case["budget"], case["sinks"], case["recent"]
    rb = st["layout"]["kv_dim"] + 4
    for i, c in enumerate(_contexts(case)):
        if c <= budget:
            kept = torch.arange(c, device="cuda")
        else:
            w = st["acc"][i, sinks:c - recent]
            order = torch.sort(w, descending=True, stable=True).indices
            mid = order[:budget - sinks - recent].sort().values + sinks
            kept = torch.cat([torch.arange(sinks, device="cuda"), mid,
                              torch.arange(c - recent, c, device="cuda")])
        k = torch.arange(kept.numel(), device="cuda")
        rec = st["pool"][st["table"][i, kept // bs].long(), kept % bs]
        st["dst_pool"][st["dst_table"][i, k // bs].long(), k % bs, :rb] = rec[:, :rb]
        st["kept"][i, :kept.numel()] = kept.to(torch.int32)
        st["kept"][i, kept.numel():] = -1
        st["new_lengths"][i] = kept.numel()
        st["acc_out"][i, :kept.numel()] = st["acc"][i, kept]
    return [st["kept"], st["new_lengths"], st["acc_out"], st["dst_pool"]]


def _verify_plain(st):
    target, draft, x = st["target"], st["draft"], st["tokens_in"].long()
    start = st["row_start"].long()
    rows, n = x.numel(), start.numel() - 1
    idx = torch.arange(rows, device="cuda")
    req = torch.searchsorted(start, idx, right=True) - 1
    p = target[idx, x].to(torch.float64)
    q = draft[idx, x].to(torch.float64) if draft is not None else torch.ones_like(p)
    ok = st["u"].to(torch.float64) * q < p
    if st["greedy"] is not None:
        ok = torch.where(st["greedy"][req] != 0, target.to(torch.float32).argmax(-1) == x, ok)
    last = idx == start[req + 1] - 1
    ok = ok & ~last
    # drafts accepted: those before the request's first refusal (its last row always refuses)
    bad = torch.where(ok, torch.full_like(idx, rows), idx)
    stop = torch.full((n,), rows, device="cuda").scatter_reduce(0, req, bad, "amin")
    a = stop - start[:-1]
    w = target[stop].to(torch.float64)
    bonus = stop == start[1:] - 1
    if draft is not None:
        res = (w - draft[stop].to(torch.float64)).clamp_min(0.0)
    else:
        res = w.clone()
        res[torch.arange(n, device="cuda"), x[stop]] = 0.0
    use = ~bonus & (res.sum(-1) > 0)
    w = torch.where(use[:, None], res, w)
    c = torch.cumsum(w, -1)
    tok = (c > st["r"].to(torch.float64)[:, None] * c[:, -1:]).to(torch.int8).argmax(-1)
    if st["greedy"] is not None:
        best = target[stop].to(torch.float32).argmax(-1)
        tok = torch.where(st["greedy"] != 0, best, tok)
    st["accepted"].copy_(a)
    out = torch.where(idx < stop[req], x, torch.full_like(x, -1))
    out[stop] = tok
    st["tokens"].copy_(out)
    return [st["accepted"], st["tokens"]]


# ------------------------------------------------------------------------------ exact
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


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "verify":
        return _verify_exact(st)
    if case["op"] == "evict":
        return _evict_exact(st)
    return _attend_exact(st)


def _attend_exact(st):
    """Row by row in 64 bits, from the stored bits."""
    case, lay = st["case"], st["layout"]
    kv, bs, dh, nq = lay["kv_dim"], lay["block_size"], lay["head_dim"], lay["n_q_heads"]
    per, n = nq // (kv // dh), case["rows"]
    lut = torch.tensor(_e4m3_table(), dtype=torch.float64, device="cuda")
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    acc = st["acc"].double() if case["weigh"] else None
    for i, c in enumerate(_contexts(case)):
        pages = st["pool"][st["table"][i, :(c + n + bs - 1) // bs].long()]
        rec = pages.reshape(-1, pages.shape[-1])[:c + n]
        scale = rec[:, kv:kv + 4].contiguous().view(torch.float32).double()
        pos = torch.arange(c + n, device="cuda")
        for j in range(n):
            row = i * n + j
            hi = c + (j if case["causal"] else n - 1)
            mask = pos <= hi
            if case["window"]:
                mask &= (pos >= hi - case["window"] + 1) | (pos < case["sinks"])
            sel = mask.nonzero()[:, 0]
            for sl in range(kv // dh):
                z = lut[rec[sel, sl * dh:(sl + 1) * dh].long()] * scale[sel]
                heads = slice(sl * per, (sl + 1) * per)
                q = st["q"][row].double().view(nq, dh)[heads]
                s = q @ z.T / math.sqrt(dh)
                norm = torch.logsumexp(s, -1)
                w = torch.exp(s - norm[:, None])
                o[row].view(nq, dh)[heads] = w @ z
                lse[row, heads] = norm
                if acc is not None:
                    acc[i].index_add_(0, sel, w.sum(0))
    return [o, lse] if acc is None else [o, lse, acc]


def _evict_exact(st):
    case = st["case"]
    acc = st["acc"].double().cpu().numpy()
    kept = np.full(st["kept"].shape, -1, np.int32)
    acc_out = np.zeros(tuple(st["acc_out"].shape), np.float64)
    lens = []
    for i, c in enumerate(_contexts(case)):
        keep = np.ones(c, bool)
        drop = c - case["budget"]
        if drop > 0:  # drop the lightest, of equals the last
            cand = np.arange(case["sinks"], c - case["recent"])
            order = np.lexsort((-cand, acc[i, cand]))
            keep[cand[order[:drop]]] = False
        ids = np.nonzero(keep)[0]
        kept[i, :len(ids)] = ids
        acc_out[i, :len(ids)] = acc[i, ids]
        lens.append(len(ids))
    return [torch.from_numpy(kept), torch.tensor(lens, dtype=torch.int32),
            torch.from_numpy(acc_out), None]


def _verify_exact(st):
    target = st["target"]
    x = st["tokens_in"].tolist()
    start, u, r = st["row_start"].tolist(), st["u"].tolist(), st["r"].tolist()
    greedy = st["greedy"].tolist() if st["greedy"] is not None else [0] * len(r)
    acc, out = [], [-1] * len(x)

    def row(t, i):
        return t[i].double().cpu().numpy()

    for i in range(len(r)):
        j = start[i]
        while True:
            p = row(target, j)
            end = j == start[i + 1] - 1
            if greedy[i]:
                best = int(np.flatnonzero(p == p.max())[0])
                if not end and best == x[j]:
                    out[j] = x[j]
                    j += 1
                    continue
                out[j] = best
                break
            if st["draft"] is not None:
                q = row(st["draft"], j)
            else:
                q = np.zeros_like(p)
                q[x[j]] = 1.0
            if not end and u[j] * q[x[j]] < p[x[j]]:
                out[j] = x[j]
                j += 1
                continue
            w = p if end else np.maximum(p - q, 0.0)
            if not w.any():
                w = p
            c = np.cumsum(w)
            out[j] = int(np.searchsorted(c, r[i] * c[-1], side="right"))
            break
        acc.append(j - start[i])
    return [torch.tensor(acc, dtype=torch.int32), torch.tensor(out, dtype=torch.int32)]
