"""64-bit references of the cache operators, on the CPU, from the stored bits and the formulas
alone (no product code)."""
from __future__ import annotations

import math

import numpy as np


def e4m3_values():
    v = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        v[b] = (math.nan if (b & 127) == 127 else x) * (-1 if b & 128 else 1)
    return v


E4M3 = e4m3_values()


def record(cache, table, b, t, bs):
    """(page, slot) of token t of request b, or None where the page is unmapped."""
    lb = t // bs
    if lb >= table.shape[1]:
        return None
    pg = int(table[b, lb])
    return (pg, t % bs) if 0 <= pg < cache.shape[0] else None


def visible(hi, window, sinks):
    t = np.arange(hi + 1)
    return t if window == 0 else t[(t > hi - window) | (t < sinks)]


def attend(spec, q, positions, row_req, table, cache, window=0, sinks=0, causal=True, scale=None,
           n_weights=0):
    """o, lse, weights added, and bounds of the errors that roundings may bring to them.

    The bounds, with a = |q|.|k| * scale the absolute score sum of a (head, token), u = 2^-24:
    a score is a sum of 128 products in f32 (128 u a), of a query carried to 2^-18 of its largest
    element (2^-18 qmax |k|_1 * scale): e_s.  A weight is then off by 2 e_s + 2^-18 relative
    (exponential, sums and normalisation in f32).  In the sum over the values weights are
    carried in two 4-bit terms (2^-4 * 2^-4 relative, 2^-17 of the largest of 32 tokens
    absolute: 2^-12 of their sum, times at most 448 of a code), and o is rounded to bf16 (2^-8)."""
    kv, dh, nq, bs = spec["kv_dim"], spec["head_dim"], spec["n_q_heads"], spec["block_size"]
    G, rows = kv // dh, len(positions)
    scale = 1.0 / math.sqrt(dh) if scale is None else scale
    o, tol = np.zeros((rows, nq * dh)), np.zeros((rows, nq * dh))
    lse, ltol = np.full((rows, nq), -np.inf), np.zeros((rows, nq))
    n_req = table.shape[0]
    w_add, w_tol = np.zeros((n_req, n_weights)), np.zeros((n_req, n_weights))
    for r in range(rows):
        b, p = int(row_req[r]), int(positions[r])
        if p < 0 or b < 0 or b >= n_req:
            continue
        hi = p if causal else max(int(positions[i]) for i in range(rows) if row_req[i] == b)
        loc = [(t, record(cache, table, b, int(t), bs)) for t in visible(hi, window, sinks)]
        toks = np.array([t for t, x in loc if x is not None], dtype=np.int64)
        if not len(toks):
            continue
        rec = np.stack([cache[x] for _, x in loc if x is not None])
        sc = np.ascontiguousarray(rec[:, kv:kv + 4]).view(np.float32).astype(np.float64)
        codes = E4M3[rec[:, :kv]].reshape(-1, G, dh)
        for g in range(G):
            hs = slice(g * (nq // G), (g + 1) * (nq // G))
            qh = q[r].reshape(nq, dh)[hs]
            k = codes[:, g] * sc
            s = qh @ k.T * scale
            a = np.abs(qh) @ np.abs(k).T * scale
            e_s = (2.0 ** -17 * a + 2.0 ** -18 * np.abs(qh).max(-1, keepdims=True)
                   * np.abs(k).sum(-1) * scale)
            m = s.max(-1, keepdims=True)
            w = np.exp(s - m)
            l = w.sum(-1, keepdims=True)
            w /= l
            out = w @ k
            o[r].reshape(nq, dh)[hs] = out
            aw = w @ np.abs(k)
            es = e_s.max(-1, keepdims=True)
            tol[r].reshape(nq, dh)[hs] = (2.0 ** -8 * np.abs(out) + 1.02 * (
                (2.0 ** -8 + 2 * es + 2.0 ** -18) * (aw + np.abs(out))
                + 2.0 ** -12 * 448 * (w @ np.abs(sc))))
            lse[r, hs] = (m + np.log(l))[:, 0]
            ltol[r, hs] = es[:, 0] + 2.0 ** -18 + 2.0 ** -22 * np.abs(lse[r, hs])
            if n_weights:
                sel = toks < n_weights
                w_add[b, toks[sel]] += w.sum(0)[sel]
                w_tol[b, toks[sel]] += (w * (2.2 * e_s + 2 * es + 2.0 ** -17)).sum(0)[sel]
    return o, tol, lse, ltol, w_add, w_tol


def evict(weights, lengths, budget, sinks, recent):
    """Kept slots per request."""
    out = []
    for b, n in enumerate(lengths):
        if n <= budget:
            out.append(list(range(max(0, n))))
            continue
        key = [(-math.inf if math.isnan(x) else x) for x in weights[b, :n].tolist()]
        mid = sorted(range(sinks, n - recent), key=lambda t: (-key[t], t))
        out.append(sorted(list(range(sinks)) + mid[:budget - sinks - recent]
                          + list(range(n - recent, n))))
    return out


def verify(target, draft, tokens_in, row_start, u, r, greedy=None):
    """(accepted, tokens) with None for tokens of rows outside every request."""
    rows, V = target.shape
    acc, out = [], [None] * rows

    def pos(x):
        return np.where(x > 0, x, 0.0)  # NaN and negatives count as 0

    for b in range(len(row_start) - 1):
        s = min(max(row_start[b], 0), rows)
        e = min(max(row_start[b + 1], s), rows)
        if s == e:
            acc.append(0)
            continue
        for j in range(s, e):
            out[j] = -1
        j = s
        while True:
            x, end = int(tokens_in[j]), j == e - 1
            ok = not end and 0 <= x < V
            if greedy is not None and greedy[b]:
                t = np.where(np.isnan(target[j]), -np.inf, target[j])
                best = int(np.argmax(t))
                if ok and best == x:
                    out[j] = x
                    j += 1
                    continue
                out[j] = best
                break
            p = pos(target[j])
            q = np.zeros(V)
            if draft is not None:
                q = pos(draft[j])
            elif 0 <= x < V:
                q[x] = 1.0
            if ok and float(u[j]) * q[x] < p[x]:
                out[j] = x
                j += 1
                continue
            w = p if end else np.maximum(p - q, 0.0)
            if not w.any():
                w = p
            if w.any():
                c = np.cumsum(w)
                out[j] = int(np.searchsorted(c, float(r[b]) * c[-1], side="right"))
            break
        acc.append(j - s)
    return acc, out
