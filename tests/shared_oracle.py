"""64-bit reference of the attention over shared prefixes, on the CPU, from the stored bits and the
formulas alone (no product code)."""
from __future__ import annotations

import math

import numpy as np

from tests.cache_oracle import E4M3, record


def attend(spec, q, positions, row_req, table, cache, prefix_table, lengths, prefix_of, causal=True,
           scale=None):
    """o, lse and bounds of the errors that roundings may bring to them.

    With a = |q|.|k| * scale the absolute score sum of a (head, token) and u = 2^-24: a score is a sum of
    128 exact products in f32 (128 u a), of a query carried to 2^-24 of its largest element: e_s.  A
    weight is then off by 2 e_s + 2^-18 relative (exponential, sums and normalisation in f32); times its
    scale it is rounded to f16, half a step being 2^-11, or absolutely 2^-25 where the largest of the
    tile that set the reference is above 2^5: 2^-30 of that, per token, times at most 448 of a code.  The
    sum over the values is one in f32 (2^-17 of the absolute sum, for long contexts too: the terms are
    added 16 tokens at a time), and o is rounded to bf16 (2^-8)."""
    kv, dh, nq, bs = spec["kv_dim"], spec["head_dim"], spec["n_q_heads"], spec["block_size"]
    G, rows, n_req = kv // dh, len(positions), table.shape[0]
    scale = 1.0 / math.sqrt(dh) if scale is None else scale
    o, tol = np.zeros((rows, nq * dh)), np.zeros((rows, nq * dh))
    lse, ltol = np.full((rows, nq), -np.inf), np.zeros((rows, nq))
    groups = {}
    for r in range(rows):
        b, p = int(row_req[r]), int(positions[r])
        if p < 0 or not 0 <= b < n_req:
            continue
        g = 0 if prefix_of is None else int(prefix_of[b])
        if not -1 <= g < len(lengths):
            continue
        hi = p if causal else max(int(positions[i]) for i in range(rows) if row_req[i] == b)
        groups.setdefault((b, g, hi), []).append(r)
    for (b, g, hi), who in groups.items():
        P = max(0, int(lengths[g])) if g >= 0 else 0
        at = [record(cache, prefix_table, g, t, bs) if t < P else record(cache, table, b, t, bs)
              for t in range(hi + 1)]
        at = [x for x in at if x is not None]
        if not at:
            continue
        rec = cache[tuple(np.array(at).T)]
        sc = np.ascontiguousarray(rec[:, kv:kv + 4]).view(np.float32).astype(np.float64)
        with np.errstate(all="ignore"):
            sc = np.where(np.abs(sc) <= 2.0 ** 64, sc, np.nan)
        codes = E4M3[rec[:, :kv]].reshape(-1, G, dh)
        for r in who:
            for s_ in range(G):
                hs = slice(s_ * (nq // G), (s_ + 1) * (nq // G))
                qh = q[r].reshape(nq, dh)[hs]
                with np.errstate(all="ignore"):
                    k = codes[:, s_] * sc
                    s = qh @ k.T * scale
                    a = np.abs(qh) @ np.abs(k).T * scale
                    e_s = (2.0 ** -17 * a + 2.0 ** -24 * np.abs(qh).max(-1, keepdims=True)
                           * np.abs(k).sum(-1) * scale)
                    m = s.max(-1, keepdims=True)
                    w = np.exp(s - m)
                    l = w.sum(-1, keepdims=True)
                    w /= l
                    out, aw = w @ k, w @ np.abs(k)
                    es = e_s.max(-1, keepdims=True)
                    o[r].reshape(nq, dh)[hs] = out
                    tol[r].reshape(nq, dh)[hs] = (2.0 ** -8 * np.abs(out) + 1.02 * (
                        (2.0 ** -11 + 2 * es + 2.0 ** -17) * (aw + np.abs(out))
                        + len(at) * 448 * 2.0 ** -30 * (w @ np.abs(sc))))
                    lse[r, hs] = (m + np.log(l))[:, 0]
                    ltol[r, hs] = es[:, 0] + 2.0 ** -18 + 2.0 ** -22 * np.abs(lse[r, hs])
    return o, tol, lse, ltol
