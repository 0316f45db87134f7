"""The paged cache's operators in 64 bits, token by token on the CPU: the
reference of the tests, with the error bounds the kernels are held to.

Tables are host int arrays, caches CPU tensors [P, Hkv, page, D]; a page
outside 0..P-1 is absent.
"""
import math

import numpy as np
import torch


def place(table, pages, page, b, j):
    """(page, slot) of token j of sequence b, or None (absent, or outside)."""
    if j < 0 or j >= table.shape[1] * page:
        return None
    p = int(table[b, j // page])
    return (p, j % page) if 0 <= p < pages else None


def append(k, v, start, table, k_cache, v_cache, scores=None, cu=None):
    """New caches (and scores) after the call."""
    k_cache, v_cache = k_cache.clone(), v_cache.clone()
    scores = None if scores is None else scores.clone()
    P, _, page, _ = k_cache.shape
    for b in range(table.shape[0]):
        kb, vb = (x[b] if cu is None else x[cu[b]:cu[b + 1]] for x in (k, v))
        for t in range(kb.shape[0]):
            at = place(table, P, page, b, int(start[b]) + t)
            if at is not None:
                k_cache[at[0], :, at[1]] = kb[t]
                v_cache[at[0], :, at[1]] = vb[t]
                if scores is not None:
                    scores[at[0], :, at[1]] = 0
    return (k_cache, v_cache) if scores is None else (k_cache, v_cache, scores)


def attend(q, k_cache, v_cache, table, seq_lens, scale, window=0, scores=None):
    """o and its bound, and (scores given) the new scores and theirs.

    The bounds, with u = 2^-24 the fp32 half step and h the half step of the
    weights and of o (bf16: 2^-8; fp32: u):
      * a logit is a sum of D products and a scaling in fp32, off by at most
        (D + 2) u scale sum |q_i k_i|; its difference to the maximum, in
        units of log2, adds 4 u (|s| + |m|), the exponential 4 u relative.
        With e the largest such error of the row, every weight is off by at
        most 2 e + (N + 16) u relative, N the tokens summed (the sum's own
        rounding, counted to first order; the few rescalings of split sums
        are the 16);
      * rounding a weight to the product's operand adds h, the product's
        sums N u, all relative to sum w |v|; storing o adds h |o|;
      * a score adds rows of such weights: (rows + 2) u of the total.
    """
    B, n, Hq, D = q.shape
    P, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    u = 2.0 ** -24
    h = 2.0 ** -8 if q.dtype == torch.bfloat16 else u
    qd = q.double().numpy()
    kc, vc = k_cache.double().numpy(), v_cache.double().numpy()
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    sc = None if scores is None else scores.double().numpy().copy()
    sb = None if scores is None else np.zeros(scores.shape)
    rows = np.zeros((P, Hkv, page))
    for b in range(B):
        L = max(0, min(int(seq_lens[b]), table.shape[1] * page))
        for t in range(n):
            p = L - n + t
            js = range(max(0, p - window + 1) if window else 0, p + 1)
            at = [x for x in (place(table, P, page, b, j) for j in js) if x is not None]
            if not at:
                continue
            pg, sl = np.array([x[0] for x in at]), np.array([x[1] for x in at])
            for hk in range(Hkv):
                k, v = kc[pg, hk, sl], vc[pg, hk, sl]
                for g in range(G):
                    x = qd[b, t, hk * G + g]
                    s = scale * (k @ x)
                    m = s.max()
                    e = np.exp(s - m)
                    w = e / e.sum()
                    o[b, t, hk * G + g] = w @ v
                    err = ((D + 2) * u * abs(scale) * (np.abs(k) @ np.abs(x)).max()
                           + 4 * u * 2 * np.abs(s).max() + 4 * u)
                    rel = 2 * err + (len(at) + 16) * u
                    bound[b, t, hk * G + g] = (
                        (rel + h + (len(at) + 16) * u) * (w @ np.abs(v))
                        + h * np.abs(o[b, t, hk * G + g])) * (1 + 2.0 ** -6)
                    if sc is not None:
                        sc[pg, hk, sl] += w
                        sb[pg, hk, sl] += rel * w * (1 + 2.0 ** -6)
                        rows[pg, hk, sl] += 1
    if sc is None:
        return o, bound
    return o, bound, sc, sb + (rows + 2) * u * np.abs(sc)


def evict(k_cache, v_cache, scores, table, seq_lens, budget, recent=0, sink=0, new_table=None):
    """(k_cache, v_cache, scores, new_lens, kept) after the call."""
    P, Hkv, page, _ = k_cache.shape
    B = table.shape[0]
    to = table if new_table is None else new_table
    out = [x.clone() for x in (k_cache, v_cache, scores)]
    kept = np.full((B, Hkv, budget), -1, np.int32)
    lens = np.zeros(B, np.int32)
    for b in range(B):
        L = max(0, min(int(seq_lens[b]), table.shape[1] * page))
        lens[b] = min(L, budget)
        for h in range(Hkv):
            keep = list(range(L))
            if L > budget:
                def rank(j):
                    at = place(table, P, page, b, j)
                    if at is None:
                        return (1, 0.0, j)
                    s = float(scores[at[0], h, at[1]])
                    return (0, math.inf if math.isnan(s) else -s, j)
                mid = sorted(range(sink, L - recent), key=rank)[:budget - sink - recent]
                keep = sorted(list(range(sink)) + mid + list(range(L - recent, L)))
            kept[b, h, :len(keep)] = keep
            for i, j in enumerate(keep):
                src, dst = place(table, P, page, b, j), place(to, P, page, b, i)
                if src is not None and dst is not None:
                    for x, y in zip(out, (k_cache, v_cache, scores)):
                        x[dst[0], h, dst[1]] = y[src[0], h, src[1]]
    return (*out, lens, kept)
