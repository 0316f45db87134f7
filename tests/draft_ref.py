"""Trees of drafts over the paged cache, what is kept of them, and page tables
that follow lengths, written out on the CPU: the reference of the tests.

Tables are host int arrays, caches CPU tensors [P, Hkv, page, D]; a page
outside 0..P-1 is absent.
"""
import numpy as np

from tests import cache_ref

U = 2.0 ** -24


def way(parents, t):
    """The drafts from the context to draft t."""
    out = []
    while True:
        out.append(t)
        p = int(parents[t])
        if not 0 <= p < t:
            return out[::-1]
        t = p


def attend(q, k_cache, v_cache, table, seq_lens, parents, scale, window=0):
    """o and its bound (those of cache_ref.attend, whose derivation holds for
    any set of tokens)."""
    import torch
    B, n, Hq, D = q.shape
    P, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    h = 2.0 ** -8 if q.dtype == torch.bfloat16 else U
    qd = q.double().numpy()
    kc, vc = k_cache.double().numpy(), v_cache.double().numpy()
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        c = max(0, min(int(seq_lens[b]), table.shape[1] * page)) - n
        for t in range(n):
            w = way(parents[b], t)
            p = c + len(w) - 1
            js = [j for j in range(max(c, 0)) if not window or j > p - window]
            js += [c + u for i, u in enumerate(w) if not window or c + i > p - window]
            at = [x for x in (cache_ref.place(table, P, page, b, j) for j in js) if x is not None]
            if not at:
                continue
            pg, sl = np.array([x[0] for x in at]), np.array([x[1] for x in at])
            for hq in range(Hq):
                k, v = kc[pg, hq // G, sl], vc[pg, hq // G, sl]
                x = qd[b, t, hq]
                s = scale * (k @ x)
                e = np.exp(s - s.max())
                wt = e / e.sum()
                o[b, t, hq] = wt @ v
                err = ((D + 2) * U * abs(scale) * (np.abs(k) @ np.abs(x)).max()
                       + 8 * U * np.abs(s).max() + 4 * U)
                rel = 2 * err + (len(at) + 16) * U
                bound[b, t, hq] = ((rel + h + (len(at) + 16) * U) * (wt @ np.abs(v))
                                   + h * np.abs(o[b, t, hq])) * (1 + 2.0 ** -6)
    return o, bound


def accept(k_cache, v_cache, table, seq_lens, parents, leaf, scores=None):
    """(k_cache, v_cache, scores, new_lens, path) after the call."""
    P, Hkv, page, _ = k_cache.shape
    B, n = parents.shape
    out = [x if x is None else x.clone() for x in (k_cache, v_cache, scores)]
    path, lens = np.full((B, n), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        L = max(0, min(int(seq_lens[b]), table.shape[1] * page))
        c = L - n
        w = way(parents[b], int(leaf[b])) if 0 <= leaf[b] < n else []
        w = [u for u in w if c + u >= 0]
        path[b, :len(w)] = w
        lens[b] = max(c, 0) + len(w)
        for i, u in enumerate(w):
            src = cache_ref.place(table, P, page, b, c + u)
            dst = cache_ref.place(table, P, page, b, max(c, 0) + i)
            if src is not None and dst is not None:
                for x, y in zip(out, (k_cache, v_cache, scores)):
                    if x is not None:
                        x[dst[0], :, dst[1]] = y[src[0], :, src[1]]
    return (*out, lens, path)


def resize(table, seq_lens, want, page, pages):
    """(table, new_lens, cu_seqlens, free) after the call."""
    table = table.copy()
    B, M = table.shape
    clamp = lambda x: max(0, min(int(x), M * page))  # noqa: E731
    old, new = [clamp(x) for x in seq_lens], [clamp(x) for x in want]
    have, need = ([-(-x // page) for x in y] for y in (old, new))
    used = set()
    for b in range(B):
        used.update(int(p) for p in table[b, :min(have[b], need[b])])
        table[b, need[b]:have[b]] = -1
    free = [p for p in range(pages) if p not in used]
    left, asked, lens, cu = list(free), 0, [], [0]
    for b in range(B):
        more = max(0, need[b] - have[b])
        asked += more
        if more and asked > len(free):
            lens.append(old[b])
        else:
            for c in range(have[b], have[b] + more):
                table[b, c] = left.pop(0)
            lens.append(new[b])
        cu.append(cu[-1] + max(0, lens[b] - old[b]))
    return table, np.array(lens, np.int32), np.array(cu, np.int32), len(left)
