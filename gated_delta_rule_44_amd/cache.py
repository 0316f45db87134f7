"""The paged key-value cache of a placement's attention layers: the write of
new tokens, attention of new tokens over the cache, and eviction by
accumulated attention weight (include/gdr_cache.h states each call in full).

k_cache, v_cache [P, Hkv, page, D] (bf16 or fp32), page one of 16, 32, 64,
128, 256 tokens; page_table int32 [B, max_pages] on the GPU names the pages of
each sequence (-1, or any entry outside 0..P-1: absent); scores
[P, Hkv, page] fp32 hold one accumulated attention weight per cached token
and key-value head.
"""
from __future__ import annotations

import ctypes

import torch

from . import GdrError, _BF16, _F32, _check, _dense, _host_i32, _load, _need, _workspace


def _i32(name, t, shape, dev):
    _dense(name, t, torch.int32, dev)
    _need(t.shape == shape, "%s must be %s, got %s" % (name, list(shape), list(t.shape)))


def _cache(k_cache, v_cache, scores, dtype=None):
    """Checks of the caches and their scores; returns P, Hkv, page, D."""
    _dense("k_cache", k_cache, dtype)
    _need(k_cache.dim() == 4 and k_cache.shape[1] >= 1, "k_cache must be [P,Hkv,page,D]")
    _dense("v_cache", v_cache, k_cache.dtype, k_cache.device)
    _need(v_cache.shape == k_cache.shape, "k_cache, v_cache shapes differ")
    if scores is not None:
        _dense("scores", scores, torch.float32, k_cache.device)
        _need(scores.shape == k_cache.shape[:3], "scores must be [P,Hkv,page]")
    return k_cache.shape


def _table(name, t, B, dev):
    _dense(name, t, torch.int32, dev)
    _need(t.dim() == 2 and t.shape[0] == B, "%s must be [B,max_pages]" % name)
    return t.shape[1]


def _host_table(name, x, shape):
    if x is None:
        return None
    import numpy as np
    a = np.ascontiguousarray(np.asarray(x, dtype=np.int32))
    _need(a.shape == shape, "%s must be %s" % (name, list(shape)))
    return a


def _dt(t):
    if t.dtype == torch.bfloat16:
        return _BF16
    if t.dtype == torch.float32:
        return _F32
    raise GdrError("the cache must be bfloat16 or float32, got %s" % t.dtype)


def _p(t):
    return None if t is None else t.data_ptr()


def _hp(a):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def _call(dev, fn, *args):
    """fn(*args, stream): the current stream of dev, with dev current."""
    stream = torch.cuda.current_stream(dev).cuda_stream
    if dev.index == torch.cuda.current_device():
        _check(fn(*args, stream))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, stream))


def cache_append(k, v, start, page_table, k_cache, v_cache, scores=None, cu_seqlens=None,
                 cu_seqlens_host=None):
    """Write new tokens into the cache, token t of sequence b at position
    start[b] + t.

    k, v [B,n,Hkv,D], or packed [T_tot,Hkv,D] with cu_seqlens int32 [B+1] on
    the GPU (rows behind the last sequence are left out; cu_seqlens_host, a
    host copy, makes the library validate it); start int32 [B] on the GPU.
    Positions outside the table or on an absent page are left out.  scores,
    when given, are set to 0 at every position written.
    """
    P, Hkv, page, D = _cache(k_cache, v_cache, scores)
    dev = k_cache.device
    _dense("k", k, k_cache.dtype, dev)
    _dense("v", v, k_cache.dtype, dev)
    _need(k.shape == v.shape, "k, v shapes differ")
    host = None
    if cu_seqlens is None:
        _need(k.dim() == 4 and k.shape[2:] == (Hkv, D), "k must be [B,n,Hkv,D]")
        B, n = k.shape[:2]
        T = B * n
        _need(cu_seqlens_host is None, "cu_seqlens_host given without cu_seqlens")
    else:
        _need(k.dim() == 3 and k.shape[1:] == (Hkv, D), "k must be [T_tot,Hkv,D]")
        _dense("cu_seqlens", cu_seqlens, torch.int32, dev)
        _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 1, "cu_seqlens must be [B+1]")
        B, n, T = cu_seqlens.numel() - 1, 0, k.shape[0]
        host = None if cu_seqlens_host is None else _host_i32(cu_seqlens_host, B + 1,
                                                               "cu_seqlens_host")
    _i32("start", start, (B,), dev)
    M = _table("page_table", page_table, B, dev)
    _call(dev, _load().gdr_cache_append, _dt(k_cache), B, n, T, Hkv, D, _p(k), _p(v),
          _p(cu_seqlens), _hp(host), _p(start), _p(page_table), M, page, P, _p(k_cache),
          _p(v_cache), _p(scores))


def attention_workspace_bytes(batch: int, n_tok: int, heads: int, kv_heads: int, dim: int,
                              max_pages: int, page_size: int, with_scores: bool = False) -> int:
    """Bytes of device workspace attention_decode needs for these sizes
    (include/gdr_cache.h, gdr_attention_workspace_bytes)."""
    return int(_load().gdr_attention_workspace_bytes(
        int(batch), int(n_tok), int(heads), int(kv_heads), int(dim), int(max_pages),
        int(page_size), int(bool(with_scores))))


def attention_decode(q, k_cache, v_cache, page_table, seq_lens, scale=None, window: int = 0,
                     scores=None, o=None, workspace=None, page_table_host=None):
    """Attention of the newest n tokens of each sequence over its cache.

    q [B,n,Hq,D], Hq a multiple of Hkv; seq_lens int32 [B] on the GPU: the
    tokens cached, the n newest included (append them first), so that query
    token t stands at position seq_lens[b] - n + t.  window 0: full attention
    over the tokens up to the row's own; W > 0: the last W of them.  scale
    defaults to 1 / sqrt(D).  scores, when given, gain each token's attention
    weights, summed over the rows that read the token (a page then belongs
    to one sequence; page_table_host, a host copy, makes the library validate
    that).  A row that attends to nothing gives zeros.  Returns o [B,n,Hq,D].
    """
    P, Hkv, page, D = _cache(k_cache, v_cache, scores)
    dev = k_cache.device
    _dense("q", q, k_cache.dtype, dev)
    _need(q.dim() == 4 and q.shape[3] == D, "q must be [B,n,Hq,D]")
    B, n, Hq, _ = q.shape
    _need(Hq >= 1 and Hq % Hkv == 0, "Hq (%d) must be a multiple of Hkv (%d)" % (Hq, Hkv))
    _i32("seq_lens", seq_lens, (B,), dev)
    M = _table("page_table", page_table, B, dev)
    host = _host_table("page_table_host", page_table_host, (B, M))
    if o is None:
        o = torch.empty_like(q)
    else:
        _dense("o", o, q.dtype, dev)
        _need(o.shape == q.shape, "o must be [B,n,Hq,D]")
    lib = _load()
    nbytes = lib.gdr_attention_workspace_bytes(B, n, Hq, Hkv, D, M, page, int(scores is not None))
    workspace = _workspace(workspace, nbytes, dev)
    _call(dev, lib.gdr_attention_decode, _dt(k_cache), B, n, Hq, Hkv, D,
          D ** -0.5 if scale is None else float(scale), int(window), _p(q), _p(k_cache),
          _p(v_cache), _p(page_table), _hp(host), M, page, P, _p(seq_lens), _p(scores), _p(o),
          _p(workspace), nbytes)
    return o


def cache_evict(k_cache, v_cache, scores, page_table, seq_lens, budget: int, recent: int = 0,
                sink: int = 0, new_page_table=None, new_lens=None, kept=None,
                page_table_host=None, new_page_table_host=None):
    """Trim every sequence to at most `budget` tokens by accumulated weight.

    Each key-value head of a longer sequence keeps the first `sink` tokens,
    the last `recent` and the highest-scored of the others (equal scores: the
    lower index), closed up in their order with their scores: in place, or,
    given new_page_table int32 [B, M'], copied into its pages (which no
    sequence uses yet).  Returns (new_lens int32 [B], kept int32
    [B,Hkv,budget]: the old index of each kept token, -1 past the new
    length).  new_lens may be seq_lens itself.  The host copies of the tables
    make the library validate them.
    """
    _need(scores is not None, "scores are required")
    P, Hkv, page, D = _cache(k_cache, v_cache, scores)
    dev = k_cache.device
    _dense("seq_lens", seq_lens, torch.int32, dev)
    _need(seq_lens.dim() == 1, "seq_lens must be [B]")
    B, budget = seq_lens.shape[0], int(budget)
    _need(budget >= 1, "budget must be at least 1")
    M = _table("page_table", page_table, B, dev)
    host = _host_table("page_table_host", page_table_host, (B, M))
    M2, host2 = 0, None
    if new_page_table is not None:
        M2 = _table("new_page_table", new_page_table, B, dev)
        host2 = _host_table("new_page_table_host", new_page_table_host, (B, M2))
    else:
        _need(new_page_table_host is None, "new_page_table_host given without new_page_table")
    if new_lens is None:
        new_lens = torch.empty_like(seq_lens)
    else:
        _i32("new_lens", new_lens, (B,), dev)
    if kept is None:
        kept = torch.empty((B, Hkv, budget), device=dev, dtype=torch.int32)
    else:
        _i32("kept", kept, (B, Hkv, budget), dev)
    _call(dev, _load().gdr_cache_evict, _dt(k_cache), B, Hkv, D, budget, int(recent), int(sink),
          _p(k_cache), _p(v_cache), _p(scores), _p(page_table), _hp(host), M,
          _p(new_page_table), _hp(host2), M2, page, P, _p(seq_lens), _p(new_lens), _p(kept))
    return new_lens, kept
