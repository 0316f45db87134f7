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

from . import (GdrError, _BF16, _F32, _check, _dense, _host_i32, _load, _need,
               _workspace)

_Tensor, _INT32, _FLOAT32 = torch.Tensor, torch.int32, torch.float32
_DTYPES = {torch.bfloat16: _BF16, torch.float32: _F32}
# the current stream's handle, without a torch.cuda.Stream object around it
# (where this torch has no such function, by way of one)
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda index: torch.cuda.current_stream(index).cuda_stream))
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


# A decode step is microseconds of GPU work, so the checks cost as little as
# they can: one test per tensor, and a message only for one that fails.
def _gpu(name, t, dtype, dev, shape=None):
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.device == dev
            and t.is_contiguous()):
        _dense(name, t, dtype, dev)
    if shape is not None and t.shape != shape:
        raise GdrError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))


def _cache(k_cache, v_cache, scores):
    """Checks of the caches and their scores; returns their device, dtype,
    dtype code and shape (P, Hkv, page, D)."""
    if not (isinstance(k_cache, _Tensor) and k_cache.is_cuda and k_cache.is_contiguous()):
        _dense("k_cache", k_cache)
    dev, dtype, shape = k_cache.device, k_cache.dtype, k_cache.shape
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise GdrError("the cache must be bfloat16 or float32, got %s" % dtype)
    if len(shape) != 4 or shape[1] < 1:
        raise GdrError("k_cache must be [P,Hkv,page,D], got %s" % list(shape))
    _gpu("v_cache", v_cache, dtype, dev, shape)
    if scores is not None:
        _gpu("scores", scores, _FLOAT32, dev, shape[:3])
    return dev, dtype, dt, shape


def _int(name, x, lo):
    """A C int (ctypes would keep the low 32 bits of a larger one)."""
    if not lo <= x < 1 << 31:
        raise GdrError("%s = %r is outside %d..2^31-1" % (name, x, lo))


def _table(name, t, B, dev):
    _gpu(name, t, _INT32, dev)
    shape = t.shape
    if len(shape) != 2 or shape[0] != B:
        raise GdrError("%s must be [B,max_pages] with B = %d, got %s" % (name, B, list(shape)))
    if B >= 1 << 31 or shape[1] >= 1 << 31:     # (as in _int)
        raise GdrError("%s is too large: %s" % (name, list(shape)))
    return shape[1]


def _host_table(name, x, shape):
    if x is None:
        return None
    import numpy as np
    a = np.ascontiguousarray(np.asarray(x, dtype=np.int32))
    _need(a.shape == shape, "%s must be %s" % (name, list(shape)))
    return a


def _scratch(workspace, dev):
    """The bytes of a workspace; the library says if they are too few."""
    if not (isinstance(workspace, _Tensor) and workspace.device == dev
            and workspace.is_contiguous()):
        _dense("workspace", workspace, None, dev)
    return workspace.nbytes


def _p(t):
    return None if t is None else t.data_ptr()


def _hp(a):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def _call(dev, fn, *args):
    """fn(*args, stream): the current stream of dev, with dev current."""
    i = dev.index
    if i == _current_device():
        rc = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(i))
    if rc:
        _check(rc)


def cache_append(k, v, start, page_table, k_cache, v_cache, scores=None, cu_seqlens=None,
                 cu_seqlens_host=None):
    """Write new tokens into the cache, token t of sequence b at position
    start[b] + t.

    k, v [B,n,Hkv,D], or packed [T_tot,Hkv,D] with cu_seqlens int32 [B+1] on
    the GPU (rows behind the last sequence are left out; cu_seqlens_host, a
    host copy, makes the library validate it); start int32 [B] on the GPU.
    Positions outside the table or on an absent page are left out.  No two
    tokens of a call may name the same place (its contents are unspecified
    then): pages written belong to one sequence each.  scores, when given, are
    set to 0 at every position written.
    """
    dev, dtype, dt, (P, Hkv, page, D) = _cache(k_cache, v_cache, scores)
    _gpu("k", k, dtype, dev)
    shape, host = k.shape, None
    _gpu("v", v, dtype, dev, shape)
    if cu_seqlens is None:
        _need(len(shape) == 4 and shape[2:] == (Hkv, D), "k must be [B,n,Hkv,D]")
        B, n = shape[0], shape[1]
        T = B * n
        _need(cu_seqlens_host is None, "cu_seqlens_host given without cu_seqlens")
    else:
        _need(len(shape) == 3 and shape[1:] == (Hkv, D), "k must be [T_tot,Hkv,D]")
        _gpu("cu_seqlens", cu_seqlens, _INT32, dev)
        _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 1, "cu_seqlens must be [B+1]")
        B, n, T = cu_seqlens.numel() - 1, 0, shape[0]
        if cu_seqlens_host is not None:
            host = _host_i32(cu_seqlens_host, B + 1, "cu_seqlens_host")
    _int("the number of tokens", T, 0)
    _gpu("start", start, _INT32, dev, (B,))
    M = _table("page_table", page_table, B, dev)
    _call(dev, _load().gdr_cache_append, dt, B, n, T, Hkv, D, k.data_ptr(), v.data_ptr(),
          _p(cu_seqlens), _hp(host), start.data_ptr(), page_table.data_ptr(), M, page, P,
          k_cache.data_ptr(), v_cache.data_ptr(), _p(scores))


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
    dev, dtype, dt, (P, Hkv, page, D) = _cache(k_cache, v_cache, scores)
    _gpu("q", q, dtype, dev)
    shape = q.shape
    if len(shape) != 4 or shape[3] != D:
        raise GdrError("q must be [B,n,Hq,D] with D = %d, got %s" % (D, list(shape)))
    B, n, Hq, _ = shape
    if Hq < 1 or Hq % Hkv:
        raise GdrError("Hq (%d) must be a multiple of Hkv (%d)" % (Hq, Hkv))
    _gpu("seq_lens", seq_lens, _INT32, dev, (B,))
    M = _table("page_table", page_table, B, dev)
    host = None
    if page_table_host is not None:
        host = _host_table("page_table_host", page_table_host, (B, M))
    if o is None:
        o = torch.empty_like(q)
    else:
        _gpu("o", o, dtype, dev, shape)
    _int("window", window, 0)
    lib = _load()
    if workspace is None:
        workspace = _workspace(None, lib.gdr_attention_workspace_bytes(
            B, n, Hq, Hkv, D, M, page, scores is not None), dev)
    nbytes = _scratch(workspace, dev)
    _call(dev, lib.gdr_attention_decode, dt, B, n, Hq, Hkv, D,
          D ** -0.5 if scale is None else scale, window, q.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), page_table.data_ptr(), _hp(host), M, page, P, seq_lens.data_ptr(),
          _p(scores), o.data_ptr(), workspace.data_ptr(), nbytes)
    return o


def evict_workspace_bytes(batch: int, kv_heads: int, max_pages: int, page_size: int) -> int:
    """Bytes of device workspace cache_evict needs for these sizes: 0 for
    most (include/gdr_cache.h, gdr_cache_evict_workspace_bytes)."""
    return int(_load().gdr_cache_evict_workspace_bytes(int(batch), int(kv_heads), int(max_pages),
                                                       int(page_size)))


def cache_evict(k_cache, v_cache, scores, page_table, seq_lens, budget: int, recent: int = 0,
                sink: int = 0, new_page_table=None, new_lens=None, kept=None,
                page_table_host=None, new_page_table_host=None, workspace=None):
    """Trim every sequence to at most `budget` tokens by accumulated weight.

    Each key-value head of a longer sequence keeps the first `sink` tokens,
    the last `recent` and the highest-scored of the others (equal scores: the
    lower index), closed up in their order with their scores: in place, or,
    given new_page_table int32 [B, M'], copied into its pages (which no
    sequence uses yet).  Returns (new_lens int32 [B], kept int32
    [B,Hkv,budget]: the old index of each kept token, -1 past the new
    length).  new_lens may be seq_lens itself.  The host copies of the tables
    make the library validate them.  workspace (a device buffer of
    evict_workspace_bytes(...) bytes) is allocated when needed and not given.
    """
    _need(scores is not None, "scores are required")
    dev, _, dt, (P, Hkv, page, D) = _cache(k_cache, v_cache, scores)
    _gpu("seq_lens", seq_lens, _INT32, dev)
    _need(seq_lens.dim() == 1, "seq_lens must be [B]")
    B = seq_lens.shape[0]
    _int("budget", budget, 1)
    _int("recent", recent, 0)
    _int("sink", sink, 0)
    M = _table("page_table", page_table, B, dev)
    host = _host_table("page_table_host", page_table_host, (B, M))
    M2, host2 = 0, None
    if new_page_table is not None:
        M2 = _table("new_page_table", new_page_table, B, dev)
        host2 = _host_table("new_page_table_host", new_page_table_host, (B, M2))
        # (an empty table has no address, which would mean in place)
        _need(M2 * page >= min(budget, M * page), "new_page_table holds %d tokens, %d are kept"
              % (M2 * page, min(budget, M * page)))
    else:
        _need(new_page_table_host is None, "new_page_table_host given without new_page_table")
    if new_lens is None:
        new_lens = torch.empty_like(seq_lens)
    else:
        _gpu("new_lens", new_lens, _INT32, dev, (B,))
    if kept is None:
        kept = torch.empty((B, Hkv, budget), device=dev, dtype=_INT32)
    else:
        _gpu("kept", kept, _INT32, dev, (B, Hkv, budget))
    lib = _load()
    if workspace is None:
        nbytes = lib.gdr_cache_evict_workspace_bytes(B, Hkv, M, page)
        if nbytes:
            workspace = _workspace(None, nbytes, dev)
    else:
        nbytes = _scratch(workspace, dev)
    _call(dev, lib.gdr_cache_evict, dt, B, Hkv, D, budget, recent, sink, k_cache.data_ptr(),
          v_cache.data_ptr(), scores.data_ptr(), page_table.data_ptr(), _hp(host), M,
          _p(new_page_table), _hp(host2), M2, page, P, seq_lens.data_ptr(), new_lens.data_ptr(),
          kept.data_ptr(), _p(workspace), nbytes)
    return new_lens, kept
