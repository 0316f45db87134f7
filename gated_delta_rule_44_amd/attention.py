"""Attention of whole prompts and its gradients, for the attention layers of a
placement (include/gdr_attention.h states each call in full).

A batch is fixed-length, q [B,T,Hq,D] with k, v [B,T,Hkv,D], or packed,
q [T_tot,Hq,D] with k, v [T_tot,Hkv,D] and cu_seqlens int32 [B+1] on the GPU;
Hq is a multiple of Hkv, and query head h reads key-value head
h / (Hq / Hkv).  bf16 or fp32; D 64 or 128.
"""
from __future__ import annotations

import torch

from . import GdrError, _dense, _host_i32, _load, _need, _workspace
from .cache import _DTYPES, _FLOAT32, _INT32, _call, _gpu, _hp, _int, _p, _scratch


def _prompts(q, k, v, cu_seqlens, cu_seqlens_host, window):
    """Checks of a batch of prompts; returns its device, dtype code and sizes
    (B, T, T_total, Hq, Hkv, D) and the host offsets."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.is_contiguous()):
        _dense("q", q)
    dev, dtype, shape, host = q.device, q.dtype, q.shape, None
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise GdrError("q must be bfloat16 or float32, got %s" % dtype)
    if len(shape) != (4 if cu_seqlens is None else 3):
        raise GdrError("q must be [B,T,Hq,D], or [T_tot,Hq,D] with cu_seqlens, got %s"
                       % list(shape))
    _gpu("k", k, dtype, dev)
    Hq, D, Hkv = shape[-2], shape[-1], k.shape[-2] if k.dim() == len(shape) else 0
    _gpu("v", v, dtype, dev, (*shape[:-2], Hkv, D))
    _gpu("k", k, dtype, dev, (*shape[:-2], Hkv, D))
    if Hkv < 1 or Hq % Hkv:
        raise GdrError("Hq (%d) must be a multiple of Hkv (%d)" % (Hq, Hkv))
    if cu_seqlens is None:
        B, T = shape[0], shape[1]
        total = B * T
        _need(cu_seqlens_host is None, "cu_seqlens_host given without cu_seqlens")
    else:
        _gpu("cu_seqlens", cu_seqlens, _INT32, dev)
        _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 1, "cu_seqlens must be [B+1]")
        B, T, total = cu_seqlens.numel() - 1, 0, shape[0]
        if cu_seqlens_host is not None:
            host = _host_i32(cu_seqlens_host, B + 1, "cu_seqlens_host")
    _int("the number of tokens", total, 0)
    _int("the number of sequences", B, 0)
    _int("Hq", Hq, 1)
    _int("D", D, 1)
    _int("window", window, 0)
    return dev, dtype, dt, (B, T, total, Hq, Hkv, D), host


def attention_prefill(q, k, v, cu_seqlens=None, cu_seqlens_host=None, scale=None, window: int = 0,
                      lse=None, o=None):
    """Attention over whole prompts: every token attends to the tokens of its
    sequence up to its own (window 0), or to the last `window` of them.

    scale defaults to 1 / sqrt(D).  Rows of a packed batch behind the last
    sequence are left as they are.  lse: None, True, or an fp32 tensor [B,T,Hq]
    ([T_tot,Hq]) that receives ln sum e^{logit} of every row, which
    attention_backward needs.  Returns o like q, or (o, lse).
    """
    dev, dtype, dt, sizes, host = _prompts(q, k, v, cu_seqlens, cu_seqlens_host, window)
    if o is None:
        o = torch.empty_like(q)
    else:
        _gpu("o", o, dtype, dev, q.shape)
    if lse is True:
        lse = torch.empty(q.shape[:-1], device=dev, dtype=_FLOAT32)
    elif lse is not None:
        _gpu("lse", lse, _FLOAT32, dev, q.shape[:-1])
    B, T, total, Hq, Hkv, D = sizes
    _call(dev, _load().gdr_attention_prefill, dt, B, T, total, Hq, Hkv, D,
          D ** -0.5 if scale is None else scale, window, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          _p(cu_seqlens), _hp(host), o.data_ptr(), _p(lse))
    return o if lse is None else (o, lse)


def attention_backward_workspace_bytes(dtype, n_seqs: int, tokens: int, heads: int, kv_heads: int,
                                       dim: int) -> int:
    """Bytes of device workspace attention_backward needs over n_seqs sequences
    of `tokens` tokens in all (include/gdr_attention.h)."""
    _need(dtype in _DTYPES, "dtype must be bfloat16 or float32, got %s" % dtype)
    return int(_load().gdr_attention_backward_workspace_bytes(
        _DTYPES[dtype], int(n_seqs), int(tokens), int(heads), int(kv_heads), int(dim)))


def attention_backward(q, k, v, o, lse, do, cu_seqlens=None, cu_seqlens_host=None, scale=None,
                       window: int = 0, dq=None, dk=None, dv=None, workspace=None):
    """Gradients of attention_prefill: o and lse as it gave them for these
    inputs, do the gradient of o.  Returns (dq, dk, dv) in the dtype and the
    shapes of q, k and v, which may be passed in; rows of a packed batch behind
    the last sequence are left as they are.  workspace (a device buffer of
    attention_backward_workspace_bytes(...) bytes) is allocated when not given.
    """
    dev, dtype, dt, sizes, host = _prompts(q, k, v, cu_seqlens, cu_seqlens_host, window)
    _gpu("o", o, dtype, dev, q.shape)
    _gpu("do", do, dtype, dev, q.shape)
    _gpu("lse", lse, _FLOAT32, dev, q.shape[:-1])
    grads = []
    for name, x, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if x is None:
            x = torch.empty_like(like)
        else:
            _gpu(name, x, dtype, dev, like.shape)
        grads.append(x)
    B, T, total, Hq, Hkv, D = sizes
    lib = _load()
    if workspace is None:
        workspace = _workspace(None, lib.gdr_attention_backward_workspace_bytes(
            dt, B, total, Hq, Hkv, D), dev)
    nbytes = _scratch(workspace, dev)
    _call(dev, lib.gdr_attention_backward, dt, B, T, total, Hq, Hkv, D,
          D ** -0.5 if scale is None else scale, window, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          _p(cu_seqlens), _hp(host), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
          *(x.data_ptr() for x in grads), workspace.data_ptr(), nbytes)
    return tuple(grads)
