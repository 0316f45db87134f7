"""CPU tests of the paged cache's C ABI (include/gdr_cache.h): every declared
symbol is exported, and bad arguments, page tables among them, are rejected
on the host before any HIP call (nothing is launched here)."""
import ctypes
import os
import re

import numpy as np
import pytest

import gated_delta_rule_44_amd as gdr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdr_cache.h")
EINVAL, EUNSUPPORTED = 1, 2
F = ctypes.c_float
FAKE = 1 << 20          # aligned, never dereferenced: validation fails first
MIS = FAKE + 2          # misaligned for every type


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdr.lib_path()):
        pytest.skip("libgdr.so not built")
    return gdr._load()


def err(lib):
    return lib.gdr_last_error().decode()


def hp(a):
    return None if a is None else np.ascontiguousarray(a, np.int32).ctypes.data_as(ctypes.c_void_p)


def test_library_exports_every_declared_symbol(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gdr_[a-z_]+)\s*\(", src)))
    assert names == ["gdr_attention_decode", "gdr_attention_workspace_bytes", "gdr_cache_append",
                     "gdr_cache_evict", "gdr_cache_evict_workspace_bytes"]
    for name in names:
        assert hasattr(ctypes.CDLL(gdr.lib_path()), name), name


def append(lib, dt=1, B=2, n=3, T=6, Hkv=2, D=128, k=FAKE, v=FAKE, cu=None, cu_host=None,
           start=FAKE, table=FAKE, M=4, page=16, P=9, kc=FAKE, vc=FAKE, sc=None):
    return lib.gdr_cache_append(dt, B, n, T, Hkv, D, k, v, cu, hp(cu_host), start, table, M, page,
                                P, kc, vc, sc, None)


CACHE = [   # what every call checks
    (dict(dt=5), EINVAL, "dtype"),
    (dict(D=96), EUNSUPPORTED, "supported widths"),
    (dict(B=-1), EINVAL, "bad sizes"),
    (dict(Hkv=0), EINVAL, "bad sizes"),
    (dict(M=-1), EINVAL, "bad sizes"),
    (dict(P=-1), EINVAL, "bad sizes"),
    (dict(page=8), EUNSUPPORTED, "page_size"),
    (dict(page=48), EUNSUPPORTED, "page_size"),
    (dict(page=512), EUNSUPPORTED, "page_size"),
    (dict(M=1 << 22, page=256), EUNSUPPORTED, "too long"),
    (dict(P=1 << 30), EUNSUPPORTED, "too large"),
    (dict(table=None), EINVAL, "page_table is NULL"),
    (dict(table=MIS), EINVAL, "page_table is not 4-byte aligned"),
    (dict(kc=None), EINVAL, "k_cache is NULL"),
    (dict(vc=MIS), EINVAL, "v_cache is not 16-byte aligned"),
    (dict(sc=MIS), EINVAL, "scores is not 16-byte aligned"),
]


@pytest.mark.parametrize("kw,code,msg", CACHE + [
    (dict(n=-1), EINVAL, "bad sizes"),
    (dict(T=-1), EINVAL, "bad sizes"),
    (dict(T=7), EINVAL, "T_total = 7 but B * n_tok = 6"),
    (dict(B=1 << 14, n=1 << 12, T=1 << 26), EUNSUPPORTED, "rows exceed"),
    (dict(k=None), EINVAL, "k is NULL"),
    (dict(v=MIS), EINVAL, "v is not 16-byte aligned"),
    (dict(start=None), EINVAL, "start is NULL"),
    (dict(cu_host=[0, 3, 6]), EINVAL, "without cu_seqlens"),
    (dict(cu=MIS), EINVAL, "cu_seqlens is not 4-byte aligned"),
    (dict(cu=FAKE, cu_host=[1, 3, 6]), EINVAL, "expected 0"),
    (dict(cu=FAKE, cu_host=[0, 4, 3]), EINVAL, "decreases"),
    (dict(cu=FAKE, cu_host=[0, 4, 7]), EINVAL, "T_total"),
])
def test_append_rejects(lib, kw, code, msg):
    assert append(lib, **kw) == code
    assert msg in err(lib)


def test_empty_calls_are_ok_without_gpu(lib):
    assert append(lib, B=0, T=0) == 0
    assert append(lib, n=0, T=0) == 0
    assert append(lib, M=0, table=None) == 0          # no place for any token
    assert append(lib, P=0, kc=None, vc=None) == 0
    assert attend(lib, B=0) == 0
    assert attend(lib, n=0) == 0
    assert evict(lib, B=0) == 0


def attend(lib, dt=1, B=2, n=1, Hq=4, Hkv=2, D=128, scale=1.0, window=0, q=FAKE, kc=FAKE, vc=FAKE,
           table=FAKE, host=None, M=4, page=16, P=9, lens=FAKE, sc=None, o=FAKE, ws=FAKE,
           ws_bytes=1 << 40):
    return lib.gdr_attention_decode(dt, B, n, Hq, Hkv, D, F(scale), window, q, kc, vc, table,
                                    hp(host), M, page, P, lens, sc, o, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code,msg", CACHE + [
    (dict(n=-1), EINVAL, "bad sizes"),
    (dict(Hq=0), EINVAL, "bad sizes"),
    (dict(Hq=5), EINVAL, "not a multiple"),
    (dict(scale=float("nan")), EINVAL, "scale"),
    (dict(scale=float("inf")), EINVAL, "scale"),
    (dict(window=-1), EINVAL, "window"),
    (dict(B=1 << 13, n=1 << 8), EUNSUPPORTED, "query rows"),
    (dict(B=1 << 30, n=1 << 30, Hq=16), EUNSUPPORTED, "query rows"),
    (dict(q=None), EINVAL, "q is NULL"),
    (dict(o=MIS), EINVAL, "o is not 16-byte aligned"),
    (dict(lens=None), EINVAL, "seq_lens is NULL"),
    (dict(ws=None, sc=FAKE), EINVAL, "workspace"),
    (dict(ws_bytes=1, sc=FAKE), EINVAL, "workspace"),
    (dict(host=[[0, 1, 2, 9], [3, 4, 5, -1]]), EINVAL, "page_table[0, 3] = 9 outside -1..8"),
    (dict(host=[[0, 1, 2, 8], [3, 4, -2, -1]]), EINVAL, "page_table[1, 2] = -2 outside"),
    (dict(host=[[0, 1, 2, 8], [3, 1, -1, -1]], sc=FAKE), EINVAL, "page 1 is in page_table twice"),
])
def test_attend_rejects(lib, kw, code, msg):
    assert attend(lib, **kw) == code
    assert msg in err(lib)


def evict(lib, dt=1, B=2, Hkv=2, D=128, budget=40, recent=8, sink=4, kc=FAKE, vc=FAKE, sc=FAKE,
          table=FAKE, host=None, M=4, new=None, new_host=None, M2=0, page=16, P=9, lens=FAKE,
          new_lens=FAKE, kept=FAKE, ws=None, ws_bytes=0):
    return lib.gdr_cache_evict(dt, B, Hkv, D, budget, recent, sink, kc, vc, sc, table, hp(host), M,
                               new, hp(new_host), M2, page, P, lens, new_lens, kept, ws, ws_bytes,
                               None)


@pytest.mark.parametrize("kw,code,msg", CACHE + [
    (dict(sc=None), EINVAL, "scores is NULL"),
    (dict(budget=0), EINVAL, "budget"),
    (dict(recent=-1), EINVAL, "budget"),
    (dict(sink=-1), EINVAL, "budget"),
    (dict(recent=30, sink=11), EINVAL, "must fit the budget"),
    (dict(recent=2 ** 31 - 1, sink=2 ** 31 - 1), EINVAL, "must fit the budget"),
    (dict(budget=1 << 30), EUNSUPPORTED, "budget"),
    (dict(B=1 << 20), EUNSUPPORTED, "pairs exceed"),
    (dict(lens=None), EINVAL, "seq_lens is NULL"),
    (dict(new_lens=None), EINVAL, "new_lens is NULL"),
    (dict(kept=MIS), EINVAL, "kept is not 4-byte aligned"),
    (dict(new=MIS, M2=3), EINVAL, "new_page_table is not 4-byte aligned"),
    (dict(new=FAKE, M2=2), EINVAL, "a new table of 2 pages of 16 tokens for 40 tokens"),
    (dict(new=FAKE, M2=3, budget=1000), EINVAL, "for 64 tokens"),
    (dict(new=FAKE, M2=1 << 26), EINVAL, "a new table of"),
    (dict(new_host=[[1], [2]]), EINVAL, "without new_page_table"),
    (dict(host=[[0, 1, 2, 3], [4, 5, 6, 9]]), EINVAL, "outside"),
    (dict(host=[[0, 1, 2, 3], [4, 5, 6, 2]]), EINVAL, "page 2 is in page_table twice"),
    (dict(new=FAKE, M2=3, new_host=[[0, 1, 2], [3, 1, 4]]), EINVAL, "page 1 is in new_page_table"),
    (dict(new=FAKE, M2=3, new_host=[[0, 1, 2], [3, 10, 4]]), EINVAL, "outside"),
    (dict(new=FAKE, M2=3, host=[[5, 6, 7, 8], [5, 6, 7, 4]], new_host=[[0, 1, 2], [3, -1, 4]]),
     EINVAL, "page 4 is in both tables"),
    (dict(M=1000), EINVAL, "workspace of"),
    (dict(M=1000, ws=MIS, ws_bytes=1 << 30), EINVAL, "workspace is not 16-byte aligned"),
])
def test_evict_rejects(lib, kw, code, msg):
    assert evict(lib, **kw) == code
    assert msg in err(lib)


def test_workspace_sizes(lib):
    ws = gdr.attention_workspace_bytes
    assert ws(0, 1, 4, 2, 128, 4, 16) == 0
    assert ws(2, 0, 4, 2, 128, 4, 16) == 0
    assert ws(2, 1, 5, 2, 128, 4, 16) == 0
    assert ws(2, 1, 4, 2, 128, 4, 24) == 0
    assert ws(2, 1, 4, 2, 128, 0, 16) == 0
    big = 2 ** 31 - 1
    assert ws(big, big, big, 1, 128, 4, 16) == 0
    assert ws(1 << 30, 1 << 30, 16, 16, 128, 4, 16) == 0
    assert ws(2, 1, 4, 2, 128, big, 256) == 0
    # grows with the table where logits are kept for the scores
    assert ws(2, 1, 4, 2, 128, 64, 16, True) >= ws(2, 1, 4, 2, 128, 64, 16)


    # the selection by many workgroups: few pairs, long tables
    assert gdr.evict_workspace_bytes(2, 2, 4, 16) == 0
    assert gdr.evict_workspace_bytes(200, 2, 4000, 16) == 0
    assert gdr.evict_workspace_bytes(2, 2, 4000, 16) > 0
    assert gdr.evict_workspace_bytes(2, 2, big, 256) == 0


def test_binding_rejects_host_tensors():
    import torch
    c = torch.zeros(3, 2, 16, 64)
    t = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(gdr.GdrError, match="k_cache must be a GPU tensor"):
        gdr.attention_decode(torch.zeros(1, 1, 2, 64), c, c, t, t[:, 0])
    with pytest.raises(gdr.GdrError, match="scores are required"):
        gdr.cache_evict(c, c, None, t, t[:, 0], 4)
