"""CPU tests of the C ABI in include/gdr_attention.h: every declared symbol is
exported, and bad arguments are rejected on the host before any HIP call
(nothing is launched here)."""
import ctypes
import os
import re

import numpy as np
import pytest

import gated_delta_rule_44_amd as gdr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdr_attention.h")
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


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gdr_[a-z_]+)\s*\(", src)))
    assert names == ["gdr_attention_backward", "gdr_attention_backward_workspace_bytes",
                     "gdr_attention_prefill", "gdr_attention_tree", "gdr_cache_accept",
                     "gdr_cache_resize"]
    for name in names:
        assert hasattr(ctypes.CDLL(gdr.lib_path()), name), name


def prefill(lib, dt=1, B=2, T=3, total=6, Hq=4, Hkv=2, D=128, scale=1.0, window=0, q=FAKE, k=FAKE,
            v=FAKE, cu=None, cu_host=None, o=FAKE, lse=None):
    return lib.gdr_attention_prefill(dt, B, T, total, Hq, Hkv, D, F(scale), window, q, k, v, cu,
                                     hp(cu_host), o, lse, None)


def backward(lib, dt=1, B=2, T=3, total=6, Hq=4, Hkv=2, D=128, scale=1.0, window=0, q=FAKE, k=FAKE,
             v=FAKE, cu=None, cu_host=None, o=FAKE, lse=FAKE, do=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
             ws=FAKE, ws_bytes=1 << 40):
    return lib.gdr_attention_backward(dt, B, T, total, Hq, Hkv, D, F(scale), window, q, k, v, cu,
                                      hp(cu_host), o, lse, do, dq, dk, dv, ws, ws_bytes, None)


PROMPTS = [
    (dict(dt=7), EINVAL, "dtype"),
    (dict(D=96), EUNSUPPORTED, "supported widths"),
    (dict(Hq=0), EINVAL, "bad sizes"),
    (dict(Hkv=0), EINVAL, "bad sizes"),
    (dict(Hq=5), EINVAL, "not a multiple"),
    (dict(scale=float("nan")), EINVAL, "scale"),
    (dict(scale=float("inf")), EINVAL, "scale"),
    (dict(window=-1), EINVAL, "window"),
    (dict(B=-1), EINVAL, "bad sizes"),
    (dict(T=-1), EINVAL, "bad sizes"),
    (dict(total=-1), EINVAL, "bad sizes"),
    (dict(total=7), EINVAL, "T_total = 7 but B * T = 6"),
    (dict(Hq=1 << 14), EUNSUPPORTED, "too wide"),
    (dict(B=1, T=1 << 30, total=1 << 30), EUNSUPPORTED, "too many"),
    (dict(B=1, T=1 << 25, total=1 << 25, Hq=64), EUNSUPPORTED, "too many"),
    (dict(B=1 << 24, T=1, total=1 << 24), EUNSUPPORTED, "too many"),
    (dict(B=1 << 23, total=64, cu=FAKE), EUNSUPPORTED, "too many"),
    (dict(q=None), EINVAL, "q is NULL"),
    (dict(k=MIS), EINVAL, "k is not 16-byte aligned"),
    (dict(v=None), EINVAL, "v is NULL"),
    (dict(o=MIS), EINVAL, "o is not 16-byte aligned"),
    (dict(lse=MIS), EINVAL, "lse is not 16-byte aligned"),
    (dict(cu=MIS), EINVAL, "cu_seqlens is not 4-byte aligned"),
    (dict(cu_host=[0, 3, 6]), EINVAL, "without cu_seqlens"),
    (dict(cu=FAKE, cu_host=[1, 3, 6]), EINVAL, "expected 0"),
    (dict(cu=FAKE, cu_host=[0, 4, 3]), EINVAL, "decreases"),
    (dict(cu=FAKE, cu_host=[0, 4, 7]), EINVAL, "cu_seqlens[B] = 7 but T_total = 6"),
]


@pytest.mark.parametrize("kw,code,msg", PROMPTS)
def test_prefill_rejects(lib, kw, code, msg):
    assert prefill(lib, **kw) == code
    assert msg in err(lib)


@pytest.mark.parametrize("kw,code,msg", PROMPTS + [
    (dict(lse=None), EINVAL, "lse is NULL"),
    (dict(do=None), EINVAL, "d_o is NULL"),
    (dict(dq=MIS), EINVAL, "dq is not 16-byte aligned"),
    (dict(dk=None), EINVAL, "dk is NULL"),
    (dict(dv=None), EINVAL, "dv is NULL"),
    (dict(ws=None), EINVAL, "workspace"),
    (dict(ws=MIS), EINVAL, "workspace"),
    (dict(ws_bytes=16), EINVAL, "workspace"),
])
def test_backward_rejects(lib, kw, code, msg):
    assert backward(lib, **kw) == code
    assert msg in err(lib)


@pytest.mark.parametrize("kw", [
    dict(B=1, T=1 << 29, total=1 << 29, Hq=1, Hkv=1, D=64),     # a row and a window: past 2^31
    dict(B=(1 << 22) - 128, total=64 * 128, cu=FAKE),            # keys in blocks of 64: 2^24
    dict(B=1, T=1 << 28, total=1 << 28),
])
def test_prompts_past_a_launch(lib, kw):
    for call in (prefill, backward):
        assert call(lib, **kw) == EUNSUPPORTED
        assert "too many" in err(lib)
        # a smaller batch fails at the next check
        assert call(lib, **{**kw, "B": 1, "T": 4096, "total": 4096, "cu": None, "q": None}) == EINVAL
        assert "q is NULL" in err(lib)
    assert lib.gdr_attention_backward_workspace_bytes(
        1, kw["B"], kw["total"], kw.get("Hq", 4), kw.get("Hkv", 2), kw.get("D", 128)) == 0


def test_empty_calls_are_ok_without_gpu(lib):
    for call in (prefill, backward):
        assert call(lib, B=0, T=0, total=0) == 0
        assert call(lib, B=0, T=5, total=0, q=None) == 0
        assert call(lib, B=3, T=0, total=0, q=None) == 0
        assert call(lib, B=3, total=0, cu=FAKE, q=None) == 0


def test_workspace_sizes(lib):
    ws = lib.gdr_attention_backward_workspace_bytes
    assert ws(1, 2, 600, 4, 2, 128) >= 2 * 600 * 4 * 4
    assert ws(1, 0, 600, 4, 2, 128) == 0
    assert ws(1, 2, 0, 4, 2, 128) == 0
    assert ws(1, 2, 600, 5, 2, 128) == 0
    assert ws(1, 2, 600, 4, 2, 96) == 0
    assert ws(5, 2, 600, 4, 2, 128) == 0
    big = 2 ** 31 - 1
    assert ws(1, big, big, big, big, 128) == 0


def test_binding_rejects_host_tensors():
    import torch
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(gdr.GdrError, match="q must be a GPU tensor"):
        gdr.attention_prefill(q, q, q)
    with pytest.raises(gdr.GdrError, match="q must be a GPU tensor"):
        gdr.attention_backward(q, q, q, q, q, q)


def tree(lib, dt=1, B=2, n=3, Hq=4, Hkv=2, D=128, scale=1.0, window=0, q=FAKE, kc=FAKE, vc=FAKE,
         table=FAKE, host=None, M=4, page=16, P=9, lens=FAKE, parents=FAKE, o=FAKE, ws=FAKE,
         ws_bytes=1 << 40):
    return lib.gdr_attention_tree(dt, B, n, Hq, Hkv, D, F(scale), window, q, kc, vc, table, hp(host),
                                  M, page, P, lens, parents, o, ws, ws_bytes, None)


def accept(lib, dt=1, B=2, n=3, Hkv=2, D=128, table=FAKE, M=4, page=16, P=9, lens=FAKE,
           parents=FAKE, leaf=FAKE, kc=FAKE, vc=FAKE, sc=None, new_lens=FAKE, path=FAKE):
    return lib.gdr_cache_accept(dt, B, n, Hkv, D, table, M, page, P, lens, parents, leaf, kc, vc, sc,
                                new_lens, path, None)


def resize(lib, B=2, M=4, page=16, P=9, table=FAKE, lens=FAKE, want=FAKE, new_lens=FAKE, cu=None,
           free=None):
    return lib.gdr_cache_resize(B, M, page, P, table, lens, want, new_lens, cu, free, None)


CACHE = [
    (dict(dt=5), EINVAL, "dtype"),
    (dict(D=96), EUNSUPPORTED, "supported widths"),
    (dict(B=-1), EINVAL, "bad sizes"),
    (dict(Hkv=0), EINVAL, "bad sizes"),
    (dict(M=-1), EINVAL, "bad sizes"),
    (dict(P=-1), EINVAL, "bad sizes"),
    (dict(page=8), EUNSUPPORTED, "page_size"),
    (dict(M=1 << 22, page=256), EUNSUPPORTED, "too long"),
    (dict(P=1 << 30), EUNSUPPORTED, "too large"),
    (dict(n=-1), EINVAL, "-1 drafts"),
    (dict(n=65), EUNSUPPORTED, "65 drafts; 0 to 64"),
    (dict(table=None), EINVAL, "page_table is NULL"),
    (dict(table=MIS), EINVAL, "page_table is not 4-byte aligned"),
    (dict(kc=None), EINVAL, "k_cache is NULL"),
    (dict(vc=MIS), EINVAL, "v_cache is not 16-byte aligned"),
    (dict(lens=None), EINVAL, "seq_lens is NULL"),
    (dict(parents=MIS), EINVAL, "parents is not 4-byte aligned"),
]


@pytest.mark.parametrize("kw,code,msg", CACHE + [
    (dict(Hq=5), EINVAL, "not a multiple"),
    (dict(scale=float("nan")), EINVAL, "scale"),
    (dict(window=-1), EINVAL, "window"),
    (dict(B=1 << 17, n=64), EUNSUPPORTED, "query rows"),
    (dict(q=None), EINVAL, "q is NULL"),
    (dict(o=MIS), EINVAL, "o is not 16-byte aligned"),
    (dict(ws=None), EINVAL, "workspace"),
    (dict(ws_bytes=1), EINVAL, "workspace"),
    (dict(host=[[0, 1, 2, 9], [3, 4, 5, -1]]), EINVAL, "page_table[0, 3] = 9 outside -1..8"),
])
def test_tree_rejects(lib, kw, code, msg):
    assert tree(lib, **kw) == code
    assert msg in err(lib)


@pytest.mark.parametrize("kw,code,msg", CACHE + [
    (dict(sc=MIS), EINVAL, "scores is not 16-byte aligned"),
    (dict(B=1 << 20), EUNSUPPORTED, "pairs exceed"),
    (dict(leaf=None), EINVAL, "leaf is NULL"),
    (dict(new_lens=None), EINVAL, "new_lens is NULL"),
    (dict(path=MIS), EINVAL, "path is not 4-byte aligned"),
])
def test_accept_rejects(lib, kw, code, msg):
    assert accept(lib, **kw) == code
    assert msg in err(lib)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(B=-1), EINVAL, "bad sizes"),
    (dict(M=-1), EINVAL, "bad sizes"),
    (dict(page=0), EINVAL, "bad sizes"),
    (dict(P=-1), EINVAL, "bad sizes"),
    (dict(P=(1 << 20) + 1), EUNSUPPORTED, "pages exceed"),
    (dict(M=1 << 26), EUNSUPPORTED, "too long"),
    (dict(P=1 << 20, page=1 << 11, M=2), EUNSUPPORTED, "too many"),
    (dict(B=1 << 30), EUNSUPPORTED, "too many"),
    (dict(table=None), EINVAL, "page_table is NULL"),
    (dict(lens=MIS), EINVAL, "seq_lens is not 4-byte aligned"),
    (dict(want=None), EINVAL, "want is NULL"),
    (dict(new_lens=None), EINVAL, "new_lens is NULL"),
    (dict(cu=MIS), EINVAL, "cu_seqlens is not 4-byte aligned"),
    (dict(free=MIS), EINVAL, "free_pages is not 4-byte aligned"),
])
def test_resize_rejects(lib, kw, code, msg):
    assert resize(lib, **kw) == code
    assert msg in err(lib)


def test_empty_draft_calls_are_ok_without_gpu(lib):
    assert tree(lib, B=0) == 0
    assert tree(lib, n=0) == 0
    assert accept(lib, B=0) == 0
    assert resize(lib, B=0, table=None, lens=None) == 0
