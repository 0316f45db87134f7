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
    assert "gdr_attention_prefill" in names and "gdr_attention_backward" in names
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
