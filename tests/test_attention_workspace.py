"""CPU tests of the workspace of attention over the paged cache: a decode takes
buffers of the sizes below, whatever a tree of as many rows would ask for."""
import os

import pytest

import gated_delta_rule_44_amd as gdr
from tests import test_attention_abi as tree_abi, test_cache_abi as cache_abi

# B, n_tok, Hq, Hkv, D, max_pages, page_size, scores: a decode's bytes
SIZES = [
    ((4, 300, 32, 8, 128, 50, 64, 0), 50585856),
    ((16, 33, 64, 8, 128, 50, 64, 0), 54579456),
    ((16, 33, 64, 8, 128, 50, 64, 1), 487117056),
    ((2, 64, 64, 8, 128, 250, 64, 0), 17039616),
    ((80, 64, 8, 4, 64, 80, 64, 0), 28115712),
    ((300, 64, 4, 2, 64, 300, 16, 0), 37588224),
    ((3, 64, 64, 4, 128, 300, 16, 0), 34078976),
    ((64, 4, 32, 8, 128, 128, 64, 0), 17039872),
]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdr.lib_path()):
        pytest.skip("libgdr.so not built")
    return gdr._load()


@pytest.mark.parametrize("size,need", SIZES)
def test_decode_bytes(lib, size, need):
    B, n, Hq, Hkv, D, M, page, scores = size
    kw = dict(B=B, n=n, Hq=Hq, Hkv=Hkv, D=D, M=M, page=page, sc=cache_abi.FAKE if scores else None)
    # one too few of them: refused, with their number
    assert cache_abi.attend(lib, ws_bytes=need - 1, **kw) == cache_abi.EINVAL
    assert "workspace of %d bytes needed" % need in cache_abi.err(lib)
    got = gdr.attention_workspace_bytes(*size)
    if scores or n > 64:
        assert got == need
    else:
        # a tree's beside them: of one round of workgroups at most 34 MB, or no more
        assert need <= got <= max(need, 35 << 20)
        del kw["sc"]
        assert tree_abi.tree(lib, ws_bytes=got - 1, **kw) == cache_abi.EINVAL
        assert "workspace of %d bytes needed" % got in cache_abi.err(lib)


def test_backward_bytes_refuse_other_types(lib):
    torch = pytest.importorskip("torch")
    assert gdr.attention_backward_workspace_bytes(torch.bfloat16, 2, 600, 4, 2, 128) > 0
    with pytest.raises(gdr.GdrError, match="bfloat16 or float32"):
        gdr.attention_backward_workspace_bytes(torch.float16, 2, 600, 4, 2, 128)
