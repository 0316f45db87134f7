"""GPU tests of the paged key-value cache at the edges of what its calls take:
tables without pages, slots longer than the page numbers a wave holds, more
sequences than are split, precision of the weights, tables past 2^31 pages."""
import numpy as np
import pytest
import torch

import gated_delta_rule_44_amd as gdr
from tests.conftest import gpu_available
from tests.gpu_util import announce

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
DEV = torch.device("cuda:0")
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
NAN = float("nan")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ------------------------------------------------------- tables without pages
# Nothing is attended to: zeros, and not a byte of the workspace (whose size is
# 0 then) or of the scores is written.
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("B,n,G", [(1, 1, 1), (5, 5, 4), (70, 10, 4), (300, 1, 2), (4096, 1, 1)])
@pytest.mark.parametrize("P,M", [(3, 0), (0, 0), (0, 4)])
def test_attend_no_pages(dt, scored, B, n, G, P, M):
    announce("attend without pages %s scores=%s B=%d n=%d G=%d P=%d M=%d" % (dt, scored, B, n, G, P, M))
    kc = torch.full((P, 2, 16, 64), NAN, device=DEV, dtype=DTYPES[dt])
    sc = torch.full((P, 2, 16), NAN, device=DEV) if scored else None
    q = torch.ones((B, n, 2 * G, 64), device=DEV, dtype=DTYPES[dt])
    o = torch.full_like(q, NAN)
    need = gdr.attention_workspace_bytes(B, n, 2 * G, 2, 64, M, 16, scored)
    if M == 0:
        assert need == 0
    guard = torch.full((need + (1 << 20),), 0xA5, device=DEV, dtype=torch.uint8)
    table = torch.zeros((B, M), device=DEV, dtype=torch.int32)
    lens = i32([7] * B)
    out = gdr.attention_decode(q, kc, kc.clone(), table, lens, scores=sc, o=o, workspace=guard)
    torch.cuda.synchronize(DEV)
    assert out is o and bool((o == 0).all())
    assert bool((guard == 0xA5).all()), "the workspace was written to"
    assert sc is None or bool(torch.isnan(sc).all())
    # the workspace that the call allocates for itself
    assert bool((gdr.attention_decode(q, kc, kc.clone(), table, lens, scores=sc) == 0).all())


@pytest.mark.parametrize("new", [False, True])
def test_evict_and_append_no_pages(new):
    """Nothing is kept, moved or written."""
    announce("evict, append without pages new=%s" % new)
    B, Hkv = 70, 2
    kc = torch.full((3, Hkv, 16, 64), NAN, device=DEV)
    sc = torch.full((3, Hkv, 16), NAN, device=DEV)
    table, lens = torch.zeros((B, 0), device=DEV, dtype=torch.int32), i32([9] * B)
    to = i32([[0]] * B) if new else None
    nl, kept = gdr.cache_evict(kc, kc.clone(), sc, table, lens, 5, 1, 1, new_page_table=to)
    k = torch.ones((B, 2, Hkv, 64), device=DEV)
    gdr.cache_append(k, k, lens, table, kc, kc.clone(), scores=sc)
    torch.cuda.synchronize(DEV)
    assert bool((nl == 0).all()) and bool((kept == -1).all())
    assert bool(torch.isnan(kc).all()) and bool(torch.isnan(sc).all())
