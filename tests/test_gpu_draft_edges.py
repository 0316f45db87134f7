"""GPU tests of trees of drafts and of the decode beside them at the edges of their
plans and values."""
import numpy as np
import pytest
import torch

import gated_delta_rule_44_amd as gdr
from tests import cache_ref, draft_ref as ref
from tests.conftest import gpu_available
from tests.gpu_util import announce
from tests.test_gpu_drafts import DEV, i32, make_cache, queries, same, sync, trees

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def check_some(o, q, kc, vc, table, lens, parents, scale, some, what):
    """The sequences `some` of a call against the reference."""
    want, bound = ref.attend(q[some], kc, vc, table[some], [lens[b] for b in some], parents[some],
                             scale)
    err = np.abs(o[some].double().cpu().numpy() - want)
    announce("  %s: worst error / bound %.3f" % (what, (err / np.maximum(bound, 1e-300)).max()))
    assert (err <= bound).all(), what


# (a decode's bytes at these sizes: what the call took before there were trees)
@pytest.mark.parametrize("B,n,Hkv,G,D,M,page,need", [
    (16, 33, 8, 8, 128, 50, 64, 54579456), (80, 64, 4, 2, 64, 80, 64, 28115712)])
def test_plans_of_many_rows(B, n, Hkv, G, D, M, page, need):
    """Past one round of workgroups a tree of over 64 rows a head has the slots that a
    decode's workspace holds, and a decode takes a buffer of that size: neither writes
    past it, long sequences lie over several slots, and a chain gives what a decode
    does."""
    announce("B=%d n=%d Hkv=%d G=%d D=%d" % (B, n, Hkv, G, D))
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 300, B)]
    long = [1, B // 2, B - 1]
    for b, x in zip(long, (M * page, 2500, 1300)):
        lens[b] = x
    kc, vc, _, table = make_cache(lens, Hkv, D, page, torch.bfloat16, seed=B, extra=0)
    table = np.pad(table, ((0, 0), (0, M - table.shape[1])), constant_values=-1)
    q = queries(B, n, Hkv * G, D, torch.bfloat16, seed=n)
    args = (q.to(DEV), kc.to(DEV), vc.to(DEV), i32(table), i32(lens))
    assert gdr.attention_workspace_bytes(B, n, Hkv * G, Hkv, D, M, page) == need
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    chain = np.tile(np.arange(n) - 1, (B, 1)).astype(np.int32)
    for what, parents in (("tree", trees(B, n, seed=3)), ("chain", chain)):
        o = gdr.attention_tree(*args, i32(parents), scale=D ** -0.5, workspace=ws[:need])
        sync()
        assert (ws[need:] == 0x5A).all(), what
        check_some(o, q, kc, vc, table, lens, parents, D ** -0.5, long[1:], what)
    d = gdr.attention_decode(*args, scale=D ** -0.5, workspace=ws[:need])
    sync()
    assert (ws[need:] == 0x5A).all()
    check_some(d, q, kc, vc, table, lens, chain, D ** -0.5, long[1:], "decode")
    # two results within a rounding of o and 2^-15 of the weights each
    assert torch.allclose(o.float(), d.float(), rtol=2 ** -7, atol=2 ** -13 * 4)
    with pytest.raises(gdr.GdrError, match="workspace"):
        gdr.attention_decode(*args, workspace=ws[:need - 16])


def test_decode_takes_its_own_bytes():
    """Where a tree of as many rows takes more, and past the 64 tokens of a tree."""
    for B, n, Hkv, G, M, page, need in ((2, 64, 8, 8, 250, 64, 17039616), (4, 300, 8, 4, 50, 64, 50585856)):
        lens = [M * page - 5] + [400] * (B - 1)
        kc, vc, _, table = make_cache(lens, Hkv, 128, page, torch.bfloat16, seed=n, extra=0)
        args = (queries(B, n, Hkv * G, 128, torch.bfloat16, n).to(DEV), kc.to(DEV), vc.to(DEV),
                i32(table), i32(lens))
        assert table.shape[1] == M
        ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        o = gdr.attention_decode(*args, workspace=ws[:need])
        sync()
        assert (ws[need:] == 0x5A).all()
        assert torch.equal(o, gdr.attention_decode(*args))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G,wide", [(8, 2, 0), (24, 1, 1), (40, 1, 1), (24, 4, 1), (64, 2, 1)])
def test_tree_large_values(D, n, G, wide):
    """Values below 2^128 / tokens give finite results, as in the decode, also where
    logits grow by a little under 8 ln 2 after the first tile and a maximum is left
    behind; in blocks of 16 to 128 rows."""
    L, page, Hkv = 500, 16, 2
    rng = np.random.default_rng(n)
    kc, vc, _, table = make_cache([L], Hkv, D, page, torch.bfloat16, seed=D,
                                  extra=wide * ((160 << 10) // (Hkv * page) + 100))
    v = torch.from_numpy(rng.choice([-1.0, 1.0], tuple(vc.shape))).bfloat16() * 2.0 ** 118
    v[..., 3] = 2.0 ** 118
    vc = torch.where(torch.isnan(vc), vc, v)
    k = torch.zeros_like(kc)
    for j in range(L):
        k[table[0, j // page], :, j % page, 0] = 0.0 if j < 64 else 5.5
    kc = torch.where(torch.isnan(kc), kc, k)
    q = torch.zeros((1, n, Hkv * G, D), dtype=torch.bfloat16)
    q[..., 0] = 8.0
    parents = trees(1, n, seed=1)
    o = gdr.attention_tree(q.to(DEV), kc.to(DEV), vc.to(DEV), i32(table), i32([L]), i32(parents),
                           scale=0.125)
    sync()
    assert bool(torch.isfinite(o).all())
    check_some(o, q, kc, vc, table, [L], parents, 0.125, [0], "n=%d G=%d" % (n, G))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_round_with_too_few_pages(dt):
    """A round of drafts in which some sequences get no pages: those that need none are
    served after them all the same, what is appended to the others falls on absent
    pages or past their lengths, and every sequence keeps its tokens."""
    B, Hkv, D, page, P, M, n = 5, 2, 64, 16, 12, 6, 4
    lens = [40, 32, 47, 20, 28]                  # 3 + 2 + 3 + 2 + 2 pages, all of them
    k0, v0, _, t0 = make_cache(lens, Hkv, D, page, dt, seed=3)
    kc, vc = (torch.full((P, Hkv, page, D), float("nan"), dtype=dt) for _ in range(2))
    full, at = np.full((B, M), -1, np.int32), np.random.default_rng(0).permutation(P).tolist()
    for b, l in enumerate(lens):
        for c in range(-(-l // page)):
            p = full[b, c] = at.pop()
            kc[p], vc[p] = k0[t0[b, c]], v0[t0[b, c]]
    dk, dv, tb, start = kc.to(DEV), vc.to(DEV), i32(full), i32(lens)
    held, free = gdr.cache_resize(tb, start, start + n, page, P)
    sync()
    served = [True, False, False, True, True]     # (the others lack a page each)
    assert held.tolist() == [l + n if s else l for l, s in zip(lens, served)] and free.item() == 0
    assert tb.cpu().numpy().tolist() == full.tolist()
    rng = np.random.default_rng(1)
    k, v = (torch.from_numpy(rng.standard_normal((B, n, Hkv, D))).to(dt) for _ in range(2))
    gdr.cache_append(k.to(DEV), v.to(DEV), start, tb, dk, dv)
    parents = trees(B, n, seed=2)
    q = queries(B, n, 2 * Hkv, D, dt, seed=5)
    o = gdr.attention_tree(q.to(DEV), dk, dv, tb, held, i32(parents), scale=0.125)
    ok = held == start + n
    ends, path = gdr.cache_accept(dk, dv, tb, held, i32(parents), torch.where(ok, n - 1, -1).int())
    ends = torch.where(ok, ends, start)
    last, free = gdr.cache_resize(tb, held, ends, page, P)
    sync()
    assert last.tolist() == ends.tolist() and free.item() == 0
    mine = tb.cpu().numpy()
    assert mine.tolist() == full.tolist()
    both = kc.clone(), vc.clone()
    for b in range(B):
        way = ref.way(parents[b], n - 1) if served[b] else []
        assert path[b].tolist() == way + [-1] * (n - len(way)) and ends[b] == lens[b] + len(way)
        for j in range(lens[b] + len(way)):
            p, s = cache_ref.place(mine, P, page, b, j)
            for x, y, z in ((dk, kc, k), (dv, vc, v)):
                assert same(x[p, :, s], y[p, :, s] if j < lens[b] else z[b, way[j - lens[b]]]), (b, j)
        if served[b]:
            for t in range(n):
                p, s = cache_ref.place(full, P, page, b, lens[b] + t)
                both[0][p, :, s], both[1][p, :, s] = k[b, t], v[b, t]
    some = [b for b in range(B) if served[b]]
    check_some(o, q, *both, full, [l + n for l in lens], parents, 0.125, some, "served")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G,wide", [(1, 1, 0), (8, 2, 0), (24, 1, 1), (20, 2, 1), (24, 4, 1), (64, 2, 1)])
def test_nan_that_a_row_attends_to(dt, D, n, G, wide):
    """NaN queries give NaN, in their rows only, and so do NaN keys, though they be all
    that a wave or a slot of a sequence sees; in trees and in the decode."""
    lens, page, Hkv = [2600, 300], 16, 2
    kc, vc, _, table = make_cache(lens, Hkv, D, page, dt, seed=D + n,
                                  extra=wide * ((160 << 10) // (Hkv * page) + 100))
    q = queries(2, n, Hkv * G, D, dt, seed=n)
    parents = trees(2, n, seed=2)
    chain = np.tile(np.arange(n) - 1, (2, 1)).astype(np.int32)

    def both(q, kc):
        args = (q.to(DEV), kc.to(DEV), vc.to(DEV), i32(table), i32(lens))
        out = [gdr.attention_tree(*args, i32(parents)), gdr.attention_tree(*args, i32(chain)),
               gdr.attention_decode(*args)]
        sync()
        return out

    clean = both(q, kc)
    mine = q.clone()
    mine[0, n - 1, 1, 3] = float("nan")
    for o, c in zip(both(mine, kc), clean):
        assert bool(torch.isnan(o[0, n - 1, 1]).all())
        o[0, n - 1, 1] = c[0, n - 1, 1]
        assert same(o, c)
    for places in (range(640, 1920), range(512, 1152), range(0, 128), range(2400, 2432)):
        mine = kc.clone()
        for j in places:
            mine[table[0, j // page], 0, j % page, 5] = float("nan")
        for o, c in zip(both(q, mine), clean):
            assert bool(torch.isnan(o[0, :, :G]).all()), places
            assert same(o[0, :, G:], c[0, :, G:]) and same(o[1], c[1]), places
