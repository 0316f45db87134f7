"""GPU tests of trees of drafts over the paged cache, of what is kept of them and
of the page tables, against their reference (tests/draft_ref.py), and a run of
them together with the calls beside them."""
import numpy as np
import pytest
import torch

import gated_delta_rule_44_amd as gdr
from tests import cache_ref, draft_ref as ref, prompt_ref
from tests.conftest import gpu_available
from tests.gpu_util import announce

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
DEV = torch.device("cuda:0")
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
NAN, INF = float("nan"), float("inf")


def sync():
    torch.cuda.synchronize(DEV)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def same(a, b):
    """Equal bit for bit (NaN included)."""
    a, b = a.detach().cpu().contiguous(), b.detach().cpu().contiguous()
    kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.shape == b.shape and torch.equal(a.view(kind), b.view(kind))


def make_cache(lens, Hkv, D, page, dt, seed, extra=1):
    """Caches (CPU) of lens[b] tokens on shuffled pages, NaN everywhere else."""
    rng = np.random.default_rng(seed)
    need = [-(-l // page) for l in lens]
    P, M = sum(need) + 2, max(need + [0]) + extra
    pages = rng.permutation(P)
    table = np.full((len(lens), M), -1, np.int32)
    kc = torch.full((P, Hkv, page, D), NAN, dtype=dt)
    vc, sc = kc.clone(), torch.full((P, Hkv, page), NAN)
    at = 0
    for b, (l, c) in enumerate(zip(lens, need)):
        table[b, :c] = pages[at:at + c]
        at += c
        for i in range(c):
            m, p = min(page, l - i * page), table[b, i]
            kc[p, :, :m] = torch.from_numpy(rng.standard_normal((Hkv, m, D))).to(dt)
            vc[p, :, :m] = torch.from_numpy(rng.standard_normal((Hkv, m, D))).to(dt)
            sc[p, :, :m] = torch.from_numpy(rng.random((Hkv, m))).float()
    return kc, vc, sc, table


def trees(B, n, seed):
    """Chains, stars and trees in between."""
    rng = np.random.default_rng(seed)
    p = np.full((B, n), -1, np.int32)
    for b in range(B):
        for t in range(1, n):
            p[b, t] = (t - 1, -1, rng.integers(-1, t), max(-1, t - 1 - rng.integers(0, 4)))[b % 4]
    return p


def queries(B, n, Hq, D, dt, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(2.0 * rng.standard_normal((B, n, Hq, D))).to(dt)


def empty_beside(table, page, Hkv, rows, n, window):
    """How many empty sequences beside these make a bf16 call one with much to
    read: over 160 K (token, head, block of 16 rows)."""
    cap = table.shape[1] * page
    seen = window + n if window and window + n < cap else cap
    return (160 << 10) // (seen * Hkv * -(-rows // 16)) + 1


def call_tree(q, kc, vc, table, lens, parents, scale, window=0, empty=0, **kw):
    """attention_tree of these sequences, and of `empty` empty ones, first and
    last."""
    B, first = len(lens), empty // 2
    rest = empty - first
    q = torch.cat([q.new_ones(first, *q.shape[1:]), q, q.new_ones(rest, *q.shape[1:])])
    table, parents = (np.pad(x, ((first, rest), (0, 0)), constant_values=-1)
                      for x in (table, np.asarray(parents)))
    lens = [0] * first + list(lens) + [0] * rest
    o = gdr.attention_tree(q.to(DEV), kc.to(DEV), vc.to(DEV), i32(table), i32(lens), i32(parents),
                           scale=scale, window=window, **kw)
    sync()
    assert not o[:first].any() and not o[first + B:].any()
    return o[first:first + B]


def check_tree(q, kc, vc, table, lens, parents, scale, window=0, what="", empty=0, **kw):
    dk, dv = kc.to(DEV), vc.to(DEV)
    o = call_tree(q, dk, dv, table, lens, parents, scale, window, empty, **kw)
    want, bound = ref.attend(q, kc, vc, table, lens, parents, scale, window)
    err = np.abs(o.double().cpu().numpy() - want)
    ratio = (err / np.maximum(bound, 1e-300)).max() if err.size else 0
    announce("  %s: worst error / bound %.3f" % (what, ratio))
    assert (err <= bound).all(), "%s: at %s" % (what, np.argwhere(~(err <= bound))[:4].tolist())
    assert same(dk, kc) and same(dv, vc), "%s: the cache changed" % what
    return o


LENS = [64, 0, 17, 3, 63, 65, 130, 200, 1]
SHAPES = [
    # D, page, Hkv, G, n, window
    (128, 16, 2, 4, 1, 0),
    (128, 64, 2, 4, 7, 0),
    (64, 16, 3, 1, 8, 0),
    (64, 32, 2, 7, 5, 0),
    (128, 256, 1, 3, 24, 0),
    (128, 16, 1, 2, 33, 0),
    (64, 128, 2, 1, 64, 0),
    (128, 32, 1, 5, 64, 0),
    (128, 16, 2, 4, 7, 1),
    (64, 32, 1, 2, 16, 3),
    (128, 64, 2, 4, 24, 33),
    (64, 16, 1, 1, 64, 20),
    (64, 64, 1, 2, 64, 100),
]


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D,page,Hkv,G,n,window", SHAPES)
def test_tree(dt, D, page, Hkv, G, n, window):
    announce("tree %s D=%d page=%d Hkv=%d G=%d n=%d window=%d" % (dt, D, page, Hkv, G, n, window))
    kc, vc, _, table = make_cache(LENS, Hkv, D, page, DTYPES[dt], seed=D + n)
    q = queries(len(LENS), n, Hkv * G, D, DTYPES[dt], seed=n)
    parents = trees(len(LENS), n, seed=n + 1)
    args = (q, kc, vc, table, LENS, parents, D ** -0.5, window)
    o = check_tree(*args, what="tree")
    assert torch.equal(o, check_tree(*args, what="again", page_table_host=table))
    # an absent page in the context, one under the drafts
    for b, l in ((7, 200), (6, 130)):
        table[b, (l - 1) // page if b == 6 else 0] = -1
    check_tree(*args, what="absent")


@pytest.mark.parametrize("D,page,Hkv,G,n,window", [x for x in SHAPES if x[3] * x[4] > 16] + [
    (64, 16, 2, 4, 24, 0), (128, 16, 3, 2, 64, 7), (64, 32, 1, 5, 64, 40), (128, 128, 2, 2, 10, 0)])
def test_tree_much_to_read(D, page, Hkv, G, n, window):
    """The blocks of 32 to 128 rows, which bf16 calls take with much to read."""
    announce("much: D=%d page=%d Hkv=%d G=%d n=%d window=%d" % (D, page, Hkv, G, n, window))
    kc, vc, _, table = make_cache(LENS, Hkv, D, page, torch.bfloat16, seed=D + n)
    q = queries(len(LENS), n, Hkv * G, D, torch.bfloat16, seed=n)
    parents = trees(len(LENS), n, seed=n + 1)
    empty = empty_beside(table, page, Hkv, n * G, n, window)
    args = (q, kc, vc, table, LENS, parents, D ** -0.5, window)
    check_tree(*args, what="much", empty=empty)
    for b, l in ((7, 200), (6, 130)):
        table[b, (l - 1) // page if b == 6 else 0] = -1
    check_tree(*args, what="absent", empty=empty)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_chain_is_decode(dt):
    """A chain gives attention_decode's bits where both take blocks of 16 rows
    (without a window, whose first tile the two choose differently), and what its
    definition says elsewhere."""
    for D, page, G, n, window in ((128, 16, 4, 4, 0), (64, 64, 2, 16, 0), (128, 32, 1, 30, 0)):
        kc, vc, _, table = make_cache(LENS, 2, D, page, DTYPES[dt], seed=n)
        q = queries(len(LENS), n, 2 * G, D, DTYPES[dt], seed=n)
        chain = np.tile(np.arange(n) - 1, (len(LENS), 1))
        args = (q.to(DEV), kc.to(DEV), vc.to(DEV), i32(table), i32(LENS))
        a = gdr.attention_decode(*args, scale=0.1, window=window)
        b = check_tree(q, kc, vc, table, LENS, chain, 0.1, window, what="chain")
        if dt == "fp32" or n * G <= 16:
            assert torch.equal(a, b)
        else:        # two results within a rounding of o and 2^-15 of the weights each
            assert torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=2 ** -13 * 4)


def test_tree_many_rows_long_table():
    """Blocks of 64 rows (a table for many tokens), and many slots of a sequence."""
    lens = [33, 700, 65, 3000]
    for D, page, n, G, window in ((128, 32, 24, 4, 0), (64, 16, 64, 2, 0), (128, 64, 40, 2, 500)):
        kc, vc, _, table = make_cache(lens, 2, D, page, torch.bfloat16, seed=n,
                                      extra=(48 << 20) // (len(lens) * 2 * D * page))
        check_tree(queries(4, n, 2 * G, D, torch.bfloat16, n), kc, vc, table, lens, trees(4, n, n),
                   D ** -0.5, window, what="rows")


def test_tree_many_sequences():
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 40, 700)]
    kc, vc, _, table = make_cache(lens, 1, 64, 16, torch.bfloat16, seed=4)
    check_tree(queries(700, 5, 2, 64, torch.bfloat16, 5), kc, vc, table, lens, trees(700, 5, 6),
               0.125, what="700 sequences")


@pytest.mark.parametrize("n,G", [(2, 1), (33, 2)])
def test_tree_65536_sequences(n, G):
    """So many that each is one slot, one more than a table of slots holds."""
    lens = [40, 0, 70, 33, 5]
    kc, vc, _, table = make_cache(lens, 1, 64, 16, torch.bfloat16, seed=11)
    check_tree(queries(5, n, G, 64, torch.bfloat16, 12), kc, vc, table, lens, trees(5, n, 13), 0.125,
               what="65,537 sequences", empty=65532)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_tree_without_pages(dt):
    """No columns, or no pages: every token is absent, o is 0, and the workspace
    that the call asks for is not exceeded."""
    for P, M in ((0, 4), (3, 0), (0, 0)):
        kc = torch.full((P, 2, 16, 64), NAN, dtype=DTYPES[dt], device=DEV)
        table = torch.zeros(3, M, dtype=torch.int32, device=DEV)
        q = torch.ones(3, 24, 8, 64, dtype=DTYPES[dt], device=DEV)
        need = gdr.attention_workspace_bytes(3, 24, 8, 2, 64, M, 16)
        ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
        o = gdr.attention_tree(q, kc, kc, table, i32([24, 50, 1]), i32(trees(3, 24, 1)),
                               o=torch.full_like(q, NAN), workspace=ws[:need])
        sync()
        assert not o.any() and (ws[need:] == 0x5A).all()


@pytest.mark.parametrize("D", [64, 128])
def test_tree_workspace_is_enough(D):
    """Nothing is written past the bytes that the library asks for, in any of the
    blocks."""
    lens, Hkv, page = [900, 0, 33, 700], 2, 32
    kc, vc, _, table = make_cache(lens, Hkv, D, page, torch.bfloat16, seed=D)
    for n, G in ((8, 4), (24, 2), (24, 4), (64, 2), (40, 4)):
        q = queries(4, n, Hkv * G, D, torch.bfloat16, n)
        for extra in (0, 100 + (160 << 10) // (4 * Hkv * page)):
            wide = np.pad(table, ((0, 0), (0, extra)), constant_values=-1)
            need = gdr.attention_workspace_bytes(4, n, Hkv * G, Hkv, D, wide.shape[1], page)
            ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
            check_tree(q, kc, vc, wide, lens, trees(4, n, n), D ** -0.5, what="%d x %d" % (n, G),
                       workspace=ws[:need])
            assert (ws[need:] == 0x5A).all(), (n, G, extra)


def test_tree_bad_parents():
    """Values that are no earlier draft mean the context."""
    lens = [40, 40, 40]
    kc, vc, _, table = make_cache(lens, 1, 64, 16, torch.float32, seed=7)
    parents = np.array([[0, 1, 5, 2], [-7, 1 << 30, -(1 << 31), 3], [2, 0, 1, 64]], np.int64)
    check_tree(queries(3, 4, 2, 64, torch.float32, 8), kc, vc, table, lens,
               parents.astype(np.int32), 0.125, what="bad parents")


def check_masked_values(dt, G, D, much):
    lens, n, window = [100, 90], 6, 30
    kc, vc, _, table = make_cache(lens, 2, D, 16, DTYPES[dt], seed=9)
    q = queries(2, n, 2 * G, D, DTYPES[dt], 10)
    parents = np.array([[-1, 0, 0, 1, 2, 3]] * 2)
    empty = empty_beside(table, 16, 2, n * G, n, window) if much else 0
    args = (table, lens, parents, 0.125, window)
    clean = check_tree(q, kc, vc, *args, what="clean", empty=empty)
    for x in (NAN, INF, -INF):
        for j, rows in ((100 - n + 2, [2, 4]), (100 - n - 30, []), (100 - n - 28, [0, 1, 2])):
            bad = vc.clone()
            p, s = cache_ref.place(table, kc.shape[0], 16, 0, j)
            bad[p, :, s, 5] = x
            o = call_tree(q, kc, bad, *args, empty=empty)
            want = clean.clone()
            want[0, rows, :, 5] = x
            got, want = (torch.nan_to_num(y, 12345.0) for y in (o, want))
            assert same(got, want), (x, j, (got != want).nonzero()[:4].tolist())


@pytest.mark.parametrize("dt,G", [("fp32", 2), ("bf16", 2), ("bf16", 8), ("bf16", 14), ("bf16", 20),
                                  ("bf16", 40)])
def test_tree_masked_values(dt, G):
    """Infinities and NaN of drafts on other ways and of tokens outside the
    window have no part in a row; on its own way they have."""
    check_masked_values(dt, G, 64, False)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [4, 8, 14, 20, 40])
def test_tree_masked_values_much_to_read(G, D):
    """The same in the blocks of 32 to 128 rows."""
    check_masked_values("bf16", G, D, True)


# ------------------------------------------------------------------- accept

def check_accept(kc, vc, sc, table, lens, parents, leaf, what="", in_place=False):
    dk, dv = kc.to(DEV), vc.to(DEV)
    ds = None if sc is None else sc.to(DEV)
    dl = i32(lens)
    new, path = gdr.cache_accept(dk, dv, i32(table), dl, i32(parents), i32(leaf), scores=ds,
                                 new_lens=dl if in_place else None)
    sync()
    want = ref.accept(kc, vc, table, lens, parents, leaf, sc)
    assert same(dk, want[0]) and same(dv, want[1]), "%s: the cache" % what
    assert sc is None or same(ds, want[2]), "%s: scores" % what
    assert new.tolist() == want[3].tolist(), what
    assert path.tolist() == want[4].tolist(), what


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D,page,Hkv,n", [(128, 16, 2, 1), (64, 16, 3, 7), (128, 64, 1, 24),
                                          (128, 32, 2, 64), (64, 256, 2, 64), (64, 16, 1, 33)])
def test_accept(dt, D, page, Hkv, n):
    announce("accept %s D=%d page=%d Hkv=%d n=%d" % (dt, D, page, Hkv, n))
    lens = LENS + [n, n + 1, n + page, 3 * page]
    B = len(lens)
    kc, vc, sc, table = make_cache(lens, Hkv, D, page, DTYPES[dt], seed=n)
    parents = trees(B, n, seed=n)
    rng = np.random.default_rng(n)
    for leaf in (np.full(B, n - 1), np.full(B, -1), rng.integers(0, n, B), np.full(B, n),
                 rng.integers(-2, n + 3, B)):
        check_accept(kc, vc, sc, table, lens, parents, leaf, "leaf %s" % leaf[:3])
        check_accept(kc, vc, None, table, lens, parents, leaf, "in place", in_place=True)
    parents[:, n // 2] = n - 1                       # no earlier draft: the context
    table[7, 0] = table[6, (130 - 1) // page] = -1
    check_accept(kc, vc, sc, table, lens, parents, np.full(B, n - 1), "absent pages")


def test_accept_none():
    kc, vc, sc, table = make_cache([5, 9], 2, 64, 16, torch.float32, seed=1)
    check_accept(kc, vc, sc, table, [5, 9], np.zeros((2, 0), np.int32), [0, 0], "no drafts")
    check_accept(kc, vc, sc, table[:0], [], np.zeros((0, 3), np.int32), [], "no sequences")


# ------------------------------------------------------------------- resize

def check_resize(table, lens, want, page, pages, what="", alias=None):
    dt, dl, dw = i32(table).view(table.shape), i32(lens), i32(want)
    B = len(lens)
    guard = torch.full((B + 1 + 8,), 77, dtype=torch.int32, device=DEV)
    cu = guard[4:4 + B + 1]
    new, free = gdr.cache_resize(dt, dl, dw, page, pages, cu_seqlens=cu,
                                 new_lens={"lens": dl, "want": dw}.get(alias))
    sync()
    x = ref.resize(table, lens, want, page, pages)
    assert dt.cpu().numpy().tolist() == x[0].tolist(), "%s: the table" % what
    assert new.tolist() == x[1].tolist() and cu.tolist() == x[2].tolist(), what
    assert free.tolist() == [x[3]], what
    assert (guard[:4] == 77).all() and (guard[4 + B + 1:] == 77).all()
    return x


@pytest.mark.parametrize("B,M,page,pages,fill", [
    (1, 1, 16, 1, 1.0), (4, 5, 16, 30, 0.5), (7, 70, 1, 300, 0.6), (300, 9, 64, 1500, 0.5),
    (1500, 4, 16, 4000, 0.6), (33, 200, 16, 3000, 0.4), (64, 130, 7, 100000, 0.9),
    (5, 40, 256, 1 << 20, 0.5), (1025, 1, 1, 700, 0.5)])
def test_resize(B, M, page, pages, fill):
    announce("resize B=%d M=%d page=%d pages=%d" % (B, M, page, pages))
    rng = np.random.default_rng(B + M)
    table = np.full((B, M), -1, np.int32)
    lens = rng.integers(0, int(M * page * fill) + 1, B)
    have = -(-lens // page)
    while have.sum() > pages:
        b = int(have.argmax())
        lens[b] = lens[b] // 2
        have[b] = -(-lens[b] // page)
    at = rng.permutation(pages)[:have.sum()]
    for b in range(B):
        table[b, :have[b]], at = at[:have[b]], at[have[b]:]
    for step in range(3):
        want = rng.integers(0, M * page + 1, B)
        still = rng.random(B) < 0.6
        want[still] = np.minimum(lens[still] + rng.integers(0, 2 * page + 1, still.sum()), M * page)
        table, lens, _, _ = check_resize(table, lens, want, page, pages, "step %d" % step,
                                         (None, "lens", "want")[step])


def test_resize_odd_tables():
    # shared pages stay while one row keeps them; entries outside the pages are absent
    table = np.array([[0, 1, 2], [0, 1, 3], [9, -5, 4], [1 << 30, 6, -(1 << 31)]], np.int64)
    table = table.astype(np.int32)
    check_resize(table, [48, 48, 48, 48], [16, 48, 10, 48], 16, 8, "shared")
    check_resize(table, [48, 48, 48, 48], [0, 0, 0, 48], 16, 8, "none kept")
    check_resize(table, [-5, 1 << 30, 48, 20], [1 << 30, -7, 48, 48], 16, 8, "lengths out of range")
    check_resize(table, [16, 0, 0, 0], [16, 0, 0, 0], 16, 0, "no pages")
    check_resize(table, [16, 0, 0, 0], [48, 1, 0, 0], 16, 0, "no pages to give")
    check_resize(table[:0], [], [], 16, 8, "no rows")
    check_resize(np.zeros((3, 0), np.int32), [0, 5, 0], [3, 0, 0], 16, 8, "no columns")


def test_resize_repeats():
    """The same call again gives the same tables: what it takes for held are the
    columns of the old lengths."""
    table = np.array([[5, -1, -1], [2, 3, -1], [-1, -1, -1]], np.int32)
    x = ref.resize(table, [10, 20, 0], [40, 3, 16], 16, 6)
    y = ref.resize(x[0], [10, 20, 0], [40, 3, 16], 16, 6)
    assert x[0].tolist() == y[0].tolist()
    check_resize(x[0], [10, 20, 0], [40, 3, 16], 16, 6, "again")


def test_refuses():
    kc = torch.zeros(4, 2, 16, 64, device=DEV)
    t = i32([[0, 1], [2, 3]])
    q, lens, par = torch.zeros(2, 3, 4, 64, device=DEV), i32([9, 20]), i32([[-1, 0, 0]] * 2)
    many = torch.zeros(2, 65, 4, 64, device=DEV)
    for f, msg in [
        (lambda: gdr.attention_tree(many, kc, kc, t, lens, i32(np.zeros((2, 65)))), "65 drafts"),
        (lambda: gdr.attention_tree(q, kc, kc, t, lens, par.long()), "parents must be"),
        (lambda: gdr.attention_tree(q, kc, kc, t, lens, par[:, :2].contiguous()), "parents must be"),
        (lambda: gdr.attention_tree(q, kc, kc, t, lens, par.cpu()), "parents must be"),
        (lambda: gdr.attention_tree(q.bfloat16(), kc, kc, t, lens, par), "q must be"),
        (lambda: gdr.attention_tree(q, kc, kc, t, lens, par, window=-2), "window"),
        (lambda: gdr.attention_tree(q, kc, kc, t, lens, par, page_table_host=[[0, 1], [2, 4]]),
         "outside"),
        (lambda: gdr.cache_accept(kc, kc, t, lens, par, i32([0])), "leaf must be"),
        (lambda: gdr.cache_accept(kc, kc, t, lens, par[:1].contiguous(), i32([0, 0])), "parents must"),
        (lambda: gdr.cache_accept(kc, kc, t, lens, i32(np.zeros((2, 65))), i32([0, 0])), "65 drafts"),
        (lambda: gdr.cache_resize(t, lens, i32([1]), 16, 4), "want must be"),
        (lambda: gdr.cache_resize(t, lens, lens, 0, 4), "page_size"),
        (lambda: gdr.cache_resize(t, lens, lens, 16, -1), "num_pages"),
        (lambda: gdr.cache_resize(t, lens, lens, 16, (1 << 20) + 1), "exceed"),
        (lambda: gdr.cache_resize(t, lens, lens, 16, 4, cu_seqlens=i32([0, 0])), "cu_seqlens must"),
        (lambda: gdr.cache_resize(t.t(), lens, lens, 16, 4), "contiguous"),
    ]:
        with pytest.raises(gdr.GdrError, match=msg):
            f()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_serving_run(dt):
    """Prompts into fresh pages, then rounds of drafted trees: every table,
    length and offset is made on the GPU, and the last round's attention is
    that of the whole kept sequences."""
    dt = DTYPES[dt]
    rng = np.random.default_rng(42)
    B, Hkv, G, D, page, P, M, n = 4, 2, 2, 64, 16, 40, 12, 9
    r = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dt).to(DEV)  # noqa: E731
    kc, vc = (torch.full((P, Hkv, page, D), NAN, device=DEV, dtype=dt) for _ in range(2))
    table = torch.full((B, M), -1, device=DEV, dtype=torch.int32)
    lens, cu = torch.zeros(B, device=DEV, dtype=torch.int32), i32([0] * (B + 1))
    prompts = [50, 1, 33, 70]
    # what the sequences hold, kept beside
    ks, vs = [[] for _ in range(B)], [[] for _ in range(B)]
    new, free = gdr.cache_resize(table, lens, i32(prompts), page, P, cu_seqlens=cu)
    sync()
    assert new.tolist() == prompts and cu.tolist() == [0, 50, 51, 84, 154]
    assert free.item() == P - sum(-(-x // page) for x in prompts)
    q, k, v = r(154, Hkv * G, D), r(154, Hkv, D), r(154, Hkv, D)
    o, lse = gdr.attention_prefill(q, k, v, cu_seqlens=cu, lse=True)
    gdr.cache_append(k, v, lens, table, kc, vc, cu_seqlens=cu)
    lens = new
    sync()
    at = cu.tolist()
    for b in range(B):
        ks[b] += list(k[at[b]:at[b + 1]].cpu())
        vs[b] += list(v[at[b]:at[b + 1]].cpu())
    want = prompt_ref.forward(q.cpu(), k.cpu(), v.cpu(), at, D ** -0.5)
    assert ((o.double().cpu() - want[0]).abs() <= want[2]).all()
    # the prompts' last rows are a decode over the cache
    last = torch.stack([q[at[b + 1] - 1] for b in range(B)])[:, None].contiguous()
    o1 = gdr.attention_decode(last, kc, vc, table, lens)
    sync()
    for b in range(B):
        i = at[b + 1] - 1
        assert ((o1[b, 0].double().cpu() - want[0][i]).abs() <= want[2][i]).all()
    for step in range(3):
        parents = trees(B, n, seed=step)
        new, _ = gdr.cache_resize(table, lens, lens + n, page, P)
        k, v, q = r(B, n, Hkv, D), r(B, n, Hkv, D), r(B, n, Hkv * G, D)
        gdr.cache_append(k, v, lens, table, kc, vc)
        o = gdr.attention_tree(q, kc, vc, table, new, i32(parents))
        leaf = rng.integers(-1, n, B)
        kept, path = gdr.cache_accept(kc, vc, table, new, i32(parents), i32(leaf))
        sync()
        for b in range(B):
            # a draft's row: the sequence so far and its way as one prompt
            c = len(ks[b])
            for t in (0, n - 1, int(leaf[b])):
                if t < 0:
                    continue
                w = ref.way(parents[b], t)
                kk = torch.stack(ks[b] + [k[b, u].cpu() for u in w])
                vv = torch.stack(vs[b] + [v[b, u].cpu() for u in w])
                qq = torch.zeros(c + len(w), Hkv * G, D, dtype=dt)
                qq[-1] = q[b, t].cpu()
                y = prompt_ref.forward(qq, kk, vv, [0, c + len(w)], D ** -0.5)
                assert ((o[b, t].double().cpu() - y[0][-1]).abs() <= y[2][-1]).all(), (step, b, t)
            w = ref.way(parents[b], int(leaf[b])) if leaf[b] >= 0 else []
            assert path[b].tolist() == w + [-1] * (n - len(w))
            ks[b] += [k[b, u].cpu() for u in w]
            vs[b] += [v[b, u].cpu() for u in w]
        assert kept.tolist() == [len(x) for x in ks]
        lens, _ = gdr.cache_resize(table, new, kept, page, P)
        sync()
        assert lens.tolist() == kept.tolist()
    host = table.cpu().numpy()
    for b in range(B):
        for j in range(len(ks[b])):
            p, s = cache_ref.place(host, P, page, b, j)
            assert same(kc[p, :, s], ks[b][j]) and same(vc[p, :, s], vs[b][j])
    # the sequences end: every page is free again
    _, free = gdr.cache_resize(table, lens, torch.zeros_like(lens), page, P)
    assert free.item() == P and (table == -1).all()


def test_slot_map():
    """A table of one column as the slot map of a state pool."""
    B, H, D = 4, 2, 64
    slot = torch.full((B, 1), -1, device=DEV, dtype=torch.int32)
    lens = torch.zeros(B, device=DEV, dtype=torch.int32)
    lens, free = gdr.cache_resize(slot, lens, i32([1, 0, 1, 1]), 1, 5)
    assert slot[:, 0].tolist() == [0, -1, 1, 2] and free.item() == 2
    lens, free = gdr.cache_resize(slot, lens, i32([0, 1, 1, 1]), 1, 5)
    assert slot[:, 0].tolist() == [-1, 0, 1, 2] and free.item() == 2
    pool = torch.zeros(5, H, D, D, device=DEV)
    x = torch.randn(B, 1, H, D, device=DEV) * 0.1
    g, beta = -torch.rand(B, 1, H, device=DEV), torch.rand(B, 1, H, device=DEV)
    gdr.decode_tokens(x, x, x, g, beta, pool, slot=slot.view(B))
    sync()
    busy = [bool(pool[i].abs().max() > 0) for i in range(5)]
    assert busy == [True, True, True, False, False]


def test_graph_and_streams():
    """A round of drafts captured once and replayed on new contents, and two at
    once on two streams."""
    B, Hkv, G, D, page, n, dt = 3, 2, 2, 128, 16, 7, torch.bfloat16
    lens = [40, 9, 100]
    total = [l + n for l in lens]
    sets = []
    for seed in range(3):
        kc, vc, sc, table = make_cache(total, Hkv, D, page, dt, seed=seed)
        sets.append(dict(kc=kc, vc=vc, sc=sc, table=torch.from_numpy(table), par=torch.from_numpy(
            trees(B, n, seed + 5)), leaf=torch.tensor([seed, 6, 4 - seed], dtype=torch.int32),
            q=queries(B, n, Hkv * G, D, dt, seed), lens=torch.tensor(total, dtype=torch.int32)))
    P = sets[0]["kc"].shape[0]

    def step(x, **kw):
        o = gdr.attention_tree(x["q"], x["kc"], x["vc"], x["table"], x["lens"], x["par"], scale=0.1,
                               o=kw.get("o"), workspace=kw.get("ws"))
        new, path = gdr.cache_accept(x["kc"], x["vc"], x["table"], x["lens"], x["par"], x["leaf"],
                                     scores=x["sc"], new_lens=kw.get("new"), path=kw.get("path"))
        end, free = gdr.cache_resize(x["table"], x["lens"], new, page, P, new_lens=x["lens"],
                                     free=kw.get("free"), cu_seqlens=kw.get("cu"))
        return [o, new, path, end, free, x["kc"], x["vc"], x["sc"], x["table"]]

    up = lambda x: {k: v.to(DEV) for k, v in x.items()}  # noqa: E731
    eager = []
    for x in sets:
        eager.append([y.clone() for y in step(up(x))])
        sync()
    streams, outs = [torch.cuda.Stream(DEV) for _ in range(2)], []
    gpu = [up(x) for x in sets]
    sync()
    for x, s in zip(gpu, streams):
        with torch.cuda.stream(s):
            outs.append(step(x))
    sync()
    for got, want in zip(outs, eager):
        assert all(same(a, b) for a, b in zip(got, want))
    x = up(sets[0])
    z = lambda *s: torch.zeros(s, device=DEV, dtype=torch.int32)  # noqa: E731
    bufs = dict(o=torch.empty_like(x["q"]), new=z(B), path=z(B, n), free=z(1), cu=z(B + 1),
                ws=torch.empty(gdr.attention_workspace_bytes(B, n, Hkv * G, Hkv, D,
                                                             x["table"].shape[1], page),
                               device=DEV, dtype=torch.uint8))
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, **bufs)
    for i in (1, 2, 0, 1):
        for k, v in sets[i].items():
            x[k].copy_(v.to(DEV))
        sync()
        graph.replay()
        sync()
        assert all(same(a, b) for a, b in zip(got, eager[i])), i
