"""GPU tests of the paged key-value cache against its 64-bit reference
(tests/cache_ref.py): token writes, attention of new tokens, eviction, and a
run of the three as a serving loop uses them.  Everything the calls must not
touch is poisoned with NaN or kept and compared bit for bit."""
import numpy as np
import pytest
import torch

import gated_delta_rule_44_amd as gdr
from tests import cache_ref as ref
from tests.conftest import gpu_available
from tests.gpu_util import announce

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
DEV = torch.device("cuda:0")
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
NAN = float("nan")


def sync():
    torch.cuda.synchronize(DEV)


def gpu(x, dtype=None):
    t = x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))
    return t.to(DEV) if dtype is None else t.to(dtype).to(DEV)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def same(a, b):
    """Equal bit for bit (NaN included)."""
    a, b = a.detach().cpu().contiguous(), b.detach().cpu().contiguous()
    kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.shape == b.shape and torch.equal(a.view(kind), b.view(kind))


def make_cache(lens, Hkv, D, page, dt, seed, spare=2, extra=1):
    """Caches (CPU) holding lens[b] tokens of each sequence on shuffled pages,
    NaN everywhere else; table has `extra` unused (-1) columns."""
    rng = np.random.default_rng(seed)
    need = [-(-l // page) for l in lens]
    P, M = sum(need) + spare, max(need + [0]) + extra
    pages = rng.permutation(P)
    table = np.full((len(lens), M), -1, np.int32)
    at = 0
    kc = torch.full((P, Hkv, page, D), NAN, dtype=dt)
    vc, sc = kc.clone(), torch.full((P, Hkv, page), NAN)
    for b, (l, c) in enumerate(zip(lens, need)):
        table[b, :c] = pages[at:at + c]
        at += c
        for i in range(c):
            m = min(page, l - i * page)
            p = table[b, i]
            kc[p, :, :m] = torch.from_numpy(rng.standard_normal((Hkv, m, D))).to(dt)
            vc[p, :, :m] = torch.from_numpy(rng.standard_normal((Hkv, m, D))).to(dt)
            sc[p, :, :m] = torch.from_numpy(np.exp(2 * rng.standard_normal((Hkv, m)))).float()
    return kc, vc, sc, table


def check_attend(q, kc, vc, table, lens, scale, window=0, sc=None, what="", **kw):
    """One call against the reference; returns its outputs (on the GPU)."""
    dk, dv = gpu(kc), gpu(vc)
    ds = None if sc is None else gpu(sc)
    o = gdr.attention_decode(gpu(q), dk, dv, i32(table), i32(lens), scale=scale, window=window,
                             scores=ds, **kw)
    sync()
    want = ref.attend(q, kc, vc, table, lens, scale, window, sc)
    err = (o.double().cpu().numpy() - want[0])
    bad = ~(np.abs(err) <= want[1])
    worst = np.abs(err / np.maximum(want[1], 1e-300)).max() if err.size else 0
    announce("  %s o: worst error / bound %.3f" % (what, worst))
    assert not bad.any(), "%s: o at %s" % (what, np.argwhere(bad)[:4].tolist())
    assert same(dk, kc) and same(dv, vc), "%s: the cache changed" % what
    if sc is None:
        return o
    new, old = ds.double().cpu().numpy(), sc.double().numpy()
    touched = want[3] > 0
    # what no row reads keeps its bits
    same_bits = ds.cpu().view(torch.int32).numpy() == sc.view(torch.int32).numpy()
    read = np.zeros(sc.shape, bool)
    for b in range(table.shape[0]):
        L = max(0, min(int(lens[b]), table.shape[1] * kc.shape[2]))
        n = q.shape[1]
        lo = max(0, L - n + 1 - window) if window else 0
        for j in range(lo, L):
            x = ref.place(table, kc.shape[0], kc.shape[2], b, j)
            if x is not None:
                read[x[0], :, x[1]] = True
    assert same_bits[~read].all(), "%s: scores of unread tokens changed" % what
    err = np.abs(new - want[2])[touched & read]
    lim = want[3][touched & read]
    announce("  %s scores: worst error / bound %.3f" % (what, (err / lim).max() if err.size else 0))
    assert (err <= lim).all(), "%s: scores (old %s)" % (what, old[touched & read][:2])
    return o, ds


def queries(B, n, Hq, D, dt, seed, amp=2.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(amp * rng.standard_normal((B, n, Hq, D))).to(dt)


# ------------------------------------------------------------------ attention
LENS = [1, 0, 16, 17, 63, 65, 130, 200]
SHAPES = [
    # D, page, Hkv, G, n, window
    (128, 16, 2, 4, 1, 0),
    (64, 16, 3, 1, 1, 0),
    (128, 64, 1, 8, 1, 0),
    (64, 32, 2, 7, 1, 0),
    (128, 256, 1, 16, 1, 0),
    (128, 32, 2, 4, 4, 0),
    (64, 128, 1, 3, 5, 0),
    (128, 16, 1, 5, 16, 0),
    (64, 16, 2, 40, 2, 0),
    (128, 16, 2, 4, 1, 1),
    (64, 32, 1, 2, 1, 50),
    (128, 64, 2, 4, 4, 33),
    (64, 16, 1, 1, 9, 7),
    (128, 16, 1, 1, 70, 20),
]


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D,page,Hkv,G,n,window", SHAPES)
def test_attend(dt, D, page, Hkv, G, n, window):
    announce("attend %s D=%d page=%d Hkv=%d G=%d n=%d window=%d" % (dt, D, page, Hkv, G, n, window))
    kc, vc, sc, table = make_cache(LENS, Hkv, D, page, DTYPES[dt], seed=D + page + n)
    q = queries(len(LENS), n, Hkv * G, D, DTYPES[dt], seed=n)
    o = check_attend(q, kc, vc, table, LENS, D ** -0.5, window, what="plain")
    o2, s2 = check_attend(q, kc, vc, table, LENS, D ** -0.5, window, sc, what="scores")
    assert torch.equal(o, o2), "o depends on whether scores are taken"
    # the same bits on a second run
    o3, s3 = check_attend(q, kc, vc, table, LENS, D ** -0.5, window, sc, what="again")
    assert torch.equal(o2, o3) and same(s2, s3)


@pytest.mark.parametrize("D,page,n,G,window", [
    (128, 16, 16, 4, 0), (128, 64, 9, 4, 0), (64, 32, 33, 2, 0), (128, 32, 70, 1, 0),
    (64, 16, 20, 5, 0), (128, 16, 40, 2, 75), (64, 256, 13, 3, 20), (128, 64, 300, 4, 0)])
def test_attend_many_rows_long_table(D, page, n, G, window):
    """Over 32 rows a head and a table for many tokens: two tiles of rows that
    share the tokens."""
    announce("attend rows D=%d page=%d n=%d G=%d window=%d" % (D, page, n, G, window))
    lens = [1, 0, 33, 700, 65, 1500]
    kc, vc, sc, table = make_cache(lens, 2, D, page, torch.bfloat16, seed=D + n,
                                   extra=(48 << 20) // (len(lens) * 2 * D * page))
    q = queries(len(lens), n, 2 * G, D, torch.bfloat16, seed=n)
    o = check_attend(q, kc, vc, table, lens, D ** -0.5, window, what="plain")
    table[3, 2] = -1
    check_attend(q, kc, vc, table, lens, D ** -0.5, window, sc, what="absent, scores")
    # infinities and NaN where a row does not attend
    clean = vc.clone()
    for b, j, x in ((5, 1499, NAN), (5, 1490, float("inf")), (4, 64, -float("inf")), (2, 20, NAN)):
        p, s = ref.place(table, kc.shape[0], page, b, j)
        vc[p, :, s, 3] = x
        clean[p, :, s, 3] = 0
    got = gdr.attention_decode(gpu(q), gpu(kc), gpu(vc), i32(table), i32(lens), window=window)
    want = gdr.attention_decode(gpu(q), gpu(kc), gpu(clean), i32(table), i32(lens), window=window)
    got, want = got.float().cpu().numpy(), want.float().cpu().numpy()
    for b, L in enumerate(lens):
        for t in range(n):
            p = L - n + t
            seen = [x for bb, j, x in ((5, 1499, NAN), (5, 1490, np.inf), (4, 64, -np.inf), (2, 20, NAN))
                    if bb == b and j <= p and (not window or j > p - window)]
            total = sum(seen) if seen else 0.0
            here, there = got[b, t, :, 3], want[b, t, :, 3]
            if not seen:
                assert np.array_equal(here, there), (b, t)
            else:
                assert (np.isnan(here).all() if np.isnan(total) else (here == total).all()), (b, t)
    o2 = np.delete(got, 3, axis=-1)
    assert np.array_equal(o2, np.delete(want, 3, axis=-1)) and o is not None


@pytest.mark.parametrize("D,page,n,window", [(128, 64, 10, 900), (64, 16, 17, 1800)])
def test_attend_many_rows_wide_window(D, page, n, window):
    """The same with a window that cuts into the longer sequences and is wide
    enough for rows to share tokens."""
    announce("attend rows D=%d page=%d n=%d window=%d" % (D, page, n, window))
    lens = [window + 500, 30, 0, window + 5, window - 3, window + n] + [33] * 18
    kc, vc, sc, table = make_cache(lens, 4, D, page, torch.bfloat16, seed=D, extra=2)
    q = queries(len(lens), n, 16, D, torch.bfloat16, seed=n)
    check_attend(q, kc, vc, table, lens, D ** -0.5, window, what="plain")
    check_attend(q, kc, vc, table, lens, D ** -0.5, window, sc, what="scores")
    # an infinity that the first rows alone attend to
    b, j = 0, lens[0] - n - window + 1
    p, s = ref.place(table, kc.shape[0], page, b, j)
    vc[p, :, s, 5] = float("inf")
    got = gdr.attention_decode(gpu(q), gpu(kc), gpu(vc), i32(table), i32(lens), window=window).cpu()
    assert (got[b, 0, :, 5] == float("inf")).all()
    assert torch.isfinite(got[b, 1:]).all() and torch.isfinite(got[1:]).all()


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,n,G,window", [
    ([4097], 1, 4, 0), ([9000, 40], 1, 8, 0), ([2500, 1, 777], 3, 2, 0), ([6000], 2, 4, 2100),
    ([1024] * 9, 1, 1, 0)])
def test_attend_long(dt, lens, n, G, window):
    """Lengths that are split over several workgroups and joined."""
    announce("attend long %s %s n=%d G=%d window=%d" % (dt, lens, n, G, window))
    kc, vc, sc, table = make_cache(lens, 2, 128, 32, DTYPES[dt], seed=len(lens))
    q = queries(len(lens), n, 2 * G, 128, DTYPES[dt], seed=n + 50)
    check_attend(q, kc, vc, table, lens, 128 ** -0.5, window, what="plain")
    check_attend(q, kc, vc, table, lens, 128 ** -0.5, window, sc, what="scores")


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_attend_many_sequences(dt):
    """More sequences than lanes of a wave, most of them short or empty."""
    announce("attend many %s" % dt)
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 40, 300)]
    lens[7], lens[250] = 1500, 900
    kc, vc, sc, table = make_cache(lens, 1, 64, 16, DTYPES[dt], seed=6)
    q = queries(len(lens), 1, 2, 64, DTYPES[dt], seed=7)
    check_attend(q, kc, vc, table, lens, 0.2, what="plain")
    check_attend(q, kc, vc, table, lens, 0.2, 0, sc, what="scores")


@pytest.mark.parametrize("B", [1025, 4096, 4500])
def test_attend_thousands_of_sequences(B):
    """Several sequences per thread of the search, and more than it takes; one
    of them long."""
    announce("attend %d sequences" % B)
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 20, B)]
    lens[B // 2] = 1400
    kc, vc, sc, table = make_cache(lens, 1, 64, 32, torch.bfloat16, seed=6)
    q = queries(B, 1, 1, 64, torch.bfloat16, seed=7)
    check_attend(q, kc, vc, table, lens, 0.2, 0, sc, what="scores")


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_attend_absent_pages_and_odd_lengths(dt):
    """Pages that are absent (below, above and far outside the range), a
    sequence with none present, lengths below zero and past the table."""
    announce("attend absent %s" % dt)
    lens = [100, 90, 48, 64, 64]
    kc, vc, sc, table = make_cache(lens, 2, 64, 16, DTYPES[dt], seed=8)
    P = kc.shape[0]
    table[0, 2], table[0, 6], table[1, 0], table[1, 5] = -1, P, 2 ** 31 - 1, -2 ** 31
    table[2, :] = -1
    said = [100, 90, 48, -7, 64 + 16 * 5]
    table[4, 4:] = [-1] * (table.shape[1] - 4)
    q = queries(5, 2, 4, 64, DTYPES[dt], seed=9)
    o, _ = check_attend(q, kc, vc, table, said, 0.125, 0, sc, what="absent")
    assert bool((o[2] == 0).all()) and bool((o[3] == 0).all())
    check_attend(q, kc, vc, table, said, 0.125, 30, what="window")


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
def test_attend_masked_tokens_have_no_part(dt, bad):
    """Drafted tokens and tokens that left the window hold NaN or infinities:
    the rows that do not attend to them are as if they held zeros."""
    announce("attend masked %s %s" % (dt, bad))
    lens, n, window = [70, 33, 3], 4, 20
    kc, vc, _, table = make_cache(lens, 1, 128, 16, DTYPES[dt], seed=10)
    q = queries(3, n, 2, 128, DTYPES[dt], seed=11)
    k2, v2 = kc.clone(), vc.clone()
    clean_k, clean_v = kc.clone(), vc.clone()
    spots = [(b, j) for b, l in enumerate(lens) for j in (l - 1, l - n - window, l - n - window + 2)
             if j >= 0]
    for b, j in spots:
        p, s = ref.place(table, kc.shape[0], 16, b, j)
        k2[p, :, s, 5], v2[p, :, s, 7] = bad, bad
        clean_k[p, :, s], clean_v[p, :, s] = 0, 0
    run = lambda k, v: gdr.attention_decode(gpu(q), gpu(k), gpu(v), i32(table), i32(lens),  # noqa: E731
                                            window=window).float().cpu().numpy()
    got, want = run(k2, v2), run(clean_k, clean_v)
    o_ref, bound = ref.attend(q, clean_k, clean_v, table, lens, 128 ** -0.5, window)
    assert (np.abs(want - o_ref) <= bound).all()
    checked = 0
    for b, l in enumerate(lens):
        for t in range(n):
            p = l - n + t
            seen = [j for bb, j in spots if bb == b and p - window < j <= p]
            if not seen:
                assert np.array_equal(got[b, t], want[b, t]), (b, t)
                checked += 1
            else:
                assert not np.isfinite(got[b, t, :, 7]).all(), (b, t)
    assert checked >= 5


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_attend_extreme_logits(dt):
    """One key far above the others, all keys equal, a scale of zero and a
    negative one, and logits near the end of fp32's range."""
    announce("attend extreme %s" % dt)
    lens = [150, 40]
    kc, vc, sc, table = make_cache(lens, 1, 64, 16, DTYPES[dt], seed=12)
    q = queries(2, 1, 3, 64, DTYPES[dt], seed=13)
    for scale in (0.0, -0.3, 8.0):
        check_attend(q, kc, vc, table, lens, scale, 0, sc, what="scale %g" % scale)
    p, s = ref.place(table, kc.shape[0], 16, 0, 77)
    kc[p, 0, s] = (1e4 * q[0, 0, 0].float()).to(kc.dtype)
    check_attend(q, kc, vc, table, lens, 0.125, what="one key")
    big = kc.clone()
    for b, l in enumerate(lens):
        for j in range(l):
            pp, ss = ref.place(table, kc.shape[0], 16, b, j)
            big[pp, 0, ss] = 0
            big[pp, 0, ss, 0] = 1e30
    q2 = torch.zeros_like(q)
    q2[..., 0] = -1e8            # every logit -1e38: far below, all equal
    check_attend(q2, big, vc, table, lens, 1.0, what="equal and far below zero")


def test_attend_all_logits_minus_infinity_gives_zero():
    kc, vc, _, table = make_cache([30], 1, 64, 16, torch.float32, seed=14)
    q = torch.zeros(1, 1, 1, 64)
    q[..., 0] = 1.0
    p = table[0, :2]
    kc[p, :, :, 0] = -float("inf")
    o = gdr.attention_decode(gpu(q), gpu(kc), gpu(vc), i32(table), i32([30]))
    sync()
    assert bool((o == 0).all())


def test_attend_shared_pages():
    """A prefix shared by two sequences (without scores)."""
    kc, vc, _, table = make_cache([64, 50], 2, 128, 16, torch.bfloat16, seed=15)
    table[1, :2] = table[0, :2]
    q = queries(2, 1, 4, 128, torch.bfloat16, seed=16)
    check_attend(q, kc, vc, table, [64, 50], 0.1, what="shared")


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_offsets_past_32_bits(dt):
    """Caches of more than 2^32 bytes (and 2^31 elements): write, attend and
    evict on their last pages, against the same call on a small cache."""
    announce("far pages %s" % dt)
    Hkv, page, D = 8, 256, 128
    P = (5 << 30) // (Hkv * page * D * 2)
    far = [P - 1, P - 2, P // 2 + 1, 0]
    lens, dtype = [700, 200], DTYPES[dt]
    kc, vc, sc, table = make_cache(lens, Hkv, D, page, dtype, seed=17, spare=0, extra=0)
    big_k = torch.empty((P, Hkv, page, D), device=DEV, dtype=dtype)
    big_v, big_s = torch.empty_like(big_k), torch.empty((P, Hkv, page), device=DEV)
    for i in range(4):
        big_k[far[i]], big_v[far[i]], big_s[far[i]] = gpu(kc[i]), gpu(vc[i]), gpu(sc[i])
    big_table = np.array(far, np.int32)[table] * (table >= 0) - (table < 0)
    q = queries(2, 2, 16, D, dtype, seed=18)
    outs = []
    for k, v, s, t in ((gpu(kc), gpu(vc), gpu(sc), table), (big_k, big_v, big_s, big_table)):
        new = gpu(queries(2, 2, Hkv, D, dtype, seed=19))
        gdr.cache_append(new, new * 2, i32([690, 198]), i32(t), k, v, scores=s)
        o = gdr.attention_decode(gpu(q), k, v, i32(t), i32(lens), scores=s)
        nl, kept = gdr.cache_evict(k, v, s, i32(t), i32(lens), 150, 20, 3)
        o2 = gdr.attention_decode(gpu(q), k, v, i32(t), nl)
        sync()
        outs.append((o, kept, o2))
    for a, b in zip(*outs):
        assert same(a, b)
    del big_k, big_v, big_s
    torch.cuda.empty_cache()


def test_attend_other_stream_and_graph():
    """On a stream of its own, and captured with append and evict: replays on
    new inputs equal the eager calls."""
    B, n, Hkv, G, D, page = 3, 2, 2, 4, 128, 16
    lens0 = [40, 90, 300]
    kc, vc, sc, table = make_cache([l + 20 for l in lens0], Hkv, D, page, torch.bfloat16, seed=20)
    sc = torch.nan_to_num(sc)
    t, start = i32(table), i32(lens0)
    k, v = (gpu(queries(B, n, Hkv, D, torch.bfloat16, seed=s)) for s in (21, 22))
    q = gpu(queries(B, n, Hkv * G, D, torch.bfloat16, seed=23))
    state = [gpu(kc), gpu(vc), gpu(sc)]
    lens = start + n
    ws = torch.empty(gdr.attention_workspace_bytes(B, n, Hkv * G, Hkv, D, t.shape[1], page, True),
                     device=DEV, dtype=torch.uint8)

    def step(k, v, q, state, start, lens, ws=None):
        gdr.cache_append(k, v, start, t, state[0], state[1], scores=state[2])
        o = gdr.attention_decode(q, state[0], state[1], t, lens, scores=state[2], workspace=ws)
        nl, kept = gdr.cache_evict(*state, t, lens, 64, 16, 2)
        return o, nl, kept

    side = torch.cuda.Stream(DEV)
    fresh = lambda: [gpu(kc), gpu(vc), gpu(sc)]  # noqa: E731
    eager_state = fresh()
    eager = step(k, v, q, eager_state, start, lens)
    sync()
    other = fresh()
    with torch.cuda.stream(side):
        out = step(k, v, q, other, start, lens, ws)
    side.synchronize()
    for a, b in zip(list(eager) + eager_state, list(out) + other):
        assert same(a, b), "another stream"
    graph = torch.cuda.CUDAGraph()
    sync()
    with torch.cuda.graph(graph):
        out = step(k, v, q, state, start, lens, ws)
    for rep in range(3):
        announce("graph replay %d" % rep)
        for x, y in zip(state, fresh()):
            x.copy_(y)
        new = np.array(lens0) - 5 * rep
        start.copy_(i32(new))
        lens.copy_(i32(new + n))
        for x, s in ((k, 30), (v, 40)):
            x.copy_(gpu(queries(B, n, Hkv, D, torch.bfloat16, seed=s + rep)))
        q.copy_(gpu(queries(B, n, Hkv * G, D, torch.bfloat16, seed=50 + rep)))
        sync()
        graph.replay()
        sync()
        got = [x.clone() for x in list(out) + state]
        eager_state = fresh()
        want = list(step(k, v, q, eager_state, start, lens)) + eager_state
        sync()
        for a, b in zip(got, want):
            assert same(a, b), "replay %d" % rep


def test_two_calls_at_once_on_two_streams():
    """Different batches on two streams, each with a workspace of its own."""
    runs, want = [], []
    for i, lens in enumerate(([3000, 10, 700], [900, 1200, 2])):
        kc, vc, sc, table = make_cache(lens, 2, 128, 32, torch.bfloat16, seed=95 + i)
        q = queries(3, 2, 8, 128, torch.bfloat16, seed=97 + i)
        args = [gpu(q), gpu(kc), gpu(vc), i32(table), i32(lens)]
        runs.append((args, torch.nan_to_num(gpu(sc))))
    sync()
    for args, sc in runs:
        s = sc.clone()
        want.append((gdr.attention_decode(*args, scores=s), s))
    sync()
    streams = [torch.cuda.Stream(DEV) for _ in runs]
    for rep in range(5):
        got = []
        for st, (args, sc) in zip(streams, runs):
            with torch.cuda.stream(st):
                s = sc.clone()
                got.append((gdr.attention_decode(*args, scores=s), s))
        sync()
        for a, b in zip(got, want):
            assert same(a[0], b[0]) and same(a[1], b[1]), rep


def test_refusals_of_the_binding():
    """Wrong dtypes, shapes, places and strides raise and write nothing."""
    kc, vc, sc, table = make_cache([40, 20], 2, 64, 16, torch.bfloat16, seed=99)
    k, v, s, t, lens = gpu(kc), gpu(vc), gpu(sc), i32(table), i32([40, 20])
    q = gpu(queries(2, 1, 4, 64, torch.bfloat16, seed=100))
    new = gpu(queries(2, 1, 2, 64, torch.bfloat16, seed=101))
    good = dict(q=q, k_cache=k, v_cache=v, page_table=t, seq_lens=lens)
    for name, bad in [("q", q.float()), ("q", q[:, :, :3].contiguous()), ("q", q.cpu()), ("q", None),
                      ("q", q[:, 0]), ("q", q.expand(2, 1, 4, 64).transpose(1, 2)),
                      ("k_cache", k.half()), ("k_cache", k[:, :, :8]), ("k_cache", kc),
                      ("v_cache", v[:-1]), ("v_cache", v.float()), ("page_table", t.long()),
                      ("page_table", t[:1].contiguous()), ("page_table", t.t()),
                      ("seq_lens", lens.float()), ("seq_lens", lens[:1]), ("seq_lens", [40, 20]),
                      ("window", -1), ("window", 2 ** 32), ("scores", s[:, :1].contiguous()),
                      ("scores", s.double()), ("o", q.float()), ("o", q[:1]),
                      ("scale", float("nan")), ("page_table_host", table[:, :1]),
                      ("page_table_host", table + 1000),
                      ("workspace", torch.empty(8, dtype=torch.uint8, device=DEV)),
                      ("workspace", torch.empty(1 << 20, dtype=torch.uint8))]:
        with pytest.raises(gdr.GdrError):
            gdr.attention_decode(**{**good, name: bad})
    good = dict(k=new, v=new, start=lens, page_table=t, k_cache=k, v_cache=v)
    for name, bad in [("k", new.float()), ("k", new[:, :, :1].contiguous()), ("v", new[:1]),
                      ("start", lens.long()), ("start", lens[:1]), ("cu_seqlens", lens),
                      ("cu_seqlens_host", [0, 1, 2]), ("scores", s[:-1])]:
        with pytest.raises(gdr.GdrError):
            gdr.cache_append(**{**good, name: bad})
    good = dict(k_cache=k, v_cache=v, scores=s, page_table=t, seq_lens=lens, budget=16)
    twice = table.copy()
    twice[1, 0] = twice[0, 0]
    for name, bad in [("scores", None), ("budget", 0), ("budget", 2 ** 31), ("recent", -1),
                      ("recent", 17), ("sink", 17), ("new_lens", lens.long()),
                      ("new_lens", lens[:1]), ("page_table_host", twice),
                      ("kept", torch.empty(2, 2, 15, dtype=torch.int32, device=DEV)),
                      ("new_page_table", t[:, :0].contiguous()), ("new_page_table_host", table)]:
        with pytest.raises(gdr.GdrError):
            gdr.cache_evict(**{**good, name: bad})
    sync()
    assert same(k, kc) and same(v, vc) and same(s, sc)


# --------------------------------------------------------------------- append
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D,page,Hkv,n", [(128, 16, 2, 1), (64, 64, 3, 5), (128, 256, 1, 40),
                                          (64, 16, 8, 33)])
def test_append(dt, D, page, Hkv, n):
    announce("append %s D=%d page=%d Hkv=%d n=%d" % (dt, D, page, Hkv, n))
    lens = [3 * page + 7, 50, 0, page]
    kc, vc, sc, table = make_cache([l + n for l in lens], Hkv, D, page, DTYPES[dt], seed=n)
    start = np.array(lens)
    start[2] = -3                                   # its first three rows have no place
    start[3] = table.shape[1] * page - 1            # one place, and that page is absent
    table[1, 50 // page] = -1
    k, v = (queries(4, n, Hkv, D, DTYPES[dt], seed=s) for s in (n + 1, n + 2))
    for scores in (None, sc):
        dk, dv = gpu(kc), gpu(vc)
        ds = None if scores is None else gpu(scores)
        gdr.cache_append(gpu(k), gpu(v), i32(start), i32(table), dk, dv, scores=ds)
        sync()
        want = ref.append(k, v, start, table, kc, vc, scores)
        for a, b in zip((dk, dv, ds), want):
            assert same(a, b)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_append_packed(dt):
    announce("append packed %s" % dt)
    n = [37, 0, 1, 100, 16]
    start = [0, 5, 31, 12, 0]
    kc, vc, sc, table = make_cache([a + b for a, b in zip(n, start)], 2, 64, 16, DTYPES[dt], seed=60)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = int(cu[-1]) + 9                              # nine padding rows behind the last sequence
    k, v = (queries(T, 1, 2, 64, DTYPES[dt], seed=s)[:, 0].contiguous() for s in (61, 62))
    for host in (None, cu):
        dk, dv, ds = gpu(kc), gpu(vc), gpu(sc)
        gdr.cache_append(gpu(k), gpu(v), i32(start), i32(table), dk, dv, scores=ds,
                         cu_seqlens=i32(cu), cu_seqlens_host=host)
        sync()
        for a, b in zip((dk, dv, ds), ref.append(k, v, start, table, kc, vc, sc, cu=cu)):
            assert same(a, b)


def test_append_many_sequences_packed():
    """More sequences than a wave's lanes, many of them empty."""
    rng = np.random.default_rng(63)
    n = rng.integers(0, 4, 500)
    n[100:180] = 0
    kc, vc, sc, table = make_cache([int(x) + 2 for x in n], 1, 64, 16, torch.bfloat16, seed=64)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    k = queries(int(cu[-1]), 1, 1, 64, torch.bfloat16, seed=65)[:, 0].contiguous()
    dk, dv = gpu(kc), gpu(vc)
    gdr.cache_append(gpu(k), gpu(k), i32([2] * 500), i32(table), dk, dv, cu_seqlens=i32(cu))
    sync()
    for a, b in zip((dk, dv), ref.append(k, k, [2] * 500, table, kc, vc, cu=cu)):
        assert same(a, b)


# ---------------------------------------------------------------------- evict
def run_evict(kc, vc, sc, table, lens, budget, recent, sink, new_table=None, what=""):
    announce("  evict %s budget=%d recent=%d sink=%d" % (what, budget, recent, sink))
    dk, dv, ds = gpu(kc), gpu(vc), gpu(sc)
    nl, kept = gdr.cache_evict(dk, dv, ds, i32(table), i32(lens), budget, recent, sink,
                               new_page_table=None if new_table is None else i32(new_table))
    sync()
    want = ref.evict(kc, vc, sc, table, lens, budget, recent, sink, new_table)
    assert np.array_equal(kept.cpu().numpy(), want[4]), what
    assert np.array_equal(nl.cpu().numpy(), want[3]), what
    for a, b, name in zip((dk, dv, ds), want, ("k_cache", "v_cache", "scores")):
        assert same(a, b), "%s: %s" % (what, name)


def odd_scores(sc, kind, seed):
    rng = np.random.default_rng(seed)
    x = sc.clone()
    if kind == "ties":
        x = torch.from_numpy(rng.integers(0, 3, x.shape)).float()
    elif kind == "special":
        pool = torch.tensor([NAN, float("inf"), -float("inf"), 0.0, -0.0, 1e-42, -1e-42, 1.0, -1.0])
        x = pool[torch.from_numpy(rng.integers(0, len(pool), x.shape))]
    elif kind == "close":
        x = (1.0 + torch.from_numpy(rng.integers(0, 600, x.shape)) * 2.0 ** -23).float()
    return x.contiguous()


@pytest.mark.parametrize("dt,D,page", [("bf16", 128, 16), ("fp32", 64, 32), ("bf16", 64, 256),
                                       ("fp32", 128, 64)])
@pytest.mark.parametrize("kind", ["weights", "ties", "special", "close"])
@pytest.mark.parametrize("pages", ["in place", "new pages"])
def test_evict(dt, D, page, kind, pages):
    announce("evict %s D=%d page=%d %s %s" % (dt, D, page, kind, pages))
    lens = [300, 64, 65, 0, 1, 777]
    Hkv = 2
    new_need = len(lens) * (-(-200 // page) + 1)
    kc, vc, sc, table = make_cache(lens, Hkv, D, page, DTYPES[dt], seed=70, spare=new_need)
    sc = odd_scores(sc, kind, 71)
    new_table = None
    if pages == "new pages":
        free = np.setdiff1d(np.arange(kc.shape[0]), table[table >= 0])
        new_table = free[:new_need].reshape(len(lens), -1).astype(np.int32)
    for budget, recent, sink in ((64, 16, 4), (200, 0, 0), (1, 0, 0), (5, 5, 0), (7, 3, 4),
                                 (128, 1, 127)):
        run_evict(kc, vc, sc, table, lens, budget, recent, sink, new_table, kind)


@pytest.mark.parametrize("pages", ["in place", "new pages"])
def test_evict_long_and_large_budget(pages):
    lens = [9001, 5000]
    kc, vc, sc, table = make_cache(lens, 1, 64, 128, torch.bfloat16, seed=72, spare=150)
    for kind in ("weights", "ties"):
        s = odd_scores(sc, kind, 73)
        for budget in (5000, 6789, 20000):
            new_table = None
            if pages == "new pages":
                free = np.setdiff1d(np.arange(kc.shape[0]), table[table >= 0])
                new_table = free[:144].reshape(2, -1).astype(np.int32)
            run_evict(kc, vc, s, table, lens, budget, 100, 10, new_table, kind)


@pytest.mark.parametrize("kind", ["weights", "ties", "special", "close"])
@pytest.mark.parametrize("others", [0, 70])
def test_evict_very_long(kind, others):
    """Past 65,536 tokens, and just at that length: with few sequences a pair's
    selection is spread over workgroups, among many it is one workgroup's."""
    announce("evict very long %s others=%d" % (kind, others))
    lens = [70001, 65536, 131] + [9] * others
    kc, vc, sc, table = make_cache(lens, 1, 64, 256, torch.bfloat16, seed=90)
    s = odd_scores(sc, kind, 91)
    for budget, recent, sink in ((30000, 1000, 10), (100, 0, 0), (5000, 4000, 1000), (66000, 1, 1)):
        run_evict(kc, vc, s, table, lens, budget, recent, sink, None, kind)


@pytest.mark.parametrize("others", [0, 70])
def test_evict_long_with_absent_pages(others):
    """More tokens wanted than are present: of those on absent pages the lowest
    are kept, across the borders of the workgroups' shares too."""
    announce("evict long absent others=%d" % others)
    lens = [13000, 9000, 8500] + [5] * others
    kc, vc, sc, table = make_cache(lens, 1, 64, 16, torch.float32, seed=92)
    rng = np.random.default_rng(93)
    table[0, rng.random(table.shape[1]) < 0.7] = -1
    table[1, :] = -1
    for budget, recent, sink in ((6000, 0, 0), (8000, 500, 70), (8990, 3, 4200)):
        run_evict(kc, vc, sc, table, lens, budget, recent, sink, None, "absent")


def test_evict_absent_pages():
    """Tokens on absent pages go first and are not moved; absent new pages
    take nothing."""
    lens = [160, 160, 30]
    kc, vc, sc, table = make_cache(lens, 2, 64, 16, torch.float32, seed=74, spare=20)
    sc = odd_scores(sc, "special", 75)
    table[0, 1], table[0, 9], table[1, 4] = -1, 10 ** 9, -5
    table[2, :] = -1
    free = np.setdiff1d(np.arange(kc.shape[0]), table[table >= 0])
    for budget in (50, 140, 155):
        run_evict(kc, vc, sc, table, lens, budget, 20, 3, None, "absent")
    new_table = np.full((3, 5), -1, np.int32)
    new_table[:, :4] = free[:12].reshape(3, 4)
    new_table[1, 2] = 2 ** 31 - 1
    run_evict(kc, vc, sc, table, lens, 70, 20, 3, new_table, "absent new")


def test_evict_shared_pages_into_new_ones():
    """Two sequences with a common prefix, trimmed into pages of their own."""
    lens = [100, 90]
    kc, vc, sc, table = make_cache(lens, 2, 128, 16, torch.bfloat16, seed=76, spare=10)
    table[1, :3] = table[0, :3]
    free = np.setdiff1d(np.arange(kc.shape[0]), table[table >= 0])
    run_evict(kc, vc, sc, table, lens, 48, 8, 2, free[:6].reshape(2, 3).astype(np.int32), "shared")


def test_evict_lens_in_place():
    """new_lens may be seq_lens; a second call finds nothing to do."""
    lens = [100, 20, 64]
    kc, vc, sc, table = make_cache(lens, 4, 128, 16, torch.bfloat16, seed=77)
    dk, dv, ds, dl = gpu(kc), gpu(vc), gpu(sc), i32(lens)
    nl, kept = gdr.cache_evict(dk, dv, ds, i32(table), dl, 40, 8, 2, new_lens=dl,
                               page_table_host=table)
    sync()
    want = ref.evict(kc, vc, sc, table, lens, 40, 8, 2)
    assert nl is dl and dl.cpu().tolist() == [40, 20, 40]
    assert np.array_equal(kept.cpu().numpy(), want[4])
    for a, b in zip((dk, dv, ds), want):
        assert same(a, b)
    gdr.cache_evict(dk, dv, ds, i32(table), dl, 40, 8, 2, new_lens=dl)
    sync()
    for a, b in zip((dk, dv, ds), want):
        assert same(a, b)


@pytest.mark.parametrize("budget", [100, 255, 256, 257, 700])
@pytest.mark.parametrize("alias", [False, True])
def test_evict_into_new_pages(budget, alias):
    """Rows moved by the selection's own workgroups or by a launch of their
    own; the new lengths may be written over the old ones either way."""
    announce("evict new pages budget=%d alias=%s" % (budget, alias))
    lens = [900, 40, 0, 701, 256] + [300] * 40
    need = -(-budget // 32)
    kc, vc, sc, table = make_cache(lens, 8, 128, 32, torch.bfloat16, seed=budget,
                                   spare=len(lens) * need)
    free = np.setdiff1d(np.arange(kc.shape[0]), table[table >= 0])
    new_table = free[:len(lens) * need].reshape(len(lens), need).astype(np.int32)
    new_table[3, 1] = -1
    dk, dv, ds, dl = gpu(kc), gpu(vc), gpu(sc), i32(lens)
    nl, kept = gdr.cache_evict(dk, dv, ds, i32(table), dl, budget, 20, 3,
                               new_page_table=i32(new_table), new_lens=dl if alias else None)
    sync()
    want = ref.evict(kc, vc, sc, table, lens, budget, 20, 3, new_table)
    assert np.array_equal(nl.cpu().numpy(), want[3])
    assert np.array_equal(kept.cpu().numpy(), want[4])
    for a, b in zip((dk, dv, ds), want):
        assert same(a, b)


# -------------------------------------------------------- as a serving loop runs
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_serving_run(dt):
    """Prompts written packed, then steps of drafted tokens (written, attended
    to with their weights accumulated, some rejected and written over), a trim
    to a budget in place, and more steps on the trimmed cache."""
    announce("serving run %s" % dt)
    dtype, B, Hkv, G, D, page, M = DTYPES[dt], 3, 2, 4, 128, 16, 12
    rng = np.random.default_rng(80)
    table = rng.permutation(B * M + 3)[:B * M].reshape(B, M).astype(np.int32)
    P = B * M + 3
    kc, vc = (torch.full((P, Hkv, page, D), NAN, dtype=dtype) for _ in range(2))
    sc = torch.full((P, Hkv, page), NAN)
    dk, dv, ds, t = gpu(kc), gpu(vc), gpu(sc), i32(table)
    scale = D ** -0.5
    prompt = [70, 1, 25]
    cu = np.concatenate([[0], np.cumsum(prompt)]).astype(np.int32)
    k, v = (queries(int(cu[-1]), 1, Hkv, D, dtype, seed=s, amp=1.0)[:, 0].contiguous() for s in (81, 82))
    gdr.cache_append(gpu(k), gpu(v), i32([0] * B), t, dk, dv, scores=ds, cu_seqlens=i32(cu))
    sync()
    kc, vc, sc = ref.append(k, v, [0] * B, table, kc, vc, sc, cu=cu)
    lens = np.array(prompt)
    for step in range(6):
        n = [1, 4, 3, 1, 2, 4][step]
        k, v = (queries(B, n, Hkv, D, dtype, seed=100 + 3 * step + s, amp=1.0) for s in (0, 1))
        q = queries(B, n, Hkv * G, D, dtype, seed=102 + 3 * step)
        gdr.cache_append(gpu(k), gpu(v), i32(lens), t, dk, dv, scores=ds)
        kc, vc, sc = ref.append(k, v, lens, table, kc, vc, ds.cpu() if step else sc)
        sync()
        assert same(dk, kc) and same(dv, vc) and same(ds, sc)
        _, ds = check_attend(q, kc, vc, table, lens + n, scale, 0, sc, what="step %d" % step)
        # the accepted prefixes: the rest is written over by the next step
        lens = lens + rng.integers(0, n + 1, B)
        if step == 3:
            sc = ds.cpu()
            nl, _ = gdr.cache_evict(dk, dv, ds, t, i32(lens), 32, 8, 2)
            sync()
            kc, vc, sc, want_lens, _ = ref.evict(kc, vc, sc, table, lens, 32, 8, 2)
            assert np.array_equal(nl.cpu().numpy(), want_lens)
            assert same(dk, kc) and same(dv, vc) and same(ds, sc)
            lens = want_lens
