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


# ------------------------------------------------------ precision of the weights
def exact_inputs(lens, Hkv, G, n, D, page, wide, seed):
    """q and k on a grid (multiples of 1/2 up to 2, of 1/4 up to 1/2) whose dot
    products fp32 holds exactly, v random but for a constant taken off per
    sequence, head and channel, such that the last row of each head's first
    query head sums its values to nearly nothing.  Returns the call's tensors
    and, per sequence, the rows' weights [Hkv, n, G, L] and v [Hkv, L, D] in
    64 bits."""
    rng = np.random.default_rng(seed)
    B, need = len(lens), [-(-l // page) for l in lens]
    P, M = sum(need) + 1, max(need) + wide
    q = rng.integers(-4, 5, (B, n, Hkv * G, D)) / 2
    kc = np.full((P, Hkv, page, D), NAN, np.float32)
    vc, table = kc.copy(), np.full((B, M), -1, np.int32)
    pages, at, rows, scale = rng.permutation(P), 0, [], 1.0 / D ** 0.5
    for b, L in enumerate(lens):
        k = rng.integers(-2, 3, (Hkv, L, D)) / 4
        v = rng.standard_normal((Hkv, L, D))
        qb = q[b].reshape(n, Hkv, G, D).transpose(1, 0, 2, 3)
        s = scale * np.einsum("hngd,hld->hngl", qb, k)
        pos = L - n + np.arange(n)
        s = np.where(np.arange(L) <= pos[:, None, None], s, -np.inf)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        v -= np.einsum("hl,hld->hd", w[:, -1, 0], v)[:, None]
        v = torch.from_numpy(v).bfloat16().double().numpy()
        table[b, :need[b]] = pages[at:at + need[b]]
        at += need[b]
        for i, p in enumerate(table[b, :need[b]]):
            m = min(page, L - i * page)
            kc[p, :, :m] = k[:, i * page:i * page + m]
            vc[p, :, :m] = v[:, i * page:i * page + m]
        rows.append((w, v, np.abs(s[np.isfinite(s)]).max()))
    return (torch.from_numpy(q).bfloat16().to(DEV), torch.from_numpy(kc).bfloat16().to(DEV),
            torch.from_numpy(vc).bfloat16().to(DEV), i32(table), i32(lens)), rows


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("n,G,wide", [(1, 4, 0), (1, 1, 0), (5, 4, 0), (10, 4, 1)])
def test_attend_weights_of_bf16_values(D, page, n, G, wide):
    """Where the values of a row nearly cancel, o shows the weights' rounding.
    With u = 2^-24 and N tokens, logits exact but for their scaling:
      * a weight is off by e = 2 (8 u max |s| + 4 u) + (N + 16) u relative;
      * as two bf16 numbers, the first cut (a rest below 2^-7) and the rest,
        with 2^-23 added, rounded (2^-8 of it), by 2^-15 + 2^-22;
      * the 2 N products' sum by (2 N + 16) u of sum w |v|;
      * storing o adds its half step, 2^-8 |o|."""
    announce("attend weights D=%d page=%d n=%d G=%d wide=%d" % (D, page, n, G, wide))
    lens, Hkv, u = [200, 65, 16, 1500], 2, 2.0 ** -24
    table_wide = (48 << 20) // (len(lens) * Hkv * D * 4 * page) if wide else 0
    args, rows = exact_inputs(lens, Hkv, G, n, D, page, table_wide, seed=D + n + G)
    o = gdr.attention_decode(*args).double().cpu().numpy()
    worst = 0.0
    for b, (L, (w, v, s)) in enumerate(zip(lens, rows)):
        want = np.einsum("hngl,hld->hngd", w, v)
        size = np.einsum("hngl,hld->hngd", w, np.abs(v))
        rel = 2 * (8 * u * s + 4 * u) + (L + 16) * u + 2.0 ** -15 + 2.0 ** -22 + (2 * L + 16) * u
        lim = (rel * size + 2.0 ** -8 * np.abs(want)) * (1 + 2.0 ** -6)
        err = np.abs(o[b].reshape(n, Hkv, G, D).transpose(1, 0, 2, 3) - want)
        worst = max(worst, (err / lim).max())
    announce("  worst error / bound %.3f" % worst)
    assert worst <= 1


@pytest.mark.parametrize("D", [64, 128])
def test_attend_fp32_logits_of_many_small_products(D):
    """Two tokens: one's product with q is 1, the other's 1 and, in every fourth
    channel but one, 0.9 * 2^-24 more, each less than half of fp32's step at 1.
    Their values are -1 and 1, so that o = tanh(scale * difference / 2).  Summed
    in four parts of D / 16 products that are not 0, a logit is off by at most
    (D / 16 + 3) u with u = 2^-24 (one sum would lose all D / 4 - 1 of them); that
    many times scale / 2, and 24 u of the weights and their sum, is o's bound."""
    announce("attend fp32 logits D=%d" % D)
    u, scale = 2.0 ** -24, 64.0
    small = [16 * i + e for i in range(D // 16) for e in range(4)][1:]
    kc, vc = (torch.zeros((1, 1, 16, D), device=DEV) for _ in range(2))
    q = torch.zeros((1, 1, 1, D), device=DEV)
    q[..., [0] + small] = 1
    kc[0, 0, :2, 0] = 1
    kc[0, 0, 1, small] = 0.9 * u
    vc[0, 0, 0], vc[0, 0, 1] = -1, 1
    o = gdr.attention_decode(q, kc, vc, i32([[0]]), i32([2]), scale=scale).double().cpu().numpy()
    diff = kc[0, 0, 1, small].double().sum().item()
    err = np.abs(o - np.tanh(scale * diff / 2)).max()
    lim = (D / 16 + 3) * u * scale / 2 + 24 * u
    announce("  error / bound %.3f" % (err / lim))
    assert err <= lim


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("n,G", [(1, 4), (5, 4), (10, 4)])
def test_attend_infinite_values_of_attended_tokens(dt, bad, n, G):
    """Every row attends to the tokens before the new ones: an infinite value of
    one of them is the row's result in that channel, also where the token's
    weight is a short binary number (the row's maximum, or all weights equal)."""
    announce("attend infinite values %s %s n=%d G=%d" % (dt, bad, n, G))
    B, Hkv, D, page, L = 2, 2, 64, 16, 150
    M = (48 << 20) // (B * Hkv * D * 4 * page)         # blocks of 64 rows where there are over 32
    g = torch.Generator(device=DEV).manual_seed(3)
    kc, vc = (torch.randn((B * 10, Hkv, page, D), device=DEV, generator=g).to(DTYPES[dt])
              for _ in range(2))
    q = torch.randn((B, n, Hkv * G, D), device=DEV, generator=g).to(DTYPES[dt])
    q[1] = 0                                           # all weights equal
    table = torch.full((B, M), -1, device=DEV, dtype=torch.int32)
    table[:, :10] = torch.arange(B * 10, device=DEV, dtype=torch.int32).view(B, 10)
    lens = i32([L] * B)
    clean = gdr.attention_decode(q, kc, vc, table, lens)
    s = torch.einsum("rd,hjd->rhj", q[0].reshape(-1, D).float(),
                     kc[:10].transpose(0, 1).reshape(Hkv, -1, D).float())
    top = int(s[0, 0, :L - n].argmax())                # the first row's maximum of these
    for b, j, c in ((0, top, 3), (0, 40, 5), (1, 0, 7), (1, L - n - 1, 11)):
        vc[b * 10 + j // page, :, j % page, c] = bad
        clean[b, :, :, c] = bad
    o = gdr.attention_decode(q, kc, vc, table, lens)
    torch.cuda.synchronize(DEV)
    assert torch.equal(o, clean)


# ------------------------------------- long slots, and more sequences than split
def check_rows(o, q, kc, vc, table, lens, scale, which, what):
    """o of the sequences `which` against 64 bits on the GPU.  With u = 2^-24, N
    tokens, products of D terms, the bound of each row is that of fp32 logits,
    weights and sums (a weight off by 2 e + (N + 16) u, e the largest logit's
    error), of weights as two bf16 numbers (2^-15 + 2^-22, none in fp32), of the
    sum over 2 N products, and of storing o (2^-8 or u)."""
    B, n, Hq, D = q.shape
    P, Hkv, page, _ = kc.shape
    G, u = Hq // Hkv, 2.0 ** -24
    bf16 = q.dtype == torch.bfloat16
    worst = 0.0
    for b in which:
        L = lens[b]
        if L == 0:
            assert bool((o[b] == 0).all())
            continue
        j = torch.arange(L, device=DEV)
        pg = table[b].long()[j // page]
        j = j[(pg >= 0) & (pg < P)]
        pg = pg[(pg >= 0) & (pg < P)]
        k, v = (x[pg, :, j % page].transpose(0, 1).contiguous().double() for x in (kc, vc))
        qb = q[b].double().view(n, Hkv, G, D).transpose(0, 1).reshape(Hkv, n * G, D)
        s = scale * torch.matmul(qb, k.transpose(1, 2).contiguous())
        pos = (L - n + torch.arange(n, device=DEV)).repeat_interleave(G)
        seen = j[None, :] <= pos[:, None]
        s = s.masked_fill(~seen[None], -float("inf"))
        w = torch.nan_to_num(torch.softmax(s, -1))
        want = torch.matmul(w, v)
        size = torch.matmul(w, v.abs())
        e = ((D + 2) * u * abs(scale) * torch.matmul(qb.abs(), k.abs().transpose(1, 2).contiguous()).amax(-1)
             + 8 * u * s.masked_fill(~seen[None], 0).abs().amax(-1) + 4 * u)
        N = len(j)
        rel = 2 * e + (N + 16 + 2 * N + 16) * u + (2.0 ** -15 + 2.0 ** -22 if bf16 else 0)
        lim = (rel[..., None] * size + (2.0 ** -8 if bf16 else u) * want.abs()) * (1 + 2.0 ** -6)
        got = o[b].double().view(n, Hkv, G, D).transpose(0, 1).reshape(Hkv, n * G, D)
        err = (got - want).abs()
        bad = err > lim
        assert not bool(bad.any()), "%s: sequence %d at %s" % (what, b, bad.nonzero()[:4].tolist())
        worst = max(worst, (err / lim.clamp_min(1e-300)).max().item())
    announce("  %s worst error / bound %.3f" % (what, worst))


# (sequences of about a third of a slot's tokens, 32 heads, so that 12 slots of
# them fill the card; a wave holds the page numbers of 64 of its tiles: 8,192
# tokens of a slot, fp32 4,096, blocks of 64 rows 2,048)
@pytest.mark.parametrize("dt,n,G,lens", [
    ("bf16", 1, 4, [26000, 26100, 25900, 26000]),
    ("bf16", 5, 4, [26000, 3, 51000, 26000]),
    ("bf16", 10, 4, [7000, 20001, 0, 7000]),
    ("fp32", 2, 3, [13000, 13100, 1, 26000])])
@pytest.mark.parametrize("D,page", [(64, 64), (128, 16)])
def test_attend_slots_past_the_pages_held(dt, n, G, lens, D, page):
    announce("attend long slots %s n=%d G=%d D=%d page=%d" % (dt, n, G, D, page))
    Hkv, P = 32, 200
    g = torch.Generator(device=DEV).manual_seed(D + n)
    kc, vc = (torch.randn((P, Hkv, page, D), device=DEV, generator=g).to(DTYPES[dt]) for _ in range(2))
    q = (2 * torch.randn((len(lens), n, Hkv * G, D), device=DEV, generator=g)).to(DTYPES[dt])
    # pages may be shared, a sequence's own ones too; some are absent
    table = torch.randint(-1, P + 1, (len(lens), -(-max(lens) // page) + 1), device=DEV, generator=g,
                          dtype=torch.int32)
    o = gdr.attention_decode(q, kc, vc, table, i32(lens))
    check_rows(o, q, kc, vc, table, lens, D ** -0.5, range(len(lens)), "long slots")


@pytest.mark.parametrize("B", [65536, 65537])
@pytest.mark.parametrize("dt,width,long,scored", [("bf16", 600, 9500, False), ("fp32", 64, 1000, True)])
def test_attend_most_sequences(B, dt, width, long, scored):
    """The most sequences whose slots are shared out, and one more: each is one
    slot then, however long."""
    announce("attend %d sequences %s scores=%s" % (B, dt, scored))
    D, page, G = 64, 16, 2
    g = torch.Generator(device=DEV).manual_seed(B)
    need = -(-long // page)
    P = B + need
    kc, vc = (torch.randn((P, 1, page, D), device=DEV, generator=g).to(DTYPES[dt]) for _ in range(2))
    lens = torch.randint(0, 17, (B,), device=DEV, generator=g, dtype=torch.int32)
    pages = torch.randperm(P, device=DEV, generator=g, dtype=torch.int32)
    table = torch.full((B, width), -1, device=DEV, dtype=torch.int32)
    table[:, 0] = pages[:B]
    at = B // 3
    lens[at] = long
    table[at, 1:need] = pages[B:B + need - 1]
    q = (2 * torch.randn((B, 1, G, D), device=DEV, generator=g)).to(DTYPES[dt])
    sc = torch.zeros((P, 1, page), device=DEV) if scored else None
    o = gdr.attention_decode(q, kc, vc, table, lens, scores=sc)
    host = lens.tolist()
    which = [0, 1, at, B - 2, B - 1] + list(range(5, B, B // 300))
    check_rows(o, q, kc, vc, table, host, D ** -0.5, which, "sequences")
    assert bool((o[lens == 0] == 0).all()) and bool(torch.isfinite(o).all())
    if scored:
        # a sequence's weights sum to the G rows that it has: off by at most
        # (2 e + (N + 16) u) relative, far below 2^-12
        each = torch.zeros(P, device=DEV, dtype=torch.float64)
        each[:] = sc.double().sum((1, 2))
        total = torch.where(table >= 0, each[table.long().clamp_min(0)], 0.0).sum(1)
        want = torch.where(lens > 0, float(G), 0.0).double()
        assert bool(((total - want).abs() <= 2.0 ** -12 * G).all())


def test_tables_past_2_31_pages_are_refused():
    """(Of no sequences, which takes no memory.)  A C int would hold the low 32
    bits of such a width."""
    table = torch.empty((0, 2 ** 32 + 2), device=DEV, dtype=torch.int32)
    kc, sc = torch.zeros((3, 1, 16, 64), device=DEV), torch.zeros((3, 1, 16), device=DEV)
    none, k = i32([]), torch.zeros((0, 1, 1, 64), device=DEV)
    for call in (lambda: gdr.cache_append(k, k, none, table, kc, kc.clone()),
                 lambda: gdr.attention_decode(k, kc, kc.clone(), table, none),
                 lambda: gdr.cache_evict(kc, kc.clone(), sc, table, none, 4),
                 lambda: gdr.cache_evict(kc, kc.clone(), sc, table[:, :2].contiguous(), none, 4,
                                         new_page_table=table)):
        with pytest.raises(gdr.GdrError, match="too large"):
            call()


# --------------------------- several launches: captured, and two calls at once
def same(a, b):
    """Equal bit for bit (NaN included)."""
    kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.shape == b.shape and torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def paged(lens, Hkv, D, page, width, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-l // page) for l in lens]
    P = sum(need) + 1
    kc, vc = (torch.randn((P, Hkv, page, D), device=DEV, generator=g).bfloat16() for _ in range(2))
    sc = torch.rand((P, Hkv, page), device=DEV, generator=g)
    table = np.full((len(lens), width), -1, np.int32)
    order, at = np.random.default_rng(seed).permutation(P), 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    return kc, vc, sc, i32(table), i32(lens)


def many_short(seed):
    """300 sequences, two of them split: a launch finds the slots' owners."""
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(0, 40, 300)]
    lens[7], lens[250] = 1500 + seed, 900
    kc, vc, sc, table, dl = paged(lens, 1, 64, 16, 110, seed)
    q = torch.randn((300, 2, 4, 64), device=DEV).bfloat16()
    ws = torch.empty(gdr.attention_workspace_bytes(300, 2, 4, 1, 64, 110, 16, True), device=DEV,
                     dtype=torch.uint8)
    inputs = [q, kc, vc, sc, dl]

    def call(q, kc, vc, sc, dl, ws):
        return [gdr.attention_decode(q, kc, vc, table, dl, scores=sc, workspace=ws), sc]
    return inputs, ws, call


def long_trim(seed):
    """Two pairs of 9,000 tokens and more, in place: a launch per digit."""
    kc, vc, sc, table, dl = paged([9000 + seed, 8700], 1, 64, 128, 80, seed)
    ws = torch.empty(gdr.evict_workspace_bytes(2, 1, 80, 128), device=DEV, dtype=torch.uint8)
    assert ws.numel() > 0

    def call(kc, vc, sc, dl, ws):
        nl, kept = gdr.cache_evict(kc, vc, sc, table, dl, 3001, 200, 4, workspace=ws)
        return [nl, kept, kc, vc, sc]
    return [kc, vc, sc, dl], ws, call


@pytest.mark.parametrize("make", [many_short, long_trim])
def test_several_launches_captured(make):
    """Replays on new contents equal eager calls made between them."""
    announce("capture %s" % make.__name__)
    inputs, ws, call = make(1)
    held = [x.clone() for x in inputs]
    call(*[x.clone() for x in inputs], ws)
    torch.cuda.synchronize(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(*held, ws)
    for rep in range(3):
        announce("  replay %d" % rep)
        new = [x.clone() for x in inputs]
        for x in new:
            if x.is_floating_point():
                x.copy_(torch.rand(x.shape, device=DEV).to(x.dtype))
            else:
                x.sub_(rep * (x > 50).int())
        want = call(*[x.clone() for x in new], torch.empty_like(ws))
        for x, y in zip(held, new):
            x.copy_(y)
        torch.cuda.synchronize(DEV)
        graph.replay()
        torch.cuda.synchronize(DEV)
        for a, b in zip(out, want):
            assert same(a, b), rep


@pytest.mark.parametrize("make", [many_short, long_trim])
def test_several_launches_on_two_streams(make):
    announce("two streams %s" % make.__name__)
    runs = [make(2), make(3)]
    want = [call(*[x.clone() for x in inputs], ws) for inputs, ws, call in runs]
    streams = [torch.cuda.Stream(DEV) for _ in runs]
    for rep in range(3):
        copies = [[x.clone() for x in inputs] for inputs, _, _ in runs]
        torch.cuda.synchronize(DEV)
        got = []
        for st, c, (_, ws, call) in zip(streams, copies, runs):
            with torch.cuda.stream(st):
                got.append(call(*c, ws))
        torch.cuda.synchronize(DEV)
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert same(x, y), rep
