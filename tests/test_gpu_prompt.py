"""GPU tests of attention over whole prompts and of its gradients against their
64-bit reference (tests/prompt_ref.py).  Rows behind the last sequence are
poisoned with NaN and must keep their bytes."""
import numpy as np
import pytest
import torch

import gated_delta_rule_44_amd as gdr
from tests import prompt_ref as ref
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


def offsets(lens):
    return [0] + list(np.cumsum(lens))


def make(lens, Hq, Hkv, D, dt, seed, tail=0, amp=2.0):
    """q, k, v, do as flat rows (CPU), `tail` rows of NaN behind the last."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    out = []
    for H, a in ((Hq, amp), (Hkv, 1.0), (Hkv, 1.0), (Hq, 1.0)):
        x = torch.full((T + tail, H, D), NAN, dtype=dt)
        x[:T] = (a * torch.randn((T, H, D), generator=g)).to(dt)
        out.append(x)
    return out


def within(what, got, want, bound):
    rows = ~torch.isnan(want)
    err = (got.double().cpu() - want).abs()
    assert not torch.isnan(err[rows]).any(), "%s: NaN at %s" % (
        what, torch.isnan(err).logical_and(rows).nonzero()[:4].tolist())
    ratio = (err[rows] / bound[rows].clamp(min=1e-300)).max().item() if rows.any() else 0.0
    announce("  %s: worst error / bound %.3f" % (what, ratio))
    assert ratio <= 1, "%s: at %s" % (what, (rows & (err > bound)).nonzero()[:4].tolist())


def shaped(x, B):
    """Flat rows as a fixed-length batch."""
    return x if B is None else x.view(B, -1, *x.shape[1:])


def run_forward(data, cu, scale, window, fixed=None, **kw):
    """One call on poisoned outputs; returns o and lse as flat rows."""
    q, k, v = (shaped(x.to(DEV), fixed) for x in data[:3])
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:-1], 7.0, device=DEV)
    offs = None if fixed is not None else i32(cu)
    r = gdr.attention_prefill(q, k, v, cu_seqlens=offs, scale=scale, window=window, lse=lse, o=o,
                              **kw)
    sync()
    assert r[0] is o and r[1] is lse
    for x, y in zip((q, k, v), data):
        assert same(x.reshape(y.shape), y), "an input changed"
    return o.view(data[0].shape), lse.view(data[0].shape[:2])


def run_backward(data, o, lse, cu, scale, window, fixed=None, **kw):
    q, k, v, do = (shaped(x.to(DEV), fixed) for x in data)
    grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
    offs = None if fixed is not None else i32(cu)
    gdr.attention_backward(q, k, v, shaped(o, fixed), shaped(lse, fixed), do, cu_seqlens=offs,
                           scale=scale, window=window, dq=grads[0], dk=grads[1], dv=grads[2], **kw)
    sync()
    return [g.view(x.shape) for g, x in zip(grads, data)]


def check(data, lens, scale, window=0, fixed=None, what="", grads=True):
    cu = offsets(lens)
    o, lse = run_forward(data, cu, scale, window, fixed)
    want = ref.forward(*data[:3], cu, scale, window)
    within(what + " o", o, want[0], want[2])
    within(what + " lse", lse, want[1], want[3])
    T = cu[-1]
    assert (o[T:] == 7).all() and (lse[T:] == 7).all(), "rows behind the last sequence"
    got = None
    if grads:
        got = run_backward(data, o, lse, cu, scale, window, fixed)
        want, bound = ref.backward(*data[:3], o.cpu(), lse.cpu(), data[3], cu, scale, window)
        for name, x, y, z in zip(("dq", "dk", "dv"), got, want, bound):
            within("%s %s" % (what, name), x, y, z)
            assert (x[T:] == 7).all(), "rows behind the last sequence"
    # the same bits without lse and on a second run
    q, k, v = (shaped(x.to(DEV), fixed) for x in data[:3])
    offs = None if fixed is not None else i32(cu)
    again = gdr.attention_prefill(q, k, v, cu_seqlens=offs, scale=scale, window=window)
    assert same(again.view(o.shape)[:T], o[:T])
    if grads:
        for x, y in zip(got, run_backward(data, o, lse, cu, scale, window, fixed)):
            assert same(x, y)
    return o, lse, got


LENS = [1, 0, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200]
SHAPES = [
    # D, Hkv, G, window
    (128, 2, 1, 0),
    (128, 1, 4, 0),
    (64, 2, 3, 0),
    (64, 1, 8, 0),
    (128, 2, 2, 1),
    (64, 1, 2, 2),
    (128, 1, 3, 50),
    (64, 2, 1, 64),
    (128, 1, 1, 129),
    (64, 3, 1, 1000),
    # (many heads: blocks of 128 rows in place of 32)
    (128, 9, 1, 0),
    (64, 9, 1, 0),
    (128, 8, 2, 50),
    (64, 10, 1, 64),
    (128, 9, 1, 129),
]


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D,Hkv,G,window", SHAPES)
def test_packed(dt, D, Hkv, G, window):
    announce("packed %s D=%d Hkv=%d G=%d window=%d" % (dt, D, Hkv, G, window))
    data = make(LENS, Hkv * G, Hkv, D, DTYPES[dt], seed=D + G, tail=9)
    check(data, LENS, D ** -0.5, window, what="packed")


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,D,Hkv,G,window", [
    (1, 1, 128, 1, 1, 0), (3, 1, 64, 2, 2, 0), (2, 40, 128, 2, 2, 0), (3, 130, 64, 1, 3, 0),
    (2, 257, 128, 1, 2, 0), (1, 700, 64, 2, 2, 0), (1, 650, 128, 1, 5, 300), (2, 300, 64, 1, 1, 31)])
def test_fixed(dt, B, T, D, Hkv, G, window):
    announce("fixed %s B=%d T=%d D=%d Hkv=%d G=%d window=%d" % (dt, B, T, D, Hkv, G, window))
    data = make([T] * B, Hkv * G, Hkv, D, DTYPES[dt], seed=T)
    check(data, [T] * B, D ** -0.5, window, fixed=B, what="fixed")


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_scales(dt):
    """Scales of other sizes and signs, zero among them, and large logits."""
    lens = [70, 3, 150]
    data = make(lens, 4, 2, 64, DTYPES[dt], seed=3, tail=3)
    for scale in (0.0, -0.125, 1.0, 2.5, 1e-30, -3.0):
        check(data, lens, scale, what="scale %g" % scale)


def test_many_sequences():
    """More sequences than one search of 64 lanes tells apart."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 4, 5000)]
    lens[4321], lens[0], lens[-1] = 200, 0, 70
    data = make(lens, 2, 1, 64, torch.bfloat16, seed=6, tail=5)
    check(data, lens, 0.125, what="5,000 sequences")
    lens = lens[:100]
    data = make(lens, 2, 1, 64, torch.float32, seed=6, tail=5)
    check(data, lens, 0.125, what="100 sequences")


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("window,H", [(0, 2), (40, 2), (0, 30), (40, 30)])
def test_masked_values(dt, window, H):
    """Infinities and NaN of tokens that a row does not attend to have no part
    in its results; those that it attends to have."""
    lens, D = [150, 90, 70], 64
    cu = offsets(lens)
    data = make(lens, H, H, D, DTYPES[dt], seed=8)
    clean = check(data, lens, D ** -0.5, window, what="clean")
    bad = cu[1] + 37                             # a token of the second sequence
    seen = torch.zeros(cu[-1], dtype=torch.bool)  # rows that attend to it
    seen[bad:cu[2] if window == 0 else min(cu[2], bad + window)] = True
    heard = torch.zeros(cu[-1], dtype=torch.bool)  # tokens it attends to
    heard[max(cu[1], bad - window + 1) if window else cu[1]:bad + 1] = True
    for name, n, x in (("q", 0, NAN), ("q", 0, INF), ("k", 1, NAN), ("k", 1, -INF), ("v", 2, NAN),
                       ("v", 2, INF), ("v", 2, -INF), ("do", 3, NAN), ("do", 3, INF)):
        mine = [y.clone() for y in data]
        mine[n][bad, :, 3] = x
        o, lse = run_forward(mine, cu, D ** -0.5, window)
        rows = torch.zeros_like(seen)            # rows the value may reach
        if name == "q":
            rows[bad] = True
        elif name in "kv":
            rows = seen
        what = "%s = %g" % (name, x)
        assert same(o[~rows], clean[0][~rows]), what
        assert same(lse[~rows], clean[1][~rows]), what
        if name == "v":
            # the one channel, by infinities of that sign
            want = clean[0].clone()
            want[seen, :, 3] = x
            assert same(torch.nan_to_num(o, NAN), torch.nan_to_num(want, NAN)), what
            assert same(lse, clean[1])
        elif name == "k" and x != x:
            assert torch.isnan(o[seen]).all() and torch.isnan(lse[seen]).all(), what
        got = run_backward(mine, o, lse, cu, D ** -0.5, window)
        # a row's dq depends on it and its tokens; a token's dk and dv on it, the
        # rows that attend to it and what these rows attend to (through o, lse)
        own = torch.zeros_like(seen)
        own[bad] = True
        touched_q = (own if name in ("q", "do") else seen)
        reach = heard.clone()
        if name in "kv":
            last = int(seen.nonzero()[-1])
            reach[:] = False
            reach[max(cu[1], bad - window + 1) if window else cu[1]:last + 1] = True
        for which, g, c, t in zip(("dq", "dk", "dv"), got, clean[2], (touched_q, reach, reach)):
            assert same(g[~t], c[~t]), "%s: %s" % (what, which)


def test_weights_that_vanish():
    """Rows whose logits are all -inf give zeros and lse = -inf, and no
    gradients; a row with some such logits ignores them."""
    lens, D = [40, 100], 64
    data = make(lens, 2, 2, D, torch.float32, seed=9)
    q, k, v, do = data
    q[:, :, 0] = q[:, :, 0].abs() + 0.1
    k[20:40, :, 0] = -INF                        # the first sequence's last tokens
    k[40:, :, 0] = -INF                          # the second: all of them
    cu = offsets(lens)
    o, lse = run_forward(data, cu, D ** -0.5, 0)
    assert (o[40:] == 0).all() and (lse[40:] == -INF).all()
    want = ref.forward(q, k, v, cu, D ** -0.5)
    within("o", o, want[0], want[2])
    within("lse of rows with weights", lse[:40], want[1][:40], want[3][:40])
    got = run_backward(data, o, lse, cu, D ** -0.5, 0)
    # (a row's dq in the channel where its keys are infinite is 0 times that)
    assert (got[0][40:, :, 1:] == 0).all() and (got[2][40:] == 0).all()


def test_long():
    """Rows far from the sequence's start, sampled, both passes' last tiles."""
    T, D = 5000, 128
    data = make([T], 2, 1, D, torch.bfloat16, seed=11)
    check(data, [T], D ** -0.5, what="5,000 tokens")
    check(data, [T], D ** -0.5, 700, what="a window of 700")
    for dt in (torch.float32, torch.bfloat16):
        data = make([2100], 8, 8, D, dt, seed=12)
        check(data, [2100], D ** -0.5, what="8 heads")


def test_bad_offsets_stay_inside():
    """Offsets that decrease or leave the rows (the host copy is not given):
    what the call computes is unspecified, where it reads and writes is not."""
    data = make([100, 60], 2, 1, 64, torch.bfloat16, seed=12)
    for cu in ([0, 150, 90], [-5, 70, 400], [0, 400, 160], [160, 0, 160], [-(1 << 31), 3, (1 << 31) - 1]):
        o, lse = run_forward(data, cu, 0.125, 0)
        run_backward(data, o, lse, cu, 0.125, 0)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("B,window", [(63, 0), (64, 0), (64, 90), (65, 0), (2, 0)])
def test_longest_blocks_first(dt, B, window):
    """Batches of few rounds of workgroups, whose longest blocks go first where they
    have up to 64 sequences; empty ones, and of equal lengths, among them."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.choice([0, 1, 127, 128, 129, 300], B)]
    lens[0], lens[-1] = 500, 260
    H = 560 // (sum(lens) // 128 + B) + 2
    data = make(lens, H, H, 64, DTYPES[dt], seed=B, tail=2)
    check(data, lens, 0.125, window, what="%d sequences of %d heads" % (B, H))


@pytest.mark.parametrize("B,T,H", [(3, 300, 70), (7, 129, 40), (5, 513, 25)])
def test_longest_blocks_first_fixed(B, T, H):
    data = make([T] * B, H, H, 64, torch.bfloat16, seed=T)
    check(data, [T] * B, 0.125, fixed=B, what="%d x %d" % (B, T))


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("H", [1, 70])
def test_backward_workspace_is_enough(dt, H):
    """Nothing is written past the bytes that the library asks for, by either
    form (blocks of 32 rows and of 128)."""
    lens, D = [200, 1, 77], 64
    data, cu = make(lens, H, H, D, DTYPES[dt], seed=31), offsets(lens)
    o, lse = run_forward(data, cu, 0.125, 0)
    want = run_backward(data, o, lse, cu, 0.125, 0)
    need = gdr.attention_backward_workspace_bytes(DTYPES[dt], 3, 278, H, H, D)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    got = run_backward(data, o, lse, cu, 0.125, 0, workspace=ws[:need])
    assert (ws[need:] == 0x5A).all()
    for x, y in zip(got, want):
        assert same(x, y)
    with pytest.raises(gdr.GdrError, match="workspace"):
        run_backward(data, o, lse, cu, 0.125, 0, workspace=ws[:need - 16])


@pytest.mark.parametrize("packed", [False, True])
def test_streams_and_graphs(packed):
    """On another stream, two at once, and captured: every replay on new
    contents equals the eager call."""
    lens, D = [130, 130], 128
    cu = offsets(lens)
    fixed = None if packed else 2
    sets = [make(lens, 4, 2, D, torch.bfloat16, seed=20 + i) for i in range(3)]
    eager = []
    for x in sets:
        o, lse = run_forward(x, cu, 0.1, 50, fixed)
        eager.append((o.clone(), lse.clone(), run_backward(x, o, lse, cu, 0.1, 50, fixed)))
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    outs = []
    for x, s in zip(sets, streams):
        q, k, v, do = (shaped(y.to(DEV), fixed) for y in x)
        offs = i32(cu) if packed else None
        sync()
        with torch.cuda.stream(s):
            o, lse = gdr.attention_prefill(q, k, v, cu_seqlens=offs, scale=0.1, window=50, lse=True)
            outs.append((o, lse, gdr.attention_backward(q, k, v, o, lse, do, cu_seqlens=offs,
                                                        scale=0.1, window=50)))
    sync()
    for got, want in zip(outs, eager):
        assert same(got[0].view(want[0].shape), want[0]) and same(got[1].view(want[1].shape), want[1])
        for x, y in zip(got[2], want[2]):
            assert same(x.view(y.shape), y)
    q, k, v, do = (shaped(y.to(DEV), fixed) for y in sets[0])
    offs = i32(cu) if packed else None
    o, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device=DEV)
    grads = [torch.empty_like(x) for x in (q, k, v)]
    ws = torch.empty(gdr.attention_backward_workspace_bytes(torch.bfloat16, 2, 260, 4, 2, D),
                     device=DEV, dtype=torch.uint8)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.attention_prefill(q, k, v, cu_seqlens=offs, scale=0.1, window=50, lse=lse, o=o)
        gdr.attention_backward(q, k, v, o, lse, do, cu_seqlens=offs, scale=0.1, window=50,
                               dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
    for i in (1, 2, 0, 1):
        for x, y in zip((q, k, v, do), sets[i]):
            x.copy_(y.to(DEV).view(x.shape))
        sync()
        graph.replay()
        sync()
        want = eager[i]
        assert same(o.view(want[0].shape), want[0]) and same(lse.view(want[1].shape), want[1])
        for x, y in zip(grads, want[2]):
            assert same(x.view(y.shape), y)


def test_gradients_by_differences():
    """fp32: the slope of sum(do . o) along random directions."""
    lens, D, scale = [37, 70], 64, 0.125
    cu = offsets(lens)
    data = make(lens, 4, 2, D, torch.float32, seed=31, amp=1.0)
    o, lse = run_forward(data, cu, scale, 20)
    grads = run_backward(data, o, lse, cu, scale, 20)
    g = torch.Generator().manual_seed(1)
    eps = 2.0 ** -6
    for n in range(3):
        d = torch.randn(data[n].shape, generator=g)
        d /= d.norm()
        vals = []
        for sign in (1, -1):
            x = [y.clone() for y in data]
            x[n] = x[n] + sign * eps * d
            y, _ = run_forward(x, cu, scale, 20)
            vals.append(float((y.double().cpu() * data[3].double()).sum()))
        slope = (vals[0] - vals[1]) / (2 * eps)
        want = float((grads[n].double().cpu() * d.double()).sum())
        # o's rounding: 2^-22 of |o| each side, over eps; the third derivative
        # times eps^2 / 6, of the size of the gradient's norm at most
        tol = (2.0 ** -22 * float((o.double().cpu() * data[3].double()).norm()) / eps * 8
               + eps ** 2 * float(grads[n].double().norm()))
        announce("  slope %d: %.6g against %.6g (%.1e)" % (n, slope, want, tol))
        assert abs(slope - want) <= tol


def test_refuses():
    q = torch.zeros(2, 8, 4, 64, device=DEV)
    k = torch.zeros(2, 8, 2, 64, device=DEV)
    cu = i32([0, 8, 16])
    flat = lambda x: x.view(-1, *x.shape[2:])  # noqa: E731
    call = gdr.attention_prefill
    for args, kw, msg in [
        ((q.cpu(), k, k), {}, "q must be a GPU tensor"),
        ((q.half(), k.half(), k.half()), {}, "bfloat16 or float32"),
        ((q, k.bfloat16(), k), {}, "k must be"),
        ((q, k, k[:, :4]), {}, "v must be"),
        ((q, k[:, :4].contiguous(), k[:, :4].contiguous()), {}, "must be"),
        ((q, k, k.transpose(1, 2)), {}, "v must be contiguous"),
        ((q[:, :, :3].contiguous(), k, k), {}, "multiple"),
        ((flat(q), flat(k), flat(k)), {}, "q must be"),
        ((q, k, k), dict(cu_seqlens=cu), "q must be"),
        ((q, k, k), dict(cu_seqlens_host=[0, 8, 16]), "without cu_seqlens"),
        ((flat(q), flat(k), flat(k)), dict(cu_seqlens=cu.long()), "cu_seqlens must be"),
        ((flat(q), flat(k), flat(k)), dict(cu_seqlens=cu, cu_seqlens_host=[0, 8]), "entries"),
        ((flat(q), flat(k), flat(k)), dict(cu_seqlens=cu, cu_seqlens_host=[0, 9, 8]), "decreases"),
        ((q, k, k), dict(window=-1), "window"),
        ((q, k, k), dict(scale=float("nan")), "scale"),
        ((q, k, k), dict(lse=torch.zeros(2, 8, 3, device=DEV)), "lse must be"),
        ((q, k, k), dict(o=torch.zeros(2, 8, 4, 64, device=DEV).bfloat16()), "o must be"),
        ((q[..., :32].contiguous(), k[..., :32].contiguous(), k[..., :32].contiguous()), {},
         "supported widths"),
    ]:
        with pytest.raises(gdr.GdrError, match=msg):
            call(*args, **kw)
    o, lse = call(q, k, k, lse=True)
    with pytest.raises(gdr.GdrError, match="do must be"):
        gdr.attention_backward(q, k, k, o, lse, o[:1].contiguous())
    with pytest.raises(gdr.GdrError, match="lse must be"):
        gdr.attention_backward(q, k, k, o, lse.bfloat16(), o)
    with pytest.raises(gdr.GdrError, match="workspace"):
        gdr.attention_backward(q, k, k, o, lse, o,
                               workspace=torch.empty(16, device=DEV, dtype=torch.uint8))
    with pytest.raises(gdr.GdrError, match="dk must be"):
        gdr.attention_backward(q, k, k, o, lse, o, dk=q)


def test_empty():
    q, k = torch.zeros(0, 4, 64, device=DEV), torch.zeros(0, 2, 64, device=DEV)
    o, lse = gdr.attention_prefill(q, k, k, cu_seqlens=i32([0, 0, 0]), lse=True)
    assert o.shape == q.shape and lse.shape == (0, 4)
    assert [x.shape for x in gdr.attention_backward(q, k, k, o, lse, q, cu_seqlens=i32([0]))] == [
        q.shape, k.shape, k.shape]
    q, k = torch.ones(3, 0, 4, 64, device=DEV), torch.ones(3, 0, 2, 64, device=DEV)
    assert gdr.attention_prefill(q, k, k).shape == q.shape
