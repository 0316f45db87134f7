"""GPU tests of attention over whole prompts at the edges of its values, in both
forms (blocks of 32 rows and of 128): NaN and infinities that a row attends to,
values of V whose sums overflow, and what it writes under bad offsets."""
import pytest
import torch

import gated_delta_rule_44_amd as gdr
from tests import prompt_ref as ref
from tests.conftest import gpu_available
from tests.test_gpu_prompt import (DEV, DTYPES, INF, NAN, make, offsets, run_forward, same,
                                   within)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
FORMS = [2, 260]         # heads: blocks of 32 rows, of 128


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", FORMS)
def test_nan_that_a_row_attends_to(dt, D, H):
    """o and lse of a row are NaN where its query or a key that it attends to is,
    also where all of its keys, or all of a tile of them, are; other rows keep
    their bits."""
    lens = [150, 40, 128]
    cu = offsets(lens)
    data = make(lens, H, H, D, DTYPES[dt], seed=D)
    for what, n, bad, window, rows in [
        ("a query", 0, [70], 0, [70]),
        ("a query of one token", 0, [150], 0, [150]),
        ("a sequence's first key", 1, [150], 0, range(150, 190)),
        ("the only key of a row", 1, [60], 1, [60]),
        ("both keys of a row", 1, [60, 61], 2, [60, 61, 62]),
        ("a tile of keys", 1, range(32, 64), 0, range(32, 150)),
        ("a tile of keys in a window", 1, range(32, 64), 40, range(32, 103)),
        ("two tiles of keys", 1, range(64, 128), 0, range(64, 150)),
        ("a sequence's keys", 1, range(190, 318), 0, range(190, 318)),
    ]:
        clean = run_forward(data, cu, D ** -0.5, window)
        mine = [x.clone() for x in data]
        mine[n][list(bad), :, 3] = NAN
        o, lse = run_forward(mine, cu, D ** -0.5, window)
        hit = torch.zeros(cu[-1], dtype=torch.bool)
        hit[list(rows)] = True
        assert bool(torch.isnan(o[hit]).all()) and bool(torch.isnan(lse[hit]).all()), what
        assert same(o[~hit], clean[0][~hit]) and same(lse[~hit], clean[1][~hit]), what


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("H", FORMS)
@pytest.mark.parametrize("low", [[40], range(32, 64), range(0, 64)])
def test_infinite_values_of_small_weights(dt, H, low):
    """An infinity of V that a row attends to reaches it whatever its weight is (of
    one token, or of a tile or two whose weights all vanish beside the others'): the
    result is not finite, in no other channel."""
    lens, D = [150], 64
    data = make(lens, H, H, D, DTYPES[dt], seed=5, amp=1.0)
    data[0][:, :, 0] = 20.0
    data[1][:, :, 0] = 0.0
    data[1][list(low), :, 0] = -80.0             # logits lower by 200
    clean = run_forward(data, [0, 150], D ** -0.5, 0)
    data[2][40, :, 5] = INF
    o, lse = run_forward(data, [0, 150], D ** -0.5, 0)
    assert not torch.isfinite(o[40:, :, 5]).any()
    o[40:, :, 5] = clean[0][40:, :, 5]
    assert same(o, clean[0]) and same(lse, clean[1])


# Where sums overflow, weights are taken relative to a number 2^38 times larger: the
# terms in |s| and |m| of a weight's error (8 u each, twice) gain 38 ln 2 < 27, those of
# lse (4 u) likewise.
LIFT = 27 * 2.0 ** -24


def check_large(data, lens, scale, window, what):
    cu = offsets(lens)
    o, lse = run_forward(data, cu, scale, window)
    want = ref.forward(*data[:3], cu, scale, window)
    size = ref.forward(data[0], data[1], data[2].abs(), cu, scale, window)[0]   # sum w |v|
    within(what + " o", o, want[0], want[2] + 16 * LIFT * size)
    within(what + " lse", lse, want[1], want[3] + 20 * LIFT)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", FORMS)
def test_large_values(dt, D, H):
    """Values up to 2^127: their sums overflow, o does not; in a single channel and
    row as in all, and beside infinities that other rows attend to."""
    lens, scale = [300, 40], D ** -0.5
    for window in (0, 70):
        data = make(lens, H, H, D, DTYPES[dt], seed=D + 1)
        v = data[2]
        v.copy_((v.sign() * (0.5 + v.abs().clamp(max=1) / 2)).double() * 2.0 ** 127)
        check_large(data, lens, scale, window, "all")
        v[:, :, ::2] = v[:, :, ::2].sign()
        v[:100] = v[:100].sign()
        check_large(data, lens, scale, window, "some")
        v.copy_(v.abs())
        check_large(data, lens, scale, window, "of one sign")
    # rows before an infinity keep what they have without it
    clean = run_forward(data, offsets(lens), scale, 0)
    data[2][200, :, 1] = -INF
    o, lse = run_forward(data, offsets(lens), scale, 0)
    hit = torch.zeros(340, dtype=torch.bool)
    hit[200:300] = True
    assert (o[hit][:, :, 1] == -INF).all() and same(lse, clean[1])
    o[200:300, :, 1] = clean[0][200:300, :, 1]
    assert same(o, clean[0])


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("H", FORMS)
def test_large_values_behind_a_maximum(dt, H):
    """Logits that grow by a little under 8 ln 2 after the first tile: the weights of
    all later tokens are near 2^8 beside a maximum that is left behind."""
    lens, D = [400], 64
    data = make(lens, H, H, D, DTYPES[dt], seed=4, amp=0.0)
    data[0][:, :, 0] = 8.0
    data[1][:, :, 0] = 0.0
    data[1][64:, :, 0] = 5.5                     # logits of 5.5 after 64 of 0
    for big in (2.0 ** 105, 2.0 ** 112, 2.0 ** 118, 2.0 ** 127):
        data[2].copy_(data[2].sign() * big)
        data[2][:, :, 5] = big
        check_large(data, lens, D ** -0.5, 0, "values of %g" % big)


def guarded(like, pad=1 << 20):
    """A tensor like that one between `pad` bytes that are to keep their value."""
    n = like.numel() * like.element_size()
    raw = torch.full((pad + n + pad,), 0x5A, dtype=torch.uint8, device=DEV)
    return raw, raw[pad:pad + n].view(like.dtype).view(like.shape), pad


def untouched(raw, pad):
    return bool((raw[:pad] == 0x5A).all()) and bool((raw[-pad:] == 0x5A).all())


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("H,D", [(2, 64), (260, 64), (260, 128)])
@pytest.mark.parametrize("window", [0, 50])
def test_bad_offsets_write_inside(dt, H, D, window):
    """Offsets that decrease, overlap or leave the rows (the host copy is not given):
    what the call computes is unspecified, but it writes within its outputs and its
    workspace only; of up to 64 sequences (whose longest blocks may go first) and of
    more."""
    T, far = 300, (1 << 31) - 1
    data = [x.to(DEV) for x in make([T], H, H, D, DTYPES[dt], seed=12)]
    q, k, v, do = data
    for cu in ([0, 250, 90], [-5, 70, 400], [0, 400, 160], [T, 0, T], [-far - 1, 3, far],
               [0, T] * 32 + [0], [T, 0] * 33, list(range(T, T - 130, -2)), [0] * 30 + [T] * 35 + [-1] * 9):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        ro, o, pad = guarded(q)
        rl, lse, _ = guarded(torch.empty((T, H), device=DEV))
        o.zero_()
        lse.zero_()
        gdr.attention_prefill(q, k, v, cu_seqlens=cu, scale=0.125, window=window, lse=lse, o=o)
        outs = [guarded(x) for x in (q, k, v)]
        need = gdr.attention_backward_workspace_bytes(DTYPES[dt], cu.numel() - 1, T, H, H, D)
        rw, ws, _ = guarded(torch.zeros(need, dtype=torch.uint8, device=DEV))
        ws.zero_()
        gdr.attention_backward(q, k, v, o, lse, do, cu_seqlens=cu, scale=0.125, window=window,
                               dq=outs[0][1], dk=outs[1][1], dv=outs[2][1], workspace=ws)
        torch.cuda.synchronize(DEV)
        for raw in [ro, rl, rw] + [x[0] for x in outs]:
            assert untouched(raw, pad), cu[:4].tolist()


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("H", FORMS)
def test_padded_batches_write_inside(dt, H):
    """Outputs and workspace between guards, sequences that end inside a block and rows
    behind the last one."""
    lens, D = [1, 129, 0, 70], 128
    data = make(lens, H, H, D, DTYPES[dt], seed=13, tail=37)
    q, k, v, do = (x.to(DEV) for x in data)
    cu = torch.tensor(offsets(lens), dtype=torch.int32, device=DEV)
    want = run_forward(data, offsets(lens), D ** -0.5, 0)
    ro, o, pad = guarded(q)
    rl, lse, _ = guarded(torch.empty(q.shape[:2], device=DEV))
    o.fill_(7.0)
    lse.fill_(7.0)
    gdr.attention_prefill(q, k, v, cu_seqlens=cu, lse=lse, o=o)
    assert same(o, want[0]) and same(lse, want[1])
    outs = [guarded(x) for x in (q, k, v)]
    for _, x, _ in outs:
        x.fill_(7.0)
    need = gdr.attention_backward_workspace_bytes(DTYPES[dt], len(lens), q.shape[0], H, H, D)
    rw, ws, _ = guarded(torch.zeros(need, dtype=torch.uint8, device=DEV))
    gdr.attention_backward(q, k, v, o, lse, do, cu_seqlens=cu, dq=outs[0][1], dk=outs[1][1],
                           dv=outs[2][1], workspace=ws)
    torch.cuda.synchronize(DEV)
    for raw in [ro, rl, rw] + [x[0] for x in outs]:
        assert untouched(raw, pad)
    for _, x, _ in outs:
        assert bool((x[sum(lens):] == 7).all())


def test_refuses_heads_without_channels():
    q = torch.zeros(2, 3, 4, 0, device=DEV)
    with pytest.raises(gdr.GdrError, match="D = 0"):
        gdr.attention_prefill(q, q, q)
    with pytest.raises(gdr.GdrError, match="D = 0"):
        gdr.attention_backward(q, q, q, q, q[..., 0:0].sum(-1), q)
    table = torch.zeros(2, 1, device=DEV, dtype=torch.int32)
    cache, lens = torch.zeros(4, 4, 16, 0, device=DEV), torch.ones(2, device=DEV, dtype=torch.int32)
    with pytest.raises(gdr.GdrError, match="k_cache must be"):
        gdr.attention_decode(q, cache, cache, table, lens)
    with pytest.raises(gdr.GdrError, match="k_cache must be"):
        gdr.attention_tree(q, cache, cache, table, lens, table.expand(2, 3).contiguous())
