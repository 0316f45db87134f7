"""GPU tests of the forms of attention over whole prompts that take blocks of 128 rows
(which calls with few rows leave to blocks of 32): every type, width and pass, with
enough heads that all of them are taken, compared on some of the heads."""
import pytest
import torch

import gated_delta_rule_44_amd as gdr
from tests import prompt_ref as ref, test_gpu_prompt as base
from tests.conftest import gpu_available
from tests.gpu_util import announce
from tests.test_gpu_prompt import (DEV, DTYPES, make, offsets, run_backward, run_forward, same,
                                   within)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def check_heads(data, lens, scale, window, fixed, heads, what):
    """The key-value heads `heads` and their query heads against the reference, all of
    them over the same bits on a second run."""
    cu = offsets(lens)
    G = data[0].shape[1] // data[1].shape[1]
    rows = [h * G + g for h in heads for g in range(G)]
    o, lse = run_forward(data, cu, scale, window, fixed)
    grads = run_backward(data, o, lse, cu, scale, window, fixed)
    q, k, v, do = (x[:, i] for x, i in zip(data, (rows, heads, heads, rows)))
    T = cu[-1]
    want = ref.forward(q, k, v, cu, scale, window)
    within(what + " o", o[:, rows], want[0], want[2])
    within(what + " lse", lse[:, rows], want[1], want[3])
    want, bound = ref.backward(q, k, v, o[:, rows].cpu(), lse[:, rows].cpu(), do, cu, scale, window)
    for name, x, i, y, z in zip(("dq", "dk", "dv"), grads, (rows, heads, heads), want, bound):
        within("%s %s" % (what, name), x[:, i], y, z)
    for x in [o, lse] + grads:
        assert bool((x[T:] == 7).all()), "rows behind the last sequence"
    again = run_forward(data, cu, scale, window, fixed)
    assert same(again[0], o) and same(again[1], lse)
    for x, y in zip(grads, run_backward(data, o, lse, cu, scale, window, fixed)):
        assert same(x, y)


SHAPES = [
    # D, Hkv, G, window
    (128, 40, 1, 0),
    (64, 40, 1, 0),
    (128, 30, 3, 0),
    (64, 60, 2, 1),
    (128, 40, 1, 50),
    (64, 40, 1, 64),
    (128, 40, 2, 129),
    (64, 40, 1, 1000),
]


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("D,Hkv,G,window", SHAPES)
def test_packed(dt, D, Hkv, G, window):
    announce("packed %s D=%d Hkv=%d G=%d window=%d" % (dt, D, Hkv, G, window))
    data = make(base.LENS, Hkv * G, Hkv, D, DTYPES[dt], seed=D + G, tail=9)
    check_heads(data, base.LENS, D ** -0.5, window, None, [0, 1, Hkv // 2, Hkv - 1], "packed")


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,D,Hkv,G,window", [
    (40, 40, 128, 16, 1, 0), (3, 130, 64, 100, 3, 0), (2, 257, 128, 70, 1, 0), (1, 700, 64, 100, 2, 0),
    (1, 650, 128, 70, 1, 300), (2, 300, 64, 100, 1, 31), (1, 2100, 128, 36, 1, 0),
    (2, 1100, 64, 40, 1, 0), (1, 2100, 64, 48, 1, 700), (1, 4200, 128, 20, 1, 3000)])
def test_fixed(dt, B, T, D, Hkv, G, window):
    announce("fixed %s B=%d T=%d D=%d Hkv=%d G=%d window=%d" % (dt, B, T, D, Hkv, G, window))
    data = make([T] * B, Hkv * G, Hkv, D, DTYPES[dt], seed=T)
    check_heads(data, [T] * B, D ** -0.5, window, B, [0, Hkv - 1], "fixed")


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("B", [64, 65])
def test_packed_orders(dt, B):
    """Of up to 64 packed sequences the longest blocks of all go first, past them
    sequence by sequence."""
    lens = [(37 * i) % 211 for i in range(B)]
    data = make(lens, 16, 16, 64, DTYPES[dt], seed=B, tail=3)
    check_heads(data, lens, 0.125, 0, None, [0, 15], "%d sequences" % B)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_scales(dt):
    lens = [70, 3, 150]
    data = make(lens, 130, 130, 64, DTYPES[dt], seed=3, tail=3)
    for scale in (0.0, -0.125, 1.0, 2.5, 1e-30, -3.0):
        check_heads(data, lens, scale, 0, None, [0, 129], "scale %g" % scale)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("window", [0, 40])
def test_masked_values(dt, window):
    base.test_masked_values(dt, window, 130)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_backward_workspace_is_enough(dt):
    base.test_backward_workspace_is_enough(dt, 130)


def test_weights_that_vanish():
    """Rows whose logits are all -inf: zeros, lse = -inf, no gradients."""
    lens, D, H = [40, 100], 64, 260
    data = make(lens, H, H, D, torch.float32, seed=9)
    q, k, _, _ = data
    q[:, :, 0] = q[:, :, 0].abs() + 0.1
    k[20:, :, 0] = -base.INF                     # the first sequence's last tokens, all others
    cu = offsets(lens)
    o, lse = run_forward(data, cu, D ** -0.5, 0)
    assert not o[40:].any() and bool((lse[40:] == -base.INF).all())
    got = run_backward(data, o, lse, cu, D ** -0.5, 0)
    assert not got[0][40:, :, 1:].any() and not got[2][40:].any()


@pytest.mark.parametrize("packed", [False, True])
def test_graph(packed):
    """Captured once and replayed on new contents, in both types."""
    lens, D, H = [130, 130], 128, 130
    cu, fixed = offsets(lens), None if packed else 2
    for dt in (torch.bfloat16, torch.float32):
        sets = [make(lens, H, H, D, dt, seed=20 + i) for i in range(3)]
        eager = []
        for x in sets:
            o, lse = run_forward(x, cu, 0.1, 50, fixed)
            eager.append([o.clone(), lse.clone()] + run_backward(x, o, lse, cu, 0.1, 50, fixed))
        q, k, v, do = (base.shaped(y.to(DEV), fixed) for y in sets[0])
        offs = base.i32(cu) if packed else None
        o, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device=DEV)
        grads = [torch.empty_like(x) for x in (q, k, v)]
        ws = torch.empty(gdr.attention_backward_workspace_bytes(dt, 2, 260, H, H, D), device=DEV,
                         dtype=torch.uint8)
        base.sync()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdr.attention_prefill(q, k, v, cu_seqlens=offs, scale=0.1, window=50, lse=lse, o=o)
            gdr.attention_backward(q, k, v, o, lse, do, cu_seqlens=offs, scale=0.1, window=50,
                                   dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
        for i in (1, 2, 0, 1):
            for x, y in zip((q, k, v, do), sets[i]):
                x.copy_(y.to(DEV).view(x.shape))
            base.sync()
            graph.replay()
            base.sync()
            for x, y in zip([o, lse] + grads, eager[i]):
                assert same(x.view(y.shape), y)


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
def test_past_2_32_bytes(dt, packed):
    """Tensors of 2.2e9 elements: the first sequence and the last ones."""
    B, T, H, D, dtype = 2100, 130, 64, 128, DTYPES[dt]
    g = torch.Generator(DEV).manual_seed(1)
    shape = (B * T, H, D) if packed else (B, T, H, D)
    q, k, v, do = (torch.randn(shape, generator=g, device=DEV, dtype=dtype) for _ in range(4))
    offs = base.i32(range(0, B * T + 1, T)) if packed else None
    o, lse = gdr.attention_prefill(q, k, v, cu_seqlens=offs, lse=True)
    grads = gdr.attention_backward(q, k, v, o, lse, do, cu_seqlens=offs)
    base.sync()
    for b in (0, B - 2, B - 1):
        rows, heads = slice(b * T, (b + 1) * T), [0, H - 1]
        cut = lambda x: x.view(B * T, *x.shape[-2:])[rows][:, heads].cpu()  # noqa: E731
        qs, ks, vs, os, ds = (cut(x) for x in (q, k, v, o, do))
        ls = lse.view(B * T, H)[rows][:, heads].cpu()
        want = ref.forward(qs, ks, vs, [0, T], D ** -0.5)
        within("o", os, want[0], want[2])
        within("lse", ls, want[1], want[3])
        want, bound = ref.backward(qs, ks, vs, os, ls, ds, [0, T], D ** -0.5)
        for name, x, y, z in zip(("dq", "dk", "dv"), grads, want, bound):
            within(name, cut(x), y, z)
