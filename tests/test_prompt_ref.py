"""CPU tests of the prompts' 64-bit reference: against a softmax written out
token by token, against automatic differentiation and against differences."""
import math

import pytest
import torch

from tests import prompt_ref as ref


def make(T, Hq, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(T, Hq, D), r(T, Hkv, D), r(T, Hkv, D), r(T, Hq, D)


@pytest.mark.parametrize("cu,window", [([0, 5], 0), ([0, 3, 3, 9], 0), ([0, 7, 8], 3), ([0, 6], 1)])
def test_forward_token_by_token(cu, window):
    q, k, v, _ = make(cu[-1] + 2, 4, 2, 8, 1)
    o, lse, _, _ = ref.forward(q, k, v, cu, 0.3, window)
    for lo, hi in zip(cu[:-1], cu[1:]):
        for i in range(hi - lo):
            js = [j for j in range(hi - lo) if j <= i and (window == 0 or i - j < window)]
            for h in range(4):
                e = [math.exp(0.3 * float(q[lo + i, h] @ k[lo + j, h // 2])) for j in js]
                want = sum(x / sum(e) * v[lo + j, h // 2] for x, j in zip(e, js))
                assert torch.allclose(o[lo + i, h], want, atol=1e-12)
                assert abs(float(lse[lo + i, h]) - math.log(sum(e))) < 1e-12
    assert torch.isnan(o[cu[-1]:]).all() and not torch.isnan(o[:cu[-1]]).any()


@pytest.mark.parametrize("cu,window", [([0, 5], 0), ([0, 3, 3, 9], 0), ([0, 9], 3)])
def test_backward_by_autograd_and_differences(cu, window):
    q, k, v, do = make(cu[-1], 4, 2, 8, 2)

    def value(q, k, v):
        total = 0
        for lo, hi in zip(cu[:-1], cu[1:]):
            for h in range(4):
                s = (0.3 * q[lo:hi, h] @ k[lo:hi, h // 2].t()).masked_fill(
                    ~ref.band(hi - lo, window), -math.inf)
                total = total + (torch.softmax(s, 1) @ v[lo:hi, h // 2] * do[lo:hi, h]).sum()
        return total

    o, lse, _, _ = ref.forward(q, k, v, cu, 0.3, window)
    grads, _ = ref.backward(q, k, v, o, lse, do, cu, 0.3, window)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    for mine, auto in zip(grads, torch.autograd.grad(value(*leaves), leaves)):
        assert torch.allclose(mine, auto, atol=1e-11)
    for n, x in enumerate((q, k, v)):
        d = torch.randn(x.shape, generator=torch.Generator().manual_seed(n), dtype=torch.float64)
        args = [q, k, v]
        up, down = list(args), list(args)
        up[n], down[n] = x + 1e-5 * d, x - 1e-5 * d
        slope = float(value(*up) - value(*down)) / 2e-5
        assert abs(slope - float((grads[n] * d).sum())) < 1e-6 * (1 + abs(slope))
