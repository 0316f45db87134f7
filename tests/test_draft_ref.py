"""CPU tests of the drafts' reference: a chain is the cache's own attention, and
hand-worked trees and tables."""
import numpy as np
import torch

from tests import cache_ref, draft_ref as ref


def test_chain_is_decode():
    rng = np.random.default_rng(1)
    r = lambda *s: torch.from_numpy(rng.standard_normal(s))  # noqa: E731
    kc, vc, q = r(5, 2, 4, 8), r(5, 2, 4, 8), r(2, 3, 4, 8)
    table = np.array([[0, 3, -1], [4, 1, 2]], np.int32)
    chain = np.array([[-1, 0, 1]] * 2)
    for lens in ([7, 12], [2, 10], [1, 0]):
        for window in (0, 1, 4):
            a = cache_ref.attend(q, kc, vc, table, lens, 0.3, window)
            b = ref.attend(q, kc, vc, table, lens, chain, 0.3, window)
            assert np.allclose(a[0], b[0], atol=1e-14)


def test_ways():
    parents = [-1, 0, 0, 2, 7, 3]
    assert ref.way(parents, 5) == [0, 2, 3, 5]
    assert ref.way(parents, 4) == [4]               # a later draft is no parent
    assert ref.way(parents, 0) == [0]


def test_accept_by_hand():
    kc = torch.arange(8.0).view(2, 1, 4, 1).repeat(1, 1, 1, 64)
    table = np.array([[1, 0]], np.int32)            # places hold 4 5 6 7 0 1 2 3
    out = ref.accept(kc, kc.clone(), table, [7], np.array([[-1, 0, -1, 1]]), [3])
    # context 3, drafts 0 1 3 from places 3 4 6 to 3 4 5
    assert out[0][:, 0, :, 0].flatten().tolist() == [0, 2, 2, 3, 4, 5, 6, 7]
    assert out[3].tolist() == [6] and out[4].tolist() == [[0, 1, 3, -1]]


def test_resize_by_hand():
    table = np.array([[3, 1, -1, -1], [0, -1, -1, -1], [2, 4, 5, -1], [-1, -1, -1, -1]], np.int32)
    t, lens, cu, free = ref.resize(table, [20, 5, 40, 0], [33, 5, 10, 64], 16, 7)
    # row 2 drops pages 4 and 5; free 4 5 6; row 0 gets 4; row 3 asks for four
    assert t.tolist() == [[3, 1, 4, -1], [0, -1, -1, -1], [2, -1, -1, -1], [-1, -1, -1, -1]]
    assert lens.tolist() == [33, 5, 10, 0] and cu.tolist() == [0, 13, 13, 13, 13] and free == 2
