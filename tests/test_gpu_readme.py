"""The README's example runs, and leaves page tables that hold together."""
import os
import re

import pytest
import torch

import gated_delta_rule_44_amd as gdr
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def check_tables(table, lens, page, pages, free):
    """Each row's pages are its first ones, no page is in two places, and the others
    are free."""
    table, held = table.tolist(), []
    for row, n in zip(table, lens.tolist()):
        c = -(-n // page)
        assert all(0 <= p < pages for p in row[:c]) and all(p == -1 for p in row[c:])
        held += row[:c]
    assert len(set(held)) == len(held) and free.item() == pages - len(held)


@pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "README.md")), reason="no README.md here")
def test_example():
    text = open(os.path.join(ROOT, "README.md")).read()
    code, = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    x = {}
    exec(code, x)
    torch.cuda.synchronize()
    check_tables(x["table"], x["lens"], x["page"], x["pages"], x["free"])
    assert x["lens"].tolist() == [2048 + 3] * x["B"]
    assert x["path"].tolist() == [[0, 2, 3, -1]] * x["B"]
    for name in ("o", "o1", "o4", "oa", "dq", "dk", "dv", "ot"):
        assert bool(torch.isfinite(x[name]).all()), name
