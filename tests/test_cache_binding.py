"""CPU tests of the paged cache's binding: what importing the package asks of
torch."""
import subprocess
import sys

from tests.conftest import ROOT


def test_import_without_gpu_functions_of_torch():
    """A torch built without GPU support lacks torch._C._cuda_*: the package and
    its build module import all the same, and a call says what it misses."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]:
    delattr(torch._C, name)
import gated_delta_rule_44_amd as gdr
import gated_delta_rule_44_amd.build, gated_delta_rule_44_amd.cache
x = torch.zeros(3, 2, 16, 64)
try:
    gdr.attention_decode(x, x, x, x, x)
except gdr.GdrError as e:
    print(e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr
    assert "k_cache must be a GPU tensor" in r.stdout
