"""Importing the package needs no GPU and no CUDA build of torch."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in dir(torch._C):
    if name.startswith("_cuda"):
        delattr(torch._C, name)              # as in a torch that was built without CUDA
import bwd_sparse_mqa_gb300 as g
assert all(hasattr(g, n) for n in g.__all__)
try:
    g.paged_plan(*[torch.zeros(1, dtype=torch.int32)] * 5, 16, 1, 1)
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("a CPU tensor was taken")
print("OK")
"""


def test_import_without_cuda_in_torch():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "OK", r.stderr[-2000:]
