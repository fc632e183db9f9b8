"""The package imports, and its host checks work, in a torch built without CUDA
(whose torch._C lacks the functions that look up device and stream)."""
from __future__ import annotations

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in dir(torch._C):
    if name.startswith("_cuda_"):
        delattr(torch._C, name)
import paged_kv_cache_14_gb300 as pa
from paged_kv_cache_14_gb300.step import SparseStep
assert pa.pa_version() > 0 and pa.pa_strerror(-1)
t = torch.zeros(2, 4, 64)
try:
    pa.pa_select_blocks(t, t, t, t, t, 4, 16, 4)
except TypeError as e:
    assert "CUDA tensor" in str(e)
else:
    raise AssertionError("took a CPU tensor")
"""


def test_import():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
