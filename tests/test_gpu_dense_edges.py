"""Edges of the expert row sort, the row calls and the dense products that the sizes of the other tests
pass by."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------------------------- sort

# (experts, pairs) whose second kernel takes 48 KB of shared memory, to within 128 bytes
NEAR_48_KB = ((360, 993), (360, 8000), (383, 960), (510, 700), (511, 700), (766, 440), (767, 440), (1021, 300),
              (1022, 300), (1023, 300))
SORTS = f"""
import sys
sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, "tests")!r}]
import numpy as np, torch
from dynamic_any_precision_b200 import dpa
from test_gpu_dense import host_sort, routing
for E, P in {NEAR_48_KB}:
    idx = routing(P, 1, E, P + E, 0.1)
    got = dpa.sort_pairs(torch.from_numpy(idx).cuda(), E, dpa.new_sort_workspace(P, E))
    for a, b in zip(got, host_sort(idx, E)):
        assert np.array_equal(a.cpu().numpy(), b), (E, P)
print("sorted")
"""


def test_sorts_that_take_48_kb():
    # in a process of its own: a larger sort before them would have raised the kernels' limit
    got = subprocess.run([sys.executable, "-c", SORTS], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "sorted" in got.stdout, got.stdout + got.stderr
