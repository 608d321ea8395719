"""kv_plan_k8v4 where the shared memory of its lists passes what a kernel has without asking, in a process of its
own: a larger call before these would have asked already."""
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

# 17 bytes a sequence, and 256 of the kernel's own: 48 KB are passed at 2,877 sequences, by the lists alone at 2,892
SCRIPT = """
import sys
sys.path[:0] = [%r, %r + "/tests"]
import numpy as np
from test_gpu_plan import batch, check
for B in (2876, 2877, 2884, 2891, 2892):
    _, _, status = check(batch(np.random.default_rng(B), B, 16, 40, 3000, most=4))
    assert status == 0, (B, status)
"""


def test_lists_about_48_kb():
    subprocess.run([sys.executable, "-c", SCRIPT % (ROOT, ROOT)], check=True, timeout=300, cwd=ROOT)
