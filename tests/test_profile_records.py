"""CPU check of the committed DRAM record: it names every source file of its kernel, and
counts for the sources as they are."""
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402

CSRC = os.path.join(ROOT, "quantized_paged_kv_q8_gb300", "csrc")


def _sources(name, seen=None):
    """A file of csrc and those of csrc that it includes (the public header holds declarations only)."""
    seen = set() if seen is None else seen
    if name not in seen and os.path.exists(os.path.join(CSRC, name)):
        seen.add(name)
        for inc in re.findall(r'#include "([^"/]+)"', open(os.path.join(CSRC, name)).read()):
            _sources(inc, seen)
    return seen


def test_the_decode_record_covers_its_kernels_sources():
    with open(os.path.join(ROOT, "profiles", "decode_kernel_237568_dram.txt")) as f:
        listed = re.search(r"^source: (.*)$", f.read(), re.M).group(1).split()
    assert {"k8v4_decode.cu", "k8v4_tma.cuh"} <= _sources("k8v4_decode.cu")
    assert set(listed) == _sources("k8v4_decode.cu")
    assert bench.traffic_record("decode_kernel_237568") is not None
