"""Waits of the single queries' kernel that run out in some pairs of a CTA's piece and not in others: every warp of the
CTA leaves at the same pair, the kernel records it and returns, and the calls after it are right."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from test_gpu_diff import decode_case, run_decode

pytestmark = pytest.mark.gpu


def test_waits_that_run_out_between_pairs():
    rng = np.random.default_rng(31)
    lens = [int(x) for x in rng.integers(1, 400, 600)]
    cache, pt, q, heads, *_ = decode_case(32, lens, 2, 16)
    good = run_decode(cache, pt, q, lens, heads)
    assert k8.k8v4_last_device_status() == 0
    try:
        for limit in (1, 1000, 1500, 2000, 3000):
            k8.k8v4_set_wait_limit_ns(limit)
            for _ in range(4):
                run_decode(cache, pt, q, lens, heads)
            torch.cuda.synchronize()
            assert k8.k8v4_last_device_status() in (0, k8.ECUDA)
    finally:
        k8.k8v4_set_wait_limit_ns(0)
    assert torch.equal(run_decode(cache, pt, q, lens, heads), good)
    assert k8.k8v4_last_device_status() == 0
