"""spec_accept_k8v4 on weights of a few subnormal units: rows, and residuals p - q,
of which only underflowed tails are left.  The tokens are compared with the
definition in exact integers (every weight is a multiple of 2^-149, u W a rational)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from test_gpu_accept import call

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -149


def drawn(weights, u):
    """The smallest index whose running sum passes u times the whole sum, without rounding."""
    units = [int(x) for x in np.asarray(weights, np.float64) * 2.0 ** 149]
    limit = Fraction(float(u)) * sum(units)
    run = 0
    for j, w in enumerate(units):
        run += w
        if run > limit:
            return j
    raise AssertionError("u is below 1")


# fp32 and bf16 (whose smallest number is 2^-133), vocabularies of one run per warp, of rows read singly and by fours
@pytest.mark.parametrize("dtype,unit", [(torch.float32, UNIT), (torch.bfloat16, 2.0 ** -133)])
@pytest.mark.parametrize("V", [1, 50, 4099, 40003, 40004])
def test_rows_of_a_few_units(dtype, unit, V):
    rng = np.random.default_rng(V)
    us = np.array([0.0, 2.0 ** -24, 0.2, 0.3, 0.45, 0.5, 0.6, 0.7, 0.9, 1 - 2.0 ** -24], np.float32)
    for counts in ({0: 1}, {V - 1: 1}, {0: 1, V // 2: 1}, {V // 3: 2, V // 2: 1, V - 1: 3},
                   {int(j): int(n) for j, n in zip(rng.integers(0, V, 9), rng.integers(1, 4, 9))}):
        p = np.zeros((len(us), 1, V), np.float32)
        for j, n in counts.items():
            p[:, 0, j] = n * unit
        got = call(p, None, np.zeros((len(us), 0), np.int32), None, np.zeros((len(us), 0), np.float32), us, dtype)[0][:, 0]
        assert got.tolist() == [drawn(p[0, 0], u) for u in us], counts
    assert k8.k8v4_last_device_status() == 0


@pytest.mark.parametrize("V", [300, 40004])
def test_residuals_of_a_few_units(V):
    """p and q differ in underflowed entries only, and the draft is refused."""
    us = np.array([0.0, 0.25, 0.4, 0.5, 0.75, 0.9, 1 - 2.0 ** -24], np.float32)
    B = len(us)
    p = np.zeros((B, 2, V), np.float32)
    p[:, :, 7] = 1.0
    q = p[:, :1].copy()
    p[:, 0, 20] = UNIT
    p[:, 0, V - 9] = 3 * UNIT
    q[:, 0, V - 9] = 2 * UNIT
    drafts = np.full((B, 1), 3, np.int32)                 # of probability 0 in both: refused
    got = call(p, q, drafts, None, np.zeros((B, 1), np.float32), us)
    assert not got[1].any()
    assert got[0][:, 0].tolist() == [drawn(np.maximum(p[0, 0] - q[0, 0], 0), u) for u in us]
    assert k8.k8v4_last_device_status() == 0


def test_large_and_small_sums_alike():
    """A row times a power of two draws the same tokens, from sums of 2^-140 up to sums of 2^120."""
    rng = np.random.default_rng(3)
    V, B = 5000, 64
    base = rng.integers(0, 1 << 10, V).astype(np.float64)
    us = rng.random(B, np.float32)
    want = [drawn(base * UNIT, u) for u in us]
    for e in (-149, -126, -60, 0, 16, 17, 18, 40, 100):
        p = np.broadcast_to((base * 2.0 ** e).astype(np.float32), (B, 1, V))
        got = call(p, None, np.zeros((B, 0), np.int32), None, np.zeros((B, 0), np.float32), us)[0][:, 0]
        assert got.tolist() == want, e
    assert k8.k8v4_last_device_status() == 0
