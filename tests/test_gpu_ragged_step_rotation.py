"""Positions of differential heads: the two maps of a head are heads of 128 lanes, and qk_norm_rope_k8v4 rotates each by
the same angles when its table holds a map's 64 cosines and sines twice, in interleaved pairs over all 256 lanes."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("turned", [64, 24])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_each_map_is_rotated_as_a_head_of_128(turned, dtype):
    """`turned` pairs of a map rotate, the others pass through (angle 0)."""
    rng = np.random.default_rng(turned)
    n, T, HQ, H = 300, 40, 16, 2
    angle = np.arange(n)[:, None] * np.concatenate([10000.0 ** (-np.arange(turned) / turned), np.zeros(64 - turned)])
    row = np.concatenate([np.cos(angle), np.cos(angle), np.sin(angle), np.sin(angle)], 1).astype(np.float32)
    table = torch.from_numpy(row).cuda()
    pos = torch.from_numpy(rng.integers(0, n, T)).cuda()
    q, k = (torch.from_numpy(rng.standard_normal((T, 1, x, 256)).astype(np.float32)).to(dtype).cuda() for x in (HQ, H))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    k8.qk_norm_rope_k8v4(q, k, pos, table, qo, ko, interleaved=True)
    assert k8.k8v4_last_device_status() == 0
    c, s = (x.double()[pos][:, None, None, None] for x in (table[:, :64], table[:, 128:192]))
    half = torch.finfo(dtype).eps / 2 + torch.finfo(torch.float32).eps
    for x, y in ((q, qo), (k, ko)):
        a, b = x.double().view(T, 1, -1, 2, 64, 2).unbind(-1)               # [.., map, pair], each its two lanes
        want = torch.stack([a * c - b * s, b * c + a * s], -1)
        got = y.double().view(want.shape)
        assert ((got - want).abs() <= half * want.abs() + 1e-30).all()
