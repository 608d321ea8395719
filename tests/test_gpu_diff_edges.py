"""attn_k8v4_diff_decode and attn_k8v4_diff at the ends of the lengths that they take."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from test_gpu_diff import decode_case, ragged, run_decode

pytestmark = pytest.mark.gpu


def test_no_cell_allowed():
    """max_seq_len 0: every length is clipped to none, whatever an earlier call left in the workspace."""
    lens = [100, 3000, 1, 0, 47]
    cache, pt, q, heads, *_ = decode_case(3, lens, 2, 16)
    ptd, lensd = torch.from_numpy(pt).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = k8.diff_decode_workspace(cache, len(lens), max(lens))
    out = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    k8.attn_k8v4_diff_decode(cache, q, ptd, lensd, max(lens), heads, out, ws)
    assert k8.k8v4_last_device_status() == 0 and (out[:3] != 0).any()
    k8.attn_k8v4_diff_decode(cache, q, ptd, lensd, 0, heads, out, ws)
    assert k8.k8v4_last_device_status() == k8.ERANGE and (out == 0).all()


@pytest.mark.parametrize("n", [[1, 2, 1], [1, 40, 70]])
def test_no_cell_allowed_ragged(n):
    lens = [100, 3000, 70]
    rng = np.random.default_rng(4)
    cache, pt, q, heads, _, _, off = ragged(rng, n, lens, 2, 16, "bf16")
    ptd, offd, lensd = torch.from_numpy(pt).cuda(), torch.from_numpy(off).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = k8.diff_workspace(cache, 3, q.shape[0], 3000)
    out = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    k8.attn_k8v4_diff(cache, q, offd, ptd, lensd, 3000, heads, out, ws)
    assert k8.k8v4_last_device_status() == 0
    k8.attn_k8v4_diff(cache, q, offd, ptd, lensd, 0, heads, out, ws)
    assert k8.k8v4_last_device_status() == k8.ERANGE and (out == 0).all()
