"""One workspace, made for the largest batch, through attn_k8v4_diff calls of smaller ones."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from test_gpu_diff import check_ragged, ragged, run_ragged

pytestmark = pytest.mark.gpu


def test_one_workspace_for_every_batch():
    rng = np.random.default_rng(41)
    seqs, tokens, cells = 8, 64, 2000
    cache, pt, q, heads, lam, w, _ = ragged(rng, [8] * seqs, [cells] * seqs, 2, 64, "bf16")
    ws = k8.diff_workspace(cache, seqs, tokens, cells)
    for n in ([8] * 8, [64], [1], [60, 4], [9] * 7, [1, 2, 0, 3], [33, 1, 0, 0, 0, 0, 0, 30]):
        lens = [cells - 3 * b for b in range(len(n))]
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        T = int(off[-1])
        out = run_ragged(cache, pt[:len(n)], q[:T], off, lens, heads, ws=ws, max_len=cells)
        assert k8.k8v4_last_device_status() == 0
        check_ragged(cache, pt[:len(n)], q[:T], off, lens, lam, w, out, 64, only=5)
