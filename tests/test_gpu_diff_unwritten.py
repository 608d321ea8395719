"""attn_k8v4_diff_decode and attn_k8v4_diff on pages whose unseen cells hold NaN scales, and on batches of thousands
of sequences."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from diff_util import all_cells, check, expected, weights
from test_gpu_diff import cells_of, queries, tables

pytestmark = pytest.mark.gpu


def written_only(rng, lens, H, P):
    """A cache of 0xff bytes (NaN in either type of scale) with the sequences' cells appended."""
    pages = sum(-(-int(n) // P) for n in lens) + 2
    cache = k8.PagedCache(pages, P, H)
    cache.pages.fill_(0xff)
    pt = tables(rng, lens, pages, P)
    for b, n in enumerate(lens):
        if n:
            k, v = (torch.from_numpy(rng.standard_normal((1, n, H, 256)).astype(np.float32)).cuda() for _ in range(2))
            k8.kv_append_k8v4(cache, torch.from_numpy(pt[b:b + 1]).cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), k, v)
    assert k8.k8v4_last_device_status() == 0
    return cache, pt


@pytest.mark.parametrize("lens,H,P", [([1, 17, 31, 1000, 0, 129], 2, 64), ([5, 255, 8190], 2, 16), ([33, 100], 8, 128)])
def test_unwritten_cells(lens, H, P):
    rng = np.random.default_rng(P)
    cache, pt = written_only(rng, lens, H, P)
    HQ = 8 * H
    heads, lam, w = weights(rng, HQ)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    cells = all_cells(cache)
    q = queries(rng, len(lens), HQ, "bf16")
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    k8.attn_k8v4_diff_decode(cache, q, torch.from_numpy(pt).cuda(), dev(lens), max(lens), heads, out,
                             k8.diff_decode_workspace(cache, len(lens), max(lens)))
    for b, n in enumerate(lens):
        want, bound = expected(cells, q[b:b + 1].double(), cells_of(pt[b], n, P), [n], lam, 0.6, w, 0.4)
        check(out[b:b + 1], want, bound)
    # the same cells seen by single tokens, by drafts and by a prompt of each sequence
    for n_new in (1, 3, 40):
        n = [min(n_new, x) for x in lens]
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        q = queries(rng, int(off[-1]), HQ, "bf16")
        out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        k8.attn_k8v4_diff(cache, q, torch.from_numpy(off).cuda(), torch.from_numpy(pt).cuda(), dev(lens), max(lens), heads, out,
                          k8.diff_workspace(cache, len(lens), int(off[-1]), max(lens)))
        for b, x in enumerate(lens):
            if n[b]:
                lo, hi = int(off[b]), int(off[b + 1])
                want, bound = expected(cells, q[lo:hi].double(), cells_of(pt[b], x, P), x - n[b] + 1 + np.arange(n[b]), lam, 0.6,
                                       w, 0.4)
                check(out[lo:hi], want, bound)
    assert k8.k8v4_last_device_status() == 0


@pytest.mark.parametrize("B,n_new", [(5000, 1), (4200, 9), (1, 3)])
def test_thousands_of_sequences(B, n_new):
    """More sequences and token tiles than the schedule keeps in shared memory; every sequence reads the same few pages,
    so that a few rows stand for all."""
    rng = np.random.default_rng(B)
    H, P, most = 1, 16, 40
    cache, pt = written_only(rng, [48], H, P)
    lens = rng.integers(0, most + 1, B).astype(np.int32)
    lens[[0, -1]] = most
    n = np.minimum(lens, n_new)
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    heads, lam, w = weights(rng, 8)
    T = int(off[-1])
    q = queries(rng, T, 8, "bf16")
    out = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    table = torch.from_numpy(pt[:1, :3]).cuda().expand(B, 3).contiguous()
    k8.attn_k8v4_diff(cache, q, torch.from_numpy(off).cuda(), table, torch.from_numpy(lens).cuda(), most, heads, out,
                      k8.diff_workspace(cache, B, T, most))
    assert k8.k8v4_last_device_status() == 0
    cells = all_cells(cache)
    for b in {0, B - 1, *(int(x) for x in rng.integers(0, B, 30))}:
        lo, hi = int(off[b]), int(off[b + 1])
        if hi > lo:
            want, bound = expected(cells, q[lo:hi].double(), cells_of(pt[0], int(lens[b]), P), lens[b] - n[b] + 1 + np.arange(n[b]),
                                   lam, 0.6, w, 0.4)
            check(out[lo:hi], want, bound)
    assert not (out == 77.0).all(-1).any()
