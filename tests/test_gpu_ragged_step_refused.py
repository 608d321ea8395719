"""A step whose plan refuses sequences, for want of pages and of packed tokens: their tokens keep their rows, and with
steps made from the plan these are 0 and the others' the rows of the same batch without them."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from diff_util import all_cells, check, expected, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,T,some", [(20, 300, {3, 5}), (100, 60, {3, 4, 5, 6})])
def test_refused_sequences_are_left_empty(pages, T, some):
    rng = np.random.default_rng(pages)
    H, HQ, P, width = 2, 16, 16, 30
    want = np.array([40, 1, 7, 150 if pages < 100 else 30, 2, 33, 1], np.int32)
    held = np.array([30, 15, 16, 20, 3, 40, 14], np.int32)       # (15 + 1, 3 + 2 and 14 + 1 need no page)
    B = len(want)
    i32, i64 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.int64, device="cuda")
    have = -(-held // P)
    cache = k8.PagedCache(int(have.sum()) + pages, P, H)
    ids = rng.permutation(cache.n_pages).astype(np.int32)
    table = torch.full((B, width), -1, **i32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = torch.from_numpy(ids[at:at + have[b]])
        at += have[b]
    free = torch.full((cache.n_pages,), -1, **i32)
    n = 8 if pages < 100 else pages
    free[:n] = torch.from_numpy(ids[at:at + n])
    n_free, lens, new = torch.tensor([n], **i32), torch.from_numpy(held).cuda(), torch.from_numpy(want).cuda()
    every = torch.from_numpy(rng.standard_normal((1, cache.n_pages * P, H, 256)).astype(np.float32)).bfloat16().cuda()
    k8.kv_append_k8v4(cache, torch.arange(cache.n_pages, **i32)[None], torch.zeros(1, **i64), every, every.flip(1).contiguous())
    off, granted = torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
    pos, slots = torch.zeros(T, **i64), torch.zeros(T, **i64)
    k8.kv_plan_k8v4(P, free, n_free, table, lens, new, off, pos, slots, granted)
    assert k8.k8v4_last_device_status() == k8.ENOSPACE
    assert set(np.flatnonzero(granted.cpu().numpy() != want)) == some
    q, k, v = (torch.from_numpy(rng.standard_normal((T, x, 256)).astype(np.float32)).bfloat16().cuda() for x in (HQ, H, H))
    k8.kv_append_k8v4_slots(cache, slots, k, v)
    heads, lam, w = weights(rng, HQ)
    steps = torch.where(slots >= 0, pos + 1, 0).int()
    out = torch.full((T, HQ, 256), 77.0, dtype=torch.bfloat16, device="cuda")
    k8.attn_k8v4_diff(cache, q, off, table, lens, width * P, heads, out, k8.diff_workspace(cache, B, T, width * P), steps=steps)
    assert k8.k8v4_last_device_status() == 0
    cells, ends, t, ln = all_cells(cache), off.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy()
    for b in range(B):
        lo, hi = ends[b], ends[b + 1]
        if b in some:
            assert ln[b] == held[b] and (out[lo:hi] == 0).all()
            continue
        assert ln[b] == held[b] + want[b] and hi - lo == want[b]
        c = np.arange(ln[b])
        mine = torch.from_numpy(t[b][c // P].astype(np.int64) * P + c % P).cuda()
        good, bound = expected(cells, q[lo:hi].double(), mine, held[b] + 1 + np.arange(want[b]), lam, 0.6, w, 0.4)
        check(out[lo:hi], good, bound)
    assert (out[ends[B]:] == 77.0).all()
