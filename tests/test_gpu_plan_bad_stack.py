"""kv_plan_k8v4 with ids on the stack that name no page: they are handed out like others and recorded, their tokens have
no slot, and the append behind it writes the other tokens alone."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from gpu_util import CANARY

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [2, 300])
def test_ids_that_name_no_page(B):
    P, n_pages, T = 16, 4 * B, 40 * B
    i32, i64 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.int64, device="cuda")
    ids = np.random.default_rng(B).permutation(n_pages).astype(np.int32)
    bad = np.arange(n_pages) % 7 == 3
    ids[bad] = np.where(np.arange(bad.sum()) % 2, -5, n_pages + 3)
    free, n_free = torch.from_numpy(ids).cuda(), torch.tensor([n_pages], **i32)
    table, lens, new = torch.full((B, 4), -1, **i32), torch.zeros(B, **i32), torch.full((B,), 40, **i32)
    off, granted, pos, slots = torch.zeros(B + 1, **i32), torch.zeros(B, **i32), torch.zeros(T, **i64), torch.zeros(T, **i64)
    k8.kv_plan_k8v4(P, free, n_free, table, lens, new, off, pos, slots, granted)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    assert (granted == 40).all() and (lens == 40).all() and n_free.item() == n_pages - 3 * B
    handed = ids[::-1][:3 * B].reshape(B, 3)
    assert np.array_equal(table[:, :3].cpu().numpy(), handed)
    c = np.arange(40)
    page = handed[:, c // P].astype(np.int64)
    want = np.where((page >= 0) & (page < n_pages), page * P + c % P, -1).ravel()
    assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(pos.cpu().numpy(), np.tile(c, B))
    cache = k8.PagedCache(n_pages, P)
    cache.pages.fill_(CANARY)
    k = torch.ones(T, 2, 256, dtype=torch.bfloat16, device="cuda")
    k8.kv_append_k8v4_slots(cache, slots, k, k)
    assert k8.k8v4_last_device_status() == 0
    codes = cache.pages.view(n_pages, -1)[:, :256 * 2 * P].reshape(n_pages * P, 512)
    written = (codes != CANARY).any(-1).cpu().numpy()
    assert np.array_equal(np.flatnonzero(written), np.sort(want[want >= 0]))
