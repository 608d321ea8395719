"""kv_plan_k8v4 at the ends of its ranges: lengths up to what int32 holds, long rows given back in whole and
in part, batches whose lists are longer than the cluster's threads."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from test_gpu_plan import batch, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length,new,granted", [(2 ** 31 - 2, 1, 1), (2 ** 31 - 2, 2, 0), (2 ** 31 - 1, 0, 0), (2 ** 31 - 1, 1, 0),
                                                (2 ** 31 - 4097, 4096, 4096)])
def test_longest_sequence(length, new, granted):
    """A table of 2^31 cells: new_lens holds no more than 2^31 - 1."""
    P, width = 4096, 2 ** 19
    i32 = dict(dtype=torch.int32, device="cuda")
    have = -(-length // P)
    n_pages = 2 ** 20
    table = torch.full((1, width), -3, **i32)
    table[0, :have] = torch.arange(have, **i32) + 7
    free = torch.full((n_pages,), -1, **i32)
    free[:2] = torch.tensor([5, 6], **i32)
    lens, want = torch.tensor([length], **i32), torch.tensor([new], **i32)
    n_free, off, ok = torch.tensor([2], **i32), torch.empty(2, **i32), torch.empty(1, **i32)
    T = max(new, 1)
    pos, slots = (torch.full((T,), -9, dtype=torch.int64, device="cuda") for _ in range(2))
    k8.kv_plan_k8v4(P, free, n_free, table, lens, want, off, pos, slots, ok)
    status = k8.k8v4_last_device_status()
    fits = length + new <= 2 ** 31 - 1
    assert (status == 0) == fits and ok.item() == (granted if fits else 0)
    assert lens.item() == (length + new if fits else length)
    need = (-(-(length + new) // P) - have) if fits else 0
    assert n_free.item() == 2 - need
    if fits and new:
        c = length + np.arange(new)
        row = table[0].cpu().numpy().astype(np.int64)
        assert (pos.cpu().numpy() == c).all() and (slots.cpu().numpy() == row[c // P] * P + c % P).all()
        assert need == 0 or table[0, have].item() == 6
    else:
        assert (slots == -1).all() and (pos == 0).all()


@pytest.mark.parametrize("B,longest,extra,most,done", [(40, 9000, 10, 400, 0.5), (9, 16000, 0, 900, 0.7), (700, 3000, 2000, 60, 0.4),
                                                       (2, 60000, 0, 3, 1.0)])
def test_long_rows_given_back(B, longest, extra, most, done):
    rng = np.random.default_rng(B)
    s = batch(rng, B, 16, longest, extra, done=done, most=most, borrow=B == 40)
    check(s)
    check(s, in_place=True)


def test_one_bad_entry_in_a_long_row():
    rng = np.random.default_rng(3)
    s = batch(rng, 30, 16, 8000, 5, done=0.5, most=100)
    rows = np.flatnonzero((s["new"] == -1) & (s["lens"] > 4000))
    s["table"][rows[0], 200] = s["n_pages"]
    s["table"][rows[1], -(-int(s["lens"][rows[1]]) // 16) - 1] = -1
    _, _, status = check(s)
    assert status == k8.ERANGE


@pytest.mark.parametrize("B,most", [(8192, 12), (3, 15000), (1, 40000)])
def test_long_lists(B, most):
    """More tokens than the cluster's threads take in one round, with and without a sequence to each."""
    rng = np.random.default_rng(most)
    s = batch(rng, B, 48, 200, 30000, prompts=1.0, done=0.1 if B > 3 else 0.0, most=most)
    check(s)
