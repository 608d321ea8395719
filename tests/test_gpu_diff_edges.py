"""attn_k8v4_diff_decode and attn_k8v4_diff at the ends of the lengths that they take."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from diff_util import all_cells, expected
from test_gpu_diff import decode_case, queries, ragged, run_decode

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


@pytest.mark.parametrize("way", ["one", "tile"])
def test_longest_sequence(way):
    """A table of 2^31 cells that names one page all over: the attention over that page, up to what sums of 2^31 terms
    lose.  A length past 2^31 - 256 is clipped and recorded, and a bound of 2^31 - 1 counts as a bound, not as cells."""
    rng = np.random.default_rng(6)
    P, width, most = 4096, 1 << 19, 2 ** 31 - 256
    cache = k8.PagedCache(1, P, 1)
    k, v = (torch.from_numpy((a + 0.5 * rng.standard_normal((1, P, 1, 256))).astype(np.float32)).cuda() for a in (0, 1))
    k8.kv_append_k8v4(cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"), k, v)
    T = 1 if way == "one" else 9
    q = queries(rng, T, 8, "bf16")
    heads = k8.DifferentialHeads(lambda_init=0.25)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.zeros(1, width, **i32)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")

    def run(n):
        out.fill_(77.0)
        lens = torch.tensor([n], **i32)
        if way == "one":
            k8.attn_k8v4_diff_decode(cache, q, table, lens, 2 ** 31 - 1, heads, out, k8.diff_decode_workspace(cache, 1, 2 ** 31 - 1))
        else:
            k8.attn_k8v4_diff(cache, q, torch.tensor([0, T], **i32), table, lens, 2 ** 31 - 1, heads, out,
                              k8.diff_workspace(cache, 1, T, 2 ** 31 - 1))
        return out.clone(), k8.k8v4_last_device_status()

    cells = all_cells(cache)
    for n in (P, 9 * P):                                   # (short ones under that bound, cut into ranges)
        got, status = run(n)
        want, bound = expected(cells, q.double(), torch.arange(n, device="cuda") % P, n - T + 1 + np.arange(T), None, 0.25, None, 1.0)
        assert status == 0 and ((got.double() - want).norm(dim=-1) <= bound).all()
    # a worker's sums of its 110,000 tiles are off by a unit of 2^-23 a tile at most, the sums of the weights by half
    want, bound = expected(cells, q.double(), torch.arange(P, device="cuda"), [P] * T, None, 0.25, None, 1.0)
    bound = bound + 1.5 * 110400 * 2.0 ** -23 * 1.25 * cells[1].norm(dim=-1).max().item()
    got, status = run(most)
    assert status == 0 and ((got.double() - want).norm(dim=-1) <= bound).all()
    again, status = run(2 ** 31 - 1)
    assert status == k8.ERANGE
    assert torch.equal(again, got)
