"""The calls of a ragged batch's step together, as a server makes them: pages planned on the
device, queries and keys rotated by the planned positions, keys and values written through the planned slots,
differential attention over what is there, its result gated, normed and added to the residual stream.  Requests come
and go; eager, and captured once for a padded batch."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from diff_util import all_cells, check, expected, weights
from test_gpu_block_norm import check as check_norm
from test_gpu_rope import table_of

pytestmark = pytest.mark.gpu

H, HQ, P, ROT, T, DIM = 2, 16, 16, 64, 160, 16 * 256


@pytest.mark.parametrize("graph", [False, True])
def test_requests_come_and_go(graph):
    rng = np.random.default_rng(21)
    B, width, n_pages = 10, 30, 150
    rope = torch.from_numpy(table_of(width * P, ROT)).cuda()
    cache = k8.PagedCache(n_pages, P, H)
    i32, i64 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.int64, device="cuda")
    table, lens = torch.full((B, width), -1, **i32), torch.zeros(B, **i32)
    free, n_free = torch.from_numpy(rng.permutation(n_pages).astype(np.int32)).cuda(), torch.tensor([n_pages], **i32)
    new, off, granted = torch.zeros(B, **i32), torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
    pos, slots = torch.zeros(T, **i64), torch.zeros(T, **i64)
    qkv = torch.zeros(T, HQ + 2 * H, 256, dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv.split([HQ, H, H], 1)
    qr, kr = torch.zeros(T, 1, HQ, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, 1, H, 256, dtype=torch.bfloat16, device="cuda")
    heads, lam, w = weights(rng, HQ)
    out = torch.zeros(T, HQ, 256, dtype=torch.bfloat16, device="cuda")
    ws = k8.diff_workspace(cache, B, T, width * P)
    gate, x = (torch.from_numpy(rng.standard_normal((T, DIM)).astype(np.float32)).bfloat16().cuda() for _ in range(2))
    post, pre = (torch.from_numpy((1 + 0.1 * rng.standard_normal(DIM)).astype(np.float32)).cuda() for _ in range(2))
    h, normed = torch.zeros_like(x), torch.zeros_like(x)

    def step():
        k8.kv_plan_k8v4(P, free, n_free, table, lens, new, off, pos, slots, granted)
        k8.qk_norm_rope_k8v4(q[:, None], k[:, None], pos, rope, qr, kr, q_weight=w, k_weight=w)
        k8.kv_append_k8v4_slots(cache, slots, kr[:, 0], v)
        k8.attn_k8v4_diff(cache, qr[:, 0], off, table, lens, width * P, heads, out, ws)
        k8.block_norm_k8v4(out.view(T, DIM), x, h, post_weight=post, gate=gate, gate_act="sigmoid", residual_scale=0.5,
                           pre_weight=pre, normed=normed, eps=1e-5)

    run = step
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        run = g.replay

    # the same rows through the calls of one sequence: its own pages, its own positions
    plain = k8.PagedCache(B * width, P, H)
    mine = torch.arange(B * width, **i32).view(B, width)
    held = np.zeros(B, int)
    wants = [[70, 1, 0, 33, 16, 17, 5, 1, 0, 0], [1, 1, 40, 1, 1, 1, 1, 15, 64, 20], [1, -1, 1, -1, 1, 3, 1, 1, 1, 1],
             [1, 50, 1, 60, -1, 1, 1, 1, 1, -1], [5, 1, 1, 1, 1, 1, 0, 2, 1, 1]]
    for want in wants:
        want = np.array(want)
        new.copy_(torch.from_numpy(want.astype(np.int32)))
        qkv.copy_(torch.from_numpy(rng.standard_normal(qkv.shape).astype(np.float32)))
        run()
        assert k8.k8v4_last_device_status() == 0
        ends = np.concatenate([[0], np.cumsum(np.maximum(want, 0))])
        assert np.array_equal(off.cpu().numpy(), ends) and np.array_equal(granted.cpu().numpy(), np.maximum(want, 0))
        t, cells, plain_cells = table.cpu().numpy(), all_cells(cache), None
        for b in range(B):
            lo, hi = ends[b], ends[b + 1]
            if want[b] == -1:
                held[b] = 0
            if hi == lo:
                continue
            first = torch.tensor([held[b]], **i64)
            q1, k1 = (torch.empty_like(y[lo:hi, 0][None]) for y in (qr, kr))
            k8.qk_norm_rope_k8v4(q[lo:hi][None], k[lo:hi][None], first, rope, q1, k1, q_weight=w, k_weight=w)
            assert torch.equal(q1[0], qr[lo:hi, 0])
            k8.kv_append_k8v4(plain, mine[b:b + 1], first, k1, v[lo:hi][None].contiguous())
            held[b] += hi - lo
        plain_cells = all_cells(plain)
        for b in range(B):
            lo, hi = ends[b], ends[b + 1]
            c = np.arange(held[b])
            ids = torch.from_numpy(t[b][c // P].astype(np.int64) * P + c % P).cuda()
            same = torch.arange(held[b], device="cuda") + b * width * P
            assert all(torch.equal(x1[ids], x2[same]) for x1, x2 in zip(cells, plain_cells))
            if hi > lo:
                sees = held[b] - (hi - lo) + 1 + np.arange(hi - lo)
                good, bound = expected(plain_cells, qr[lo:hi, 0].double(), same, sees, lam, 0.6, w, 0.4)
                check(out[lo:hi], good, bound)
        assert np.array_equal(lens.cpu().numpy(), held)
        n = ends[-1]
        again = check_norm(out.view(T, DIM)[:n], DIM, "bf16", gate=gate[:n], act="sigmoid", residual=x[:n], alpha=0.5, post=post, pre=pre)
        assert torch.equal(again[0], h[:n]) and torch.equal(again[1], normed[:n])
