"""The calls of a serving step together, as an engine makes them: queries and keys
normed and rotated, keys and values appended on the way, attention over the shared
prefix and each sequence's own cells, a speculative window verified and its drafts
accepted, positions moved on by what was kept -- every attention result against the
oracle fed with 64-bit rotations, the cache's bytes against the oracle's."""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_kv_q8_gb300 as k8
from gpu_util import TOL, rel_err
from test_gpu_accept import plain as accept_plain
from test_gpu_rope import rotate64, table_of

pytestmark = pytest.mark.gpu

H, HQ, P, ROT = 2, 16, 64, 64


def rows_of(rng, *shape):
    """bf16 rows as the device has them and as float64."""
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16()
    return x.cuda(), x.double().numpy()


def bf16(x64):
    return torch.from_numpy(x64.astype(np.float32)).bfloat16().float().numpy()


@pytest.mark.parametrize("graph", [False, True])
def test_shared_prompt_then_decode_and_speculation(graph):
    rng = np.random.default_rng(31)
    n, prompt, V, n_draft = 40, 2000, 500, 3
    steps, pages_each = 3, 2
    table = table_of(prompt + 100, ROT)
    td = torch.from_numpy(table).cuda()
    # one prompt for all: its pages, the last of them copied per sequence (2,000 cells end inside a page)
    full = prompt // P
    n_pages = full + n * pages_each + 3
    ids = rng.permutation(n_pages).astype(np.int32)
    pt = np.empty((n, full + pages_each), np.int32)
    pt[:, :full] = ids[:full]
    pt[:, full:] = ids[full:full + n * pages_each].reshape(n, -1)
    cache, ref = k8.PagedCache(n_pages, P, H), oracle.Cache(n_pages, P, H)
    ptd = torch.from_numpy(pt).cuda()
    k, k64 = rows_of(rng, 1, prompt, H, 256)
    v, v64 = rows_of(rng, 1, prompt, H, 256)
    kr = bf16(rotate64(k64, table[:prompt].astype(np.float64)[None, :, None], False)[0])
    for b in range(n):
        lo = full * P if b else 0
        k8.kv_append_k8v4_rope(cache, ptd[b:b + 1].contiguous(), torch.tensor([lo], device="cuda"), k[:, lo:], v[:, lo:], td)
        ref.append(pt[b:b + 1], np.array([lo]), np.ascontiguousarray(kr[:, lo:]), np.ascontiguousarray(v64[:, lo:].astype(np.float32)))
    assert k8.k8v4_last_device_status() == 0
    assert np.array_equal(cache.pages.cpu().numpy(), ref.buf)

    # ---- decode steps out of a packed projection; the sequences' lengths are the program's device state
    lens = torch.full((n,), prompt, dtype=torch.int32, device="cuda")
    pos = torch.full((n,), prompt, dtype=torch.int64, device="cuda")
    qkv = torch.empty(n, 1, HQ + 2 * H, 256, dtype=torch.bfloat16, device="cuda")
    q, kn, vn = qkv.split([HQ, H, H], 2)
    w = torch.linspace(0.5, 1.5, 256, device="cuda")
    qr, out = torch.empty(n, 1, HQ, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(n, HQ, 256, device="cuda")
    max_len = prompt + 60
    ws = k8.shared_workspace(cache, n, prompt, max_len)

    def step():
        k8.qk_norm_rope_k8v4(q, None, pos, td, qr, None, q_weight=w, eps=1e-6)
        k8.kv_append_k8v4_rope(cache, ptd, pos, kn, vn, td, k_weight=w, eps=1e-6)
        lens.add_(1)
        k8.attn_k8v4_decode_shared(cache, qr.view(n, HQ, 256), ptd, lens, max_len, prompt, out, ws)
        pos.add_(1)

    run = step
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        lens.fill_(prompt)
        pos.fill_(prompt)
        run = g.replay
    for t in range(steps):
        new, new64 = rows_of(rng, n, 1, HQ + 2 * H, 256)
        qkv.copy_(new)
        run()
        assert k8.k8v4_last_device_status() == 0
        # the oracle takes what the library's norm gave (its rounding is tested with the call itself), rotated by it
        kd = torch.empty(n, 1, H, 256, dtype=torch.bfloat16, device="cuda")
        k8.qk_norm_rope_k8v4(kn, None, pos - 1, td, kd, None, q_weight=w, eps=1e-6)
        ref.append(pt, np.full(n, prompt + t), kd.float().cpu().numpy(), np.ascontiguousarray(new64[:, :, HQ + H:].astype(np.float32)))
        assert np.array_equal(cache.pages.cpu().numpy(), ref.buf)
        ln = np.full(n, prompt + t + 1)
        rs, rh, rv = oracle.decode_rows(n, HQ, ln)
        want = ref.attention(pt, rs, rh, rv, qr.float().cpu().numpy().reshape(-1, 256))
        assert rel_err(out.cpu().numpy().reshape(-1, 256), want) <= TOL

    # ---- a window of drafts: append them all, verify, accept, keep what was accepted
    new, new64 = rows_of(rng, n, n_draft + 1, HQ + 2 * H, 256)
    q2, k2, v2 = new.split([HQ, H, H], 2)
    qv = torch.empty(n, n_draft + 1, HQ, 256, dtype=torch.bfloat16, device="cuda")
    k8.qk_norm_rope_k8v4(q2, None, pos, td, qv, None)
    k8.kv_append_k8v4_rope(cache, ptd, pos, k2, v2, td)
    base = prompt + steps
    st = torch.arange(base + 1, base + n_draft + 2, dtype=torch.int32, device="cuda").expand(n, -1).contiguous()
    vout = torch.empty(n, n_draft + 1, HQ, 256, device="cuda")
    k8.attn_k8v4_verify(cache, qv, ptd, st, max_len, vout, k8.workspace(cache, n, n_draft + 1, max_len))
    row = table[base:base + n_draft + 1].astype(np.float64)[None, :, None]
    ref.append(pt, np.full(n, base), bf16(rotate64(new64[:, :, HQ:HQ + H], row, False)[0]),
               np.ascontiguousarray(new64[:, :, HQ + H:].astype(np.float32)))
    rs, rh, rv = oracle.multi_query_rows(st.cpu().numpy(), HQ)
    qref = bf16(rotate64(new64[:, :, :HQ], row, False)[0])
    want = ref.attention(pt, rs, rh, rv, qref.reshape(-1, 256))
    assert rel_err(vout.cpu().numpy().reshape(-1, 256), want) <= TOL
    # a head over the attention's output gives the target's probabilities, a rough copy of it the drafts'
    head = torch.from_numpy(rng.standard_normal((HQ * 256, V)).astype(np.float32)).cuda() * 0.05
    p = torch.softmax(vout.view(n, n_draft + 1, -1) @ head, -1)
    qd = torch.softmax((vout[:, :n_draft].reshape(n, n_draft, -1) @ head) * 0.8, -1)
    drafts = qd.argmax(-1).int()
    u, us = torch.rand(n, n_draft, device="cuda"), torch.rand(n, device="cuda")
    tokens = torch.empty(n, n_draft + 1, dtype=torch.int32, device="cuda")
    kept = torch.empty(n, dtype=torch.int32, device="cuda")
    k8.spec_accept_k8v4(p, qd, drafts, u, us, tokens, kept)
    lens.add_(kept + 1)                          # no host round trip: the next step's lengths
    want = accept_plain(p.double().cpu().numpy(), qd.double().cpu().numpy(), drafts.cpu().numpy(), np.full(n, n_draft),
                        u.cpu().numpy(), us.cpu().numpy())
    assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(kept.cpu().numpy(), want[1])
    assert np.array_equal(lens.cpu().numpy(), prompt + steps + want[1] + 1)
    assert k8.k8v4_last_device_status() == 0
