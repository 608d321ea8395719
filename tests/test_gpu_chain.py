"""The library's calls one behind the other on a stream, nothing between them: each
starts while the one before it drains, and reads what that one wrote.  Equal, bit for
bit, to the same calls with a synchronisation behind each."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from gpu_util import TOL, rel_err
from test_gpu_rope import table_of

pytestmark = pytest.mark.gpu

H, HQ, P = 2, 16, 64


@pytest.mark.parametrize("n_seqs,shared", [(40, 2000), (70, 700), (5, 27008), (3, 300)])
def test_steps_back_to_back(n_seqs, shared):
    """Serving steps of a batch on a shared prefix: queries rotated, the step's cells appended, decode with the prefix
    shared and without, a verify window, two acceptances, cells read back.  Every step's rows are new, so
    an attention that read a cell, a query or a partial row too early would differ.  (The last two sizes: few sequences
    on a long prefix, and the per-sequence route.)"""
    rounds, drafts, V = 12, 3, 2000
    own = rounds + drafts + 1
    full = shared // P
    each = -(-(shared + own) // P) - full
    n_pages = full + n_seqs * each
    gen = torch.Generator(device="cuda").manual_seed(n_seqs)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").int()
    pt = torch.empty(n_seqs, full + each, dtype=torch.int32, device="cuda")
    pt[:, :full] = ids[:full]
    pt[:, full:] = ids[full:].view(n_seqs, each)
    table = torch.from_numpy(table_of(shared + own, 128)).cuda()
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    q, k, v = (normal(rounds, n_seqs, 1, n, 256) for n in (HQ, H, H))
    kd, vd, qd = (normal(rounds, n_seqs, drafts + 1, n, 256) for n in (H, H, HQ))
    prompt = normal(2, 1, shared, H, 256)
    rest = prompt[:, :, full * P:].expand(2, n_seqs, -1, H, 256).contiguous()   # each sequence's copy of the last page
    w = torch.linspace(0.5, 1.5, 256, device="cuda")
    probs = torch.softmax(3 * torch.randn(rounds, n_seqs, drafts + 1, V, generator=gen, device="cuda"), -1)
    tokens = torch.randint(0, V, (rounds, n_seqs, drafts), generator=gen, device="cuda").int()
    u, us = torch.rand(rounds, n_seqs, drafts, generator=gen, device="cuda"), torch.rand(rounds, n_seqs, generator=gen, device="cuda")
    pos = [torch.full((n_seqs,), shared + i, dtype=torch.int64, device="cuda") for i in range(rounds)]
    lens = [(p + 1).int() for p in pos]
    steps = [(p[:, None] + 1 + torch.arange(drafts + 1, device="cuda")).int() for p in pos]
    zero, tail = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.full((n_seqs,), full * P, dtype=torch.int64, device="cuda")
    one = pt[:1].contiguous()
    max_len = shared + own

    def chain(pause):
        cache = k8.PagedCache(n_pages, P, H)
        cache.pages.zero_()
        out = dict(shared=torch.empty(rounds, n_seqs, HQ, 256, device="cuda"), alone=torch.empty(rounds, n_seqs, HQ, 256, device="cuda"),
                   again=torch.empty(rounds, n_seqs, HQ, 256, device="cuda"),
                   window=torch.empty(rounds, n_seqs, drafts + 1, HQ, 256, device="cuda"),
                   back=torch.empty(rounds, 2, own, H, 256, device="cuda"),
                   tokens=torch.empty(rounds, n_seqs, drafts + 1, dtype=torch.int32, device="cuda"),
                   kept=torch.empty(rounds, n_seqs, dtype=torch.int32, device="cuda"))
        qr, qv = torch.zeros(n_seqs, 1, HQ, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(n_seqs, drafts + 1, HQ, 256, dtype=torch.bfloat16, device="cuda")
        ws_shared = k8.shared_workspace(cache, n_seqs, shared, max_len).zero_()
        ws = k8.workspace(cache, n_seqs, 1, max_len).zero_()
        ws_v = k8.workspace(cache, n_seqs, drafts + 1, max_len).zero_()
        torch.cuda.synchronize()
        k8.kv_append_k8v4_rope(cache, one, zero, prompt[0], prompt[1], table, k_weight=w)
        if shared % P:
            k8.kv_append_k8v4_rope(cache, pt, tail, rest[0], rest[1], table, k_weight=w)
        for i in range(rounds):
            for call in (lambda: k8.qk_norm_rope_k8v4(q[i], None, pos[i], table, qr, None, q_weight=w),
                         lambda: k8.kv_append_k8v4_rope(cache, pt, pos[i], k[i], v[i], table, k_weight=w),
                         lambda: k8.attn_k8v4_decode_shared(cache, qr.view(n_seqs, HQ, 256), pt, lens[i], max_len, shared, out["shared"][i], ws_shared),
                         lambda: k8.kv_dequant_k8v4(cache, pt[n_seqs - 1], shared, own, out["back"][i, 0], out["back"][i, 1]),
                         lambda: k8.attn_k8v4_decode(cache, qr.view(n_seqs, HQ, 256), pt, lens[i], max_len, out["alone"][i], ws),
                         lambda: k8.qk_norm_rope_k8v4(qd[i], None, pos[i], table, qv, None),
                         lambda: k8.kv_append_k8v4(cache, pt, pos[i], kd[i], vd[i]),
                         lambda: k8.attn_k8v4_decode_shared(cache, qr.view(n_seqs, HQ, 256), pt, lens[i], max_len, shared, out["again"][i], ws_shared),
                         lambda: k8.attn_k8v4_verify(cache, qv, pt, steps[i], max_len, out["window"][i], ws_v),
                         lambda: k8.spec_accept_k8v4(probs[i], None, tokens[i], u[i], us[i], out["tokens"][i], out["kept"][i])):
                call()
                if pause:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return out, cache.pages

    got, want = chain(False), chain(True)
    assert k8.k8v4_last_device_status() == 0
    for name in want[0]:
        assert torch.equal(got[0][name], want[0][name]), name
    assert torch.equal(got[1], want[1])
    assert all(bool(torch.isfinite(x).all()) for x in want[0].values())


@pytest.mark.parametrize("n_seqs,shared,heads", [(128, 640, 2), (40, 1984, 2), (70, 1090, 8), (33, 4160, 1)])
def test_short_sweeps_back_to_back(n_seqs, shared, heads):
    """CTA pairs that sweep one to a few tiles, hundreds of such grids in a row: a pair's shared memory passes to the
    next pair at once, and no completion of the first may reach it.  Every call gives the bits of the first."""
    gen = torch.Generator(device="cuda").manual_seed(shared)
    n_pages = -(-shared // P)
    cache = k8.PagedCache(n_pages, P, heads)
    pt = torch.randperm(n_pages, generator=gen, device="cuda").int()[None]
    k, v = (torch.randn(1, shared, heads, 256, generator=gen, device="cuda").bfloat16() for _ in range(2))
    k8.kv_append_k8v4(cache, pt, torch.zeros(1, dtype=torch.int64, device="cuda"), k, v)
    ptd = pt.expand(n_seqs, -1).contiguous()
    q = torch.randn(n_seqs, 8 * heads, 256, generator=gen, device="cuda").bfloat16()
    lens = torch.randint(0, shared + 1, (n_seqs,), generator=gen, device="cuda").int()
    assert k8.attn_k8v4_shared_workspace_bytes(cache, n_seqs, shared, shared) != k8.attn_k8v4_workspace_bytes(cache, n_seqs, 1, shared)
    ws = k8.shared_workspace(cache, n_seqs, shared, shared)
    outs = torch.full((200, n_seqs, 8 * heads, 256), float("nan"), device="cuda")
    torch.cuda.synchronize()
    for o in outs:
        k8.attn_k8v4_decode_shared(cache, q, ptd, lens, shared, shared, o, ws)
    torch.cuda.synchronize()
    assert k8.k8v4_last_device_status() == 0
    want = torch.empty_like(outs[0])
    k8.attn_k8v4_decode(cache, q, ptd, lens, shared, want, k8.workspace(cache, n_seqs, 1, shared))
    assert rel_err(outs[0].cpu().numpy(), want.cpu().numpy()) <= 2 * TOL     # each is within TOL of the exact result
    assert bool((outs == outs[:1]).all())
