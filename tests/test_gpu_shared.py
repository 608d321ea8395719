"""attn_k8v4_decode_shared against the oracle (64-bit attention over its own
cache) and, at sizes the oracle is slow for, against attn_k8v4_decode: prefixes that
end inside a tile or a page, sequences that end inside the prefix or see nothing,
group sizes around the 16 and 32 sequences of a CTA and a pair, page sizes, head
counts, bad pages, the bounded waits, and graphs."""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_kv_q8_gb300 as k8
import synth
from gpu_util import TOL, dev_tensor, rel_err

pytestmark = pytest.mark.gpu


def build(seed, n_seqs, shared, own, P, H=2, with_oracle=True):
    """A cache whose sequences share their first `shared` cells (the page the prefix ends in is each
    sequence's own copy), `own` cells behind it each: (gpu cache, oracle cache, page table)."""
    n_sh, full = -(-shared // P), shared // P
    total = shared + own
    n_pages = n_sh + n_seqs * (-(-total // P) - full) + 2
    ids = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    pt = np.empty((n_seqs, -(-total // P)), np.int32)
    pt[:, :full] = ids[:full]
    pt[:, full:] = ids[n_sh:n_sh + n_seqs * (pt.shape[1] - full)].reshape(n_seqs, -1)
    gpu = k8.PagedCache(n_pages, P, H)
    gpu.pages.random_(0, 256)                       # pages nobody fills hold anything
    gpu.pages.bitwise_and_(0x7b)                    # but no NaN scale
    ref = oracle.Cache(n_pages, P, H) if with_oracle else None
    kv = [synth.kv_values(seed, t, 0, shared, H, 3, "bf16") for t in (synth.T_K, synth.T_V)]
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    for b in range(n_seqs if shared % P else 1):    # the shared cells, and every copy of the page they end in
        lo = full * P if b else 0
        part = [t.f32[lo:].reshape(1, shared - lo, H, 256) for t in kv]
        kd, vd = (torch.from_numpy(np.ascontiguousarray(x)).bfloat16().cuda() for x in part)
        row = pt[b:b + 1]
        k8.kv_append_k8v4(gpu, torch.from_numpy(row.copy()).cuda(), pos + lo, kd, vd)
        if ref is not None:
            ref.append(row, np.array([lo]), np.ascontiguousarray(part[0]), np.ascontiguousarray(part[1]))
    if own:
        for b in range(n_seqs):
            mine = [synth.kv_values(seed + 1 + b, t, 1, own, H, 3, "bf16") for t in (synth.T_K, synth.T_V)]
            kd, vd = (dev_tensor(t, (1, own, H, 256)) for t in mine)
            row = pt[b:b + 1]
            k8.kv_append_k8v4(gpu, torch.from_numpy(row.copy()).cuda(), pos + shared, kd, vd)
            if ref is not None:
                ref.append(row, np.array([shared]), mine[0].f32.reshape(1, own, H, 256), mine[1].f32.reshape(1, own, H, 256))
    return gpu, ref, pt


def run(gpu, q, pt, lens, max_len, shared):
    lens_d = torch.from_numpy(np.asarray(lens, np.int32)).cuda()
    out = torch.full(q.shape, float("nan"), device="cuda")
    ws = k8.shared_workspace(gpu, q.shape[0], shared, max_len)
    ws.fill_(0xFF)                                  # NaN partials where nothing is written
    k8.attn_k8v4_decode_shared(gpu, q, pt, lens_d, max_len, shared, out, ws)
    return out


@pytest.mark.parametrize("n_seqs,shared,own,P,H,pair", [
    # enough sequences and cells for the pair kernel: around 16 and 32 sequences of a CTA and a pair, prefixes that end
    # inside a tile, a 16-cell group or a page, every page size class, one to eight KV heads
    (128, 1000, 5, 16, 1, True), (16, 4096, 0, 64, 2, True), (17, 5001, 33, 128, 2, True), (32, 2064, 100, 64, 2, True),
    (33, 2111, 1, 16, 3, True), (70, 1531, 30, 48, 2, True), (9, 9999, 17, 64, 2, True), (5, 27008, 40, 4096, 2, True),
    (100, 640, 700, 32, 2, True), (40, 1027, 3, 64, 8, True), (65, 2048, 0, 16, 4, True),
    # too few for it: the per-sequence decode
    (2, 64, 0, 64, 2, False), (3, 128, 5, 16, 1, False), (5, 1000, 40, 16, 2, False), (4, 64, 200, 32, 2, False),
    (9, 15, 100, 16, 2, False), (1, 3000, 9, 64, 2, False), (200, 40, 9, 64, 2, False)])
def test_shared_decode_against_oracle(n_seqs, shared, own, P, H, pair):
    seed = synth.config_seed(3) + 31 * n_seqs + shared
    gpu, ref, pt = build(seed, n_seqs, shared, own, P, H)
    assert pair == (k8.attn_k8v4_shared_workspace_bytes(gpu, n_seqs, shared, shared + own)
                    != k8.attn_k8v4_workspace_bytes(gpu, n_seqs, 1, shared + own))
    rng = np.random.default_rng(seed)
    lens = shared + rng.integers(0, own + 1, n_seqs)
    lens[0] = shared + own
    if n_seqs > 3:                                  # inside the prefix (also its first tile), nothing, just behind it
        lens[1], lens[2], lens[3] = rng.integers(1, shared), 0, min(shared + own, shared + 1)
        lens[-1] = min(3, shared)
    q = synth.q_values(seed, 7, n_seqs, H, "bf16")
    got = run(gpu, dev_tensor(q, (n_seqs, 8 * H, 256)), torch.from_numpy(pt).cuda(), lens, shared + own, shared)
    assert k8.k8v4_last_device_status() == 0
    rs, rh, rv = oracle.decode_rows(n_seqs, 8 * H, lens)
    want = ref.attention(pt, rs, rh, rv, q.f32.reshape(-1, 256))
    assert rel_err(got.cpu().numpy().reshape(-1, 256), want) <= TOL


@pytest.mark.parametrize("n_seqs,shared,own", [(32, 32768, 300), (48, 20011, 64), (128, 16384, 16)])
def test_shared_decode_against_decode_long(n_seqs, shared, own):
    """Both calls are within TOL of the exact result, so within 2 TOL of each other."""
    seed = synth.config_seed(3) + n_seqs
    gpu, _, pt = build(seed, n_seqs, shared, own, 64, with_oracle=False)
    rng = np.random.default_rng(seed)
    lens = (shared + rng.integers(0, own + 1, n_seqs)).astype(np.int32)
    lens[3], lens[5] = 0, shared // 3
    q = dev_tensor(synth.q_values(seed, 7, n_seqs, 2, "bf16"), (n_seqs, 16, 256))
    ptd = torch.from_numpy(pt).cuda()
    got = run(gpu, q, ptd, lens, shared + own, shared)
    want = torch.empty_like(got)
    ws = k8.workspace(gpu, n_seqs, 1, shared + own)
    k8.attn_k8v4_decode(gpu, q, ptd, torch.from_numpy(lens).cuda(), shared + own, want, ws)
    assert k8.k8v4_last_device_status() == 0
    assert rel_err(got.cpu().numpy(), want.cpu().numpy()) <= 2 * TOL


def test_shared_decode_moving_maxima_and_extreme_queries():
    """Scores that grow along the prefix by far more than 2^8 (every few tiles a row's reference maximum
    moves), next to zero queries and queries of 1e30 and 1e-30."""
    n_seqs, shared, P, H = 40, 2048, 64, 2
    seed = synth.config_seed(3) + 5
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((1, shared, H, 256)).astype(np.float32)
    k *= (np.linspace(0, 6, shared)[None, :, None, None] * rng.choice([0.2, 1.0], shared)[None, :, None, None]).astype(np.float32)
    v = rng.standard_normal((1, shared, H, 256)).astype(np.float32)
    q = rng.standard_normal((n_seqs, 16, 256)).astype(np.float32)
    q[3] = 0
    q[5] *= 1e-30
    q[7, 2] *= 40
    kt, vt, qt = (torch.from_numpy(x).bfloat16() for x in (k, v, q))
    pt = np.random.default_rng(1).permutation(shared // P).astype(np.int32)[None]
    gpu, ref = k8.PagedCache(shared // P, P, H), oracle.Cache(shared // P, P, H)
    k8.kv_append_k8v4(gpu, torch.from_numpy(pt).cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), kt.cuda(), vt.cuda())
    ref.append(pt, np.array([0]), kt.float().numpy(), vt.float().numpy())
    ptn = np.repeat(pt, n_seqs, 0)
    lens = np.full(n_seqs, shared)
    lens[9] = 130
    got = run(gpu, qt.cuda(), torch.from_numpy(ptn).cuda(), lens, shared, shared)
    assert k8.k8v4_last_device_status() == 0
    rs, rh, rv = oracle.decode_rows(n_seqs, 16, lens)
    want = ref.attention(ptn, rs, rh, rv, qt.float().numpy().reshape(-1, 256))
    assert rel_err(got.cpu().numpy().reshape(-1, 256), want) <= TOL


@pytest.mark.parametrize("n_seqs,shared", [(40, 24000), (100, 12345)])
def test_shared_decode_moving_maxima_long(n_seqs, shared):
    """Scores growing in jumps along a prefix that every CTA pair sweeps for tens of tiles: the reference maxima move
    inside a chain of tiles, at its end and at its beginning.  Against attn_k8v4_decode (2 TOL)."""
    P, H = 64, 2
    rng = np.random.default_rng(n_seqs)
    n_pages = -(-shared // P)
    pt = rng.permutation(n_pages).astype(np.int32)[None]
    gpu = k8.PagedCache(n_pages, P, H)
    gen = torch.Generator(device="cuda").manual_seed(n_seqs)
    k = torch.randn(1, shared, H, 256, generator=gen, device="cuda")
    v = torch.randn(1, shared, H, 256, generator=gen, device="cuda")
    k *= torch.from_numpy((np.linspace(0.1, 5, shared) * rng.choice([0.1, 0.5, 1.0], shared)).astype(np.float32)).cuda()[None, :, None, None]
    q = torch.randn(n_seqs, 16, 256, generator=gen, device="cuda").bfloat16()
    k8.kv_append_k8v4(gpu, torch.from_numpy(pt).cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), k.bfloat16(), v.bfloat16())
    ptd = torch.from_numpy(np.repeat(pt, n_seqs, 0)).cuda()
    lens = rng.integers(shared // 2, shared + 1, n_seqs).astype(np.int32)
    got = run(gpu, q, ptd, lens, shared, shared)
    want = torch.empty_like(got)
    k8.attn_k8v4_decode(gpu, q, ptd, torch.from_numpy(lens).cuda(), shared, want, k8.workspace(gpu, n_seqs, 1, shared))
    assert k8.k8v4_last_device_status() == 0
    assert rel_err(got.cpu().numpy(), want.cpu().numpy()) <= 2 * TOL


@pytest.mark.parametrize("n_seqs,shared,longest", [(40, 4096, 3001), (70, 2000, 1999), (64, 6400, 17), (33, 8192, 0)])
def test_shared_decode_nothing_behind_the_lengths_is_read(n_seqs, shared, longest):
    """Every sequence ends inside the prefix (each pair's somewhere else): pages behind hold NaN scales, and the table
    has no page there at all."""
    P, H = 16, 2
    seed = synth.config_seed(3) + 11
    n_pages = -(-shared // P)
    pt = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)[None]
    gpu, ref = k8.PagedCache(n_pages, P, H), oracle.Cache(n_pages, P, H)
    gpu.pages.fill_(0xFF)                           # NaN fp16 and fp32 scales
    if longest:
        kv = [synth.kv_values(seed, t, 0, longest, H, 3, "bf16") for t in (synth.T_K, synth.T_V)]
        kd, vd = (dev_tensor(t, (1, longest, H, 256)) for t in kv)
        k8.kv_append_k8v4(gpu, torch.from_numpy(pt).cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), kd, vd)
        ref.append(pt, np.array([0]), *(t.f32.reshape(1, longest, H, 256) for t in kv))
    pt[:, -(-longest // P):] = -1
    pt = np.repeat(pt, n_seqs, 0)
    lens = np.random.default_rng(seed).integers(0, longest + 1, n_seqs)
    lens[:32] = np.minimum(lens[:32], longest // 2)  # the first pair's sequences are the shorter ones
    lens[-1] = longest
    q = synth.q_values(seed, 7, n_seqs, H, "bf16")
    assert k8.attn_k8v4_shared_workspace_bytes(gpu, n_seqs, shared, shared) != k8.attn_k8v4_workspace_bytes(gpu, n_seqs, 1, shared)
    got = run(gpu, dev_tensor(q, (n_seqs, 16, 256)), torch.from_numpy(pt).cuda(), lens, shared, shared)
    assert k8.k8v4_last_device_status() == 0
    rs, rh, rv = oracle.decode_rows(n_seqs, 16, lens)
    want = ref.attention(np.maximum(pt, 0), rs, rh, rv, q.f32.reshape(-1, 256))
    assert rel_err(got.cpu().numpy().reshape(-1, 256), want) <= TOL


def test_shared_decode_scale_carried_by_the_queries():
    """Queries times 2^e with sm_scale times 2^-e are the same scores exactly, so the output has the same bits; a
    product of the two scales that underflows leaves all visible cells alike and hides the others."""
    n_seqs, shared = 40, 2048
    seed = synth.config_seed(3) + 12
    gpu, _, pt = build(seed, n_seqs, shared, 0, 64, with_oracle=False)
    q = dev_tensor(synth.q_values(seed, 7, n_seqs, 2, "bf16"), (n_seqs, 16, 256))
    ptd = torch.from_numpy(pt).cuda()
    lens = torch.from_numpy(np.random.default_rng(2).integers(0, shared + 1, n_seqs).astype(np.int32)).cuda()
    ws = k8.shared_workspace(gpu, n_seqs, shared, shared)
    outs = {}
    for e in (0, 90, 120, -60):
        outs[e] = torch.empty(q.shape, device="cuda")
        k8.attn_k8v4_decode_shared(gpu, q * 2.0 ** e, ptd, lens, shared, shared, outs[e], ws, sm_scale=2.0 ** (-4 - e))
        assert torch.equal(outs[e], outs[0])
    flat = torch.empty_like(outs[0])
    k8.attn_k8v4_decode_shared(gpu, q * 2.0 ** -90, ptd, lens, shared, shared, flat, ws, sm_scale=2.0 ** -60)
    zero = torch.empty_like(flat)
    k8.attn_k8v4_decode_shared(gpu, torch.zeros_like(q), ptd, lens, shared, shared, zero, ws)
    assert k8.k8v4_last_device_status() == 0
    assert rel_err(flat.cpu().numpy(), zero.cpu().numpy()) <= 2 * TOL


def test_shared_decode_bad_pages_and_lengths():
    """A page id out of range inside the prefix: its cells are skipped and recorded; a length past max_seq_len is
    clipped, one below 0 counts as 0."""
    n_seqs, shared, P = 60, 1600, 16
    seed = synth.config_seed(3) + 6
    gpu, ref, pt = build(seed, n_seqs, shared, 0, P)
    q = synth.q_values(seed, 7, n_seqs, 2, "bf16")
    qd = dev_tensor(q, (n_seqs, 16, 256))
    bad = pt.copy()
    bad[:, 2] = gpu.n_pages + 3
    bad[:, 61] = -1
    lens = np.full(n_seqs, shared)
    got = run(gpu, qd, torch.from_numpy(bad).cuda(), lens, shared, shared)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    # the same attention with those cells cut out: a table without the two pages
    keep = np.delete(pt, [2, 61], 1)
    rs, rh, rv = oracle.decode_rows(n_seqs, 16, np.full(n_seqs, shared - 2 * P))
    want = ref.attention(keep, rs, rh, rv, q.f32.reshape(-1, 256))
    assert rel_err(got.cpu().numpy().reshape(-1, 256), want) <= TOL
    lens[4], lens[6] = shared + 9, -3
    got = run(gpu, qd, torch.from_numpy(pt).cuda(), lens, shared, shared)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    rs, rh, rv = oracle.decode_rows(n_seqs, 16, np.clip(lens, 0, shared))
    want = ref.attention(pt, rs, rh, rv, q.f32.reshape(-1, 256))
    assert rel_err(got.cpu().numpy().reshape(-1, 256), want) <= TOL
    assert k8.k8v4_last_device_status() == 0


def test_shared_decode_wait_timeout_then_recovery():
    """With the wait bound below 1 us the pair kernel's waits give up at their first poll: it records K8V4_ECUDA,
    waits for its own products, frees its tensor memory and returns; a normal call afterwards is right."""
    n_seqs, shared = 33, 4096
    seed = synth.config_seed(3) + 8
    gpu, ref, pt = build(seed, n_seqs, shared, 0, 64)
    q = synth.q_values(seed, 7, n_seqs, 2, "bf16")
    qd, ptd = dev_tensor(q, (n_seqs, 16, 256)), torch.from_numpy(pt).cuda()
    lens = np.full(n_seqs, shared)
    assert k8.k8v4_last_device_status() == 0
    try:
        k8.k8v4_set_wait_limit_ns(1)
        run(gpu, qd, ptd, lens, shared, shared)
        assert k8.k8v4_last_device_status() == k8.ECUDA
    finally:
        k8.k8v4_set_wait_limit_ns(0)
    got = run(gpu, qd, ptd, lens, shared, shared)
    assert k8.k8v4_last_device_status() == 0
    rs, rh, rv = oracle.decode_rows(n_seqs, 16, lens)
    want = ref.attention(pt, rs, rh, rv, q.f32.reshape(-1, 256))
    assert rel_err(got.cpu().numpy().reshape(-1, 256), want) <= TOL


def test_shared_decode_captured_and_repeatable():
    """Captured and replayed with new queries and lengths in place; equal bits each time and on another stream."""
    n_seqs, shared, own = 24, 4000, 200
    seed = synth.config_seed(3) + 9
    gpu, _, pt = build(seed, n_seqs, shared, own, 64, with_oracle=False)
    q = dev_tensor(synth.q_values(seed, 7, n_seqs, 2, "bf16"), (n_seqs, 16, 256))
    ptd = torch.from_numpy(pt).cuda()
    lens = torch.full((n_seqs,), shared + own, dtype=torch.int32, device="cuda")
    out = torch.empty(q.shape, device="cuda")
    ws = k8.shared_workspace(gpu, n_seqs, shared, shared + own)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k8.attn_k8v4_decode_shared(gpu, q, ptd, lens, shared + own, shared, out, ws)
    side = torch.cuda.Stream()
    for step in range(3):
        lens.sub_(37)
        q.neg_()
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = torch.empty_like(out)
            k8.attn_k8v4_decode_shared(gpu, q, ptd, lens, shared + own, shared, want, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert k8.k8v4_last_device_status() == 0
