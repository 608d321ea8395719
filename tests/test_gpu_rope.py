"""qk_norm_rope_k8v4 and kv_append_k8v4_rope against plain 64-bit implementations:
pairings, partial rotation, strided tokens, norms, far positions, odd sizes, the
positions and pages that are refused, and the equality of the rotating append
with the rotation followed by the plain append (bytes)."""
import ctypes
import functools

import numpy as np
import pytest
import torch

import oracle
import quantized_paged_kv_q8_gb300 as k8
from gpu_util import CANARY

pytestmark = pytest.mark.gpu

F32_HALF = torch.finfo(torch.float32).eps / 2        # 2^-24: one rounding to fp32
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2      # 2^-8


@functools.lru_cache(maxsize=4)
def table_of(n_pos, rot, base=1e6):
    j = np.arange(rot // 2, dtype=np.float64)
    a = np.arange(n_pos, dtype=np.float64)[:, None] * base ** (-2.0 * j / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rotate64(x, row, inter):
    """x float64 [..., 256], row float64 [..., rot] -> rotated, and |x1| + |x2| of each element's pair."""
    half = row.shape[-1] // 2
    c, s = row[..., :half], row[..., half:]
    y, size = x.copy(), np.abs(x)
    i1 = np.arange(0, 2 * half, 2) if inter else np.arange(half)
    i2 = i1 + 1 if inter else i1 + half
    a, b = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = a * c - b * s, b * c + a * s
    size[..., i1] = size[..., i2] = np.abs(a) + np.abs(b)
    return y, size


def norm64(x, w, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def case(seed, n_seqs, n_tok, heads, dtype, packed):
    """Per entry of `heads`: a device tensor [n_seqs, n_tok, heads, 256] and its float64 values."""
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.from_numpy(rng.standard_normal((n_seqs, n_tok, sum(heads), 256)).astype(np.float32)).to(dt).cuda()
    parts = x.split(heads, 2) if packed else [p.contiguous() for p in x.split(heads, 2)]
    return list(parts), [p.double().cpu().numpy() for p in parts]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n_seqs,n_tok,hq,hk,rot,packed,norm", [
    (1, 1, 16, 2, 64, True, True), (1, 1, 16, 2, 256, False, False), (3, 5, 16, 2, 48, True, False),
    (2, 7, 8, 1, 16, False, True), (1, 301, 16, 2, 240, True, True), (5, 67, 13, 3, 128, True, False),
    (1, 9, 16, 0, 256, False, True), (2, 400, 5, 7, 256, True, True)])
def test_norm_rope_against_64_bits(dtype, inter, n_seqs, n_tok, hq, hk, rot, packed, norm):
    parts, ref = case(7 + rot + n_tok, n_seqs, n_tok, [hq, hk], dtype, packed)
    pos = np.array([[199990, 3, 70000, 0, 123456][b] for b in range(n_seqs)], np.int64)
    table = table_of(200400, rot)
    rng = np.random.default_rng(5)
    w = [(1 + 0.3 * rng.standard_normal(256)).astype(np.float32) for _ in range(2)]
    outs = [torch.empty(p.shape, dtype=p.dtype, device="cuda") for p in parts]
    wd = [torch.from_numpy(a).cuda() if norm else None for a in w]
    k8.qk_norm_rope_k8v4(parts[0], parts[1] if hk else None, torch.from_numpy(pos).cuda(),
                         torch.from_numpy(table).cuda(), outs[0], outs[1] if hk else None, q_weight=wd[0],
                         k_weight=wd[1] if hk else None, eps=1e-5, interleaved=inter)
    assert k8.k8v4_last_device_status() == 0
    rows = table[pos[:, None] + np.arange(n_tok)].astype(np.float64)[:, :, None]
    for out, x, wi in zip(outs[:2 if hk else 1], ref, w):
        y, size = rotate64(norm64(x, wi.astype(np.float64), 1e-5) if norm else x, rows, inter)
        # the norm in fp32: the squares' sum 14 roundings (halved by the root), rsqrtf 2 units, three products,
        # below 2^-20 of an element, and so of the pair; then one rounding to fp32 and one to the type.  Without
        # a norm the exact value is rounded once to fp32 (to 2^-44 of the pair)
        tol = size * (2.0 ** -20 if norm else 2.0 ** -44) + np.abs(y) * F32_HALF * 1.001
        if dtype == "bf16":
            tol = tol + (np.abs(y) + tol) * BF16_HALF
        assert np.all(np.abs(out.double().cpu().numpy() - y) <= tol)


def test_norm_rope_in_place_and_zero_rows():
    parts, ref = case(1, 2, 3, [16, 2], "bf16", False)
    parts[1].zero_()
    pos = torch.tensor([5, 40], dtype=torch.int64, device="cuda")
    table = torch.from_numpy(table_of(64, 128)).cuda()
    w = torch.ones(256, device="cuda")
    want = [torch.empty_like(p) for p in parts]
    k8.qk_norm_rope_k8v4(*parts, pos, table, *want, q_weight=w, k_weight=w)
    k8.qk_norm_rope_k8v4(*parts, pos, table, *parts, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(parts[0], want[0]) and torch.equal(parts[1], want[1])
    assert not want[1].any() and want[0].isfinite().all()


def test_norm_rope_refuses_overlapping_in_place():
    parts, _ = case(1, 1, 3, [16, 2], "bf16", True)
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    table = torch.from_numpy(table_of(64, 128)).cuda()
    r = ctypes.byref(k8.k8v4_rope(table.data_ptr(), 64, 128, 0))
    rc = k8.lib().qk_norm_rope_k8v4(k8._ptr(parts[0]), 18 * 256, 16, None, 0, 0, k8.BF16, None, None, 0.0, k8._ptr(pos),
                                    1, 3, r, k8._ptr(parts[0]), None, k8._stream(None))
    assert rc == k8.EINVAL


@pytest.mark.parametrize("start", [-2, 61])
def test_norm_rope_positions_outside_the_table(start):
    """Tokens at positions -2, -1 (or 64, 65, ...) have no table row: recorded, their output rows untouched."""
    parts, ref = case(3, 1, 6, [16, 2], "f32", False)
    table = table_of(64, 64)
    outs = [torch.full_like(p, 7.0) for p in parts]
    k8.qk_norm_rope_k8v4(*parts, torch.tensor([start], dtype=torch.int64, device="cuda"), torch.from_numpy(table).cuda(), *outs)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    assert k8.k8v4_last_device_status() == 0
    for out, x in zip(outs, ref):
        got = out.double().cpu().numpy()
        for t in range(6):
            if 0 <= start + t < 64:
                y, size = rotate64(x[0, t], table[start + t].astype(np.float64)[None], False)
                assert np.all(np.abs(got[0, t] - y) <= size * 2.0 ** -44 + np.abs(y) * F32_HALF * 1.001)
            else:
                assert np.all(got[0, t] == 7.0)


def _append_inputs(seed, n_seqs, n_tok, dtype, packed, P, pos, H=2):
    parts, ref = case(seed, n_seqs, n_tok, [16, H, H] if packed else [H, H], dtype, packed)
    k, v = parts[-2], parts[-1]
    need = -(-(max(pos) + n_tok) // P)
    perm = np.random.default_rng(seed + 1).permutation(n_seqs * need + 3).astype(np.int32)
    pt = perm[:n_seqs * need].reshape(n_seqs, need)
    return k, v, ref[-2], ref[-1], pt, n_seqs * need + 3


@pytest.mark.parametrize("fmt", [k8.FORMAT_K8V4, k8.FORMAT_INT8, k8.FORMAT_Q4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_seqs,n_tok,rot,inter,packed,P", [
    (1, 1, 64, False, True, 16), (7, 1, 256, True, False, 64), (3, 5, 48, False, True, 48),
    (1, 1501, 256, False, True, 64), (2, 777, 80, True, True, 16)])
def test_append_rope_bytes_against_oracle(fmt, dtype, n_seqs, n_tok, rot, inter, packed, P):
    """K rotated in 64 bits, rounded to fp32 and to its type, then the oracle's append:
    every byte of every page, the untouched ones among them."""
    pos = [(37 * b + 5) % 90 for b in range(n_seqs)]
    k, v, k64, v64, pt, n_pages = _append_inputs(11 + n_tok, n_seqs, n_tok, dtype, packed, P, pos)
    table = table_of(max(pos) + n_tok, rot)
    gpu = k8.PagedCache(n_pages, P, 2, fmt)
    gpu.pages.fill_(CANARY)
    ref = oracle.Cache(n_pages, P, 2, fmt, fill=CANARY)
    posd = torch.tensor(pos, dtype=torch.int64, device="cuda")
    k8.kv_append_k8v4_rope(gpu, torch.from_numpy(pt).cuda(), posd, k, v, torch.from_numpy(table).cuda(), interleaved=inter)
    assert k8.k8v4_last_device_status() == 0
    rows = table[np.array(pos)[:, None] + np.arange(n_tok)].astype(np.float64)[:, :, None]
    y, _ = rotate64(k64, rows, inter)
    y = torch.from_numpy(y.astype(np.float32))
    y = (y.bfloat16().float() if dtype == "bf16" else y).numpy()
    ref.append(pt, np.array(pos), y, v64.astype(np.float32))
    assert np.array_equal(gpu.pages.cpu().numpy(), ref.buf)


@pytest.mark.parametrize("fmt", [k8.FORMAT_K8V4, k8.FORMAT_INT8, k8.FORMAT_Q4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_tok,H", [(1, 2), (3, 8), (900, 1), (1700, 3)])
def test_append_rope_is_norm_rope_then_append(fmt, dtype, n_tok, H):
    """With a norm: byte for byte the two calls it stands for."""
    pos = [0, 51]
    k, v, _, _, pt, n_pages = _append_inputs(3 + n_tok, 2, n_tok, dtype, True, 32, pos, H)
    table = torch.from_numpy(table_of(51 + n_tok, 128)).cuda()
    w = torch.linspace(0.5, 1.5, 256, device="cuda")
    ptd, posd = torch.from_numpy(pt).cuda(), torch.tensor(pos, dtype=torch.int64, device="cuda")
    one, two = k8.PagedCache(n_pages, 32, H, fmt), k8.PagedCache(n_pages, 32, H, fmt)
    k8.kv_append_k8v4_rope(one, ptd, posd, k, v, table, k_weight=w, eps=1e-6)
    kr = torch.empty(k.shape, dtype=k.dtype, device="cuda")
    k8.qk_norm_rope_k8v4(k, None, posd, table, kr, None, q_weight=w, eps=1e-6)
    k8.kv_append_k8v4(two, ptd, posd, kr, v.contiguous())
    assert k8.k8v4_last_device_status() == 0
    assert torch.equal(one.pages, two.pages)


@pytest.mark.parametrize("n_tok", [6, 1300])
def test_append_rope_skips_what_has_no_row_or_page(n_tok):
    """A cell past the table, past max_pages, below 0 or on a bad page id is skipped
    and recorded; the other cells are written."""
    P, H = 16, 2
    total = 64 + n_tok
    k, v, k64, v64, pt, n_pages = _append_inputs(9, 1, total, "bf16", False, P, [0])
    pt = pt.copy()
    pt[0, 1] = n_pages + 5
    table = table_of(total - 30, 64)
    gpu = k8.PagedCache(n_pages, P, H)
    gpu.pages.fill_(CANARY)
    ref = oracle.Cache(n_pages, P, H, k8.FORMAT_K8V4, fill=CANARY)
    k8.kv_append_k8v4_rope(gpu, torch.from_numpy(pt).cuda(), torch.tensor([-20], dtype=torch.int64, device="cuda"), k, v,
                           torch.from_numpy(table).cuda())
    assert k8.k8v4_last_device_status() == k8.ERANGE
    good = pt.copy()
    good[0, 1] = 0
    for lo, hi in ((0, 16), (32, total - 30)):
        t = np.arange(lo, hi) + 20
        y, _ = rotate64(k64[:, t], table[lo:hi].astype(np.float64)[None, :, None], False)
        y = torch.from_numpy(y.astype(np.float32)).bfloat16().float().numpy()
        ref.append(good, np.array([lo]), np.ascontiguousarray(y), np.ascontiguousarray(v64[:, t].astype(np.float32)))
    assert np.array_equal(gpu.pages.cpu().numpy(), ref.buf)


def test_rope_calls_captured_replayed_and_on_another_stream():
    """Both calls captured into one graph on a side stream and replayed with new inputs in
    place give what eager calls give."""
    P, pos = 16, [3, 30]
    k, v, _, _, pt, n_pages = _append_inputs(21, 2, 4, "bf16", True, P, pos)
    q, k2 = case(22, 2, 4, [16, 2], "bf16", False)[0]
    table = torch.from_numpy(table_of(64, 64)).cuda()
    ptd, posd = torch.from_numpy(pt).cuda(), torch.tensor(pos, dtype=torch.int64, device="cuda")
    outs = [torch.empty_like(q), torch.empty_like(k2)]
    cache, eager = k8.PagedCache(n_pages, P), k8.PagedCache(n_pages, P)

    def step(c, o):
        k8.qk_norm_rope_k8v4(q, k2, posd, table, *o)
        k8.kv_append_k8v4_rope(c, ptd, posd, k, v, table)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(cache, outs)
    for scale in (1.0, -0.5):
        q.mul_(scale)
        k.mul_(scale)
        posd.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(o) for o in outs]
        with torch.cuda.stream(side):
            step(eager, want)
        torch.cuda.synchronize()
        assert torch.equal(cache.pages, eager.pages) and all(torch.equal(a, b) for a, b in zip(outs, want))
    assert k8.k8v4_last_device_status() == 0


def test_calls_back_to_back_read_what_the_call_before_wrote():
    """Chains of these calls on one stream with nothing between them (each starts while the one before it drains):
    rows rotated to and fro between two buffers, cells overwritten and read back, equal to the same calls one by one."""
    n_tok, H, P = 700, 2, 16
    table = torch.from_numpy(table_of(n_tok, 128)).cuda()
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    start = torch.randn(1, n_tok, H, 256, generator=gen, device="cuda")
    v = torch.randn(1, n_tok, H, 256, generator=gen, device="cuda")
    n_pages = -(-n_tok // P)
    pt = torch.randperm(n_pages, device="cuda").int()[None].contiguous()
    rounds = 24

    def chain(pause):
        a, b = start.clone(), torch.empty_like(start)
        cache = k8.PagedCache(n_pages, P, H)
        back = torch.empty(rounds, 2, n_tok, H, 256, device="cuda")
        torch.cuda.synchronize()
        for i in range(rounds):
            for call in (lambda: k8.qk_norm_rope_k8v4(a, None, pos, table, b, None),
                         lambda: k8.qk_norm_rope_k8v4(b, None, pos, table, a, None, interleaved=True),
                         lambda: k8.kv_append_k8v4_rope(cache, pt, pos, a, v, table),
                         lambda: k8.kv_dequant_k8v4(cache, pt[0], 0, n_tok, back[i, 0], back[i, 1])):
                call()
                if pause:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return a, back

    got, want = chain(False), chain(True)
    assert k8.k8v4_last_device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
