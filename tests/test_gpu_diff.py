"""attn_k8v4_diff_decode and attn_k8v4_diff against differential attention in 64 bits over
the cache's bytes: lengths from none to long ones, ragged batches, heads, page sizes, query types, weights,
steps that leave rows empty, what is refused and recorded, streams and captured calls."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from diff_util import all_cells, check, expected, filled_cache, weights

pytestmark = pytest.mark.gpu


def tables(rng, lens, n_pages, P, extra=1):
    """A row of distinct pages per sequence, behind them entries that no cell reaches."""
    need = [-(-int(n) // P) for n in lens]
    width = max(need + [1]) + extra
    ids = rng.permutation(n_pages).astype(np.int32)
    pt = np.full((len(lens), width), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        pt[b, :n] = ids[at:at + n]
        at += n
    return pt


def cells_of(pt_row, n, P):
    c = np.arange(n)
    return torch.from_numpy(pt_row[c // P].astype(np.int64) * P + c % P).cuda()


def queries(rng, n, HQ, dtype, gain=1.0):
    q = torch.from_numpy((gain * rng.standard_normal((n, HQ, 256))).astype(np.float32)).cuda()
    return q if dtype == "f32" else q.bfloat16()


def fp16_of(q):
    """The fp16 values that fp32 queries enter the products as: a power of two per row and map puts the largest at
    2^14 .. 2^15."""
    if q.dtype != torch.float32:
        return q.double()
    x = q.double().unflatten(-1, (2, 128))
    top = x.abs().amax(-1, keepdim=True)
    up = torch.where(top > 0, 2.0 ** (14 - torch.floor(torch.log2(top.clamp(min=1e-300)))), 1.0)
    return ((x * up).half().double() / up).flatten(-2)


def decode_case(seed, lens, H, P, dtype="bf16", n_lambda=1, norm=True, q_gain=1.0, k_gain=1.0, v_gain=1.0, init=0.6):
    rng = np.random.default_rng(seed)
    pages = sum(-(-int(n) // P) for n in lens) + 2
    cache = filled_cache(rng, pages, P, H, k_gain, v_gain)
    pt = tables(rng, lens, pages, P)
    HQ = 8 * H
    q = queries(rng, len(lens), HQ, dtype, q_gain)
    heads, lam, w = weights(rng, HQ if n_lambda > 1 else n_lambda, init=init, norm=norm)
    return cache, pt, q, heads, lam, w, init


def run_decode(cache, pt, q, lens, heads, max_len=None, stream=None):
    max_len = int(max(lens)) if max_len is None else max_len
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    ws = k8.diff_decode_workspace(cache, len(lens), max_len)
    k8.attn_k8v4_diff_decode(cache, q, torch.from_numpy(pt).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             max_len, heads, out, ws, stream=stream)
    return out


def check_decode(cache, pt, q, lens, lam, w, init, out, P, out_scale=0.4):
    cells = all_cells(cache)
    for b, n in enumerate(lens):
        want, bound = expected(cells, fp16_of(q)[b:b + 1], cells_of(pt[b], int(n), P), [int(n)], lam, init, w, out_scale)
        check(out[b:b + 1], want, bound)


@pytest.mark.parametrize("lens,H,P,dtype,n_lambda,norm", [
    ([1], 2, 16, "bf16", 1, True), ([0, 3, 15, 16, 17], 2, 16, "bf16", 2, True), ([31, 33, 0, 250], 1, 48, "f32", 1, True),
    ([1000], 2, 64, "bf16", 0, False), ([4099, 5, 2048], 3, 64, "bf16", 2, True), ([513, 1024], 8, 128, "f32", 2, False),
    ([20011], 2, 64, "bf16", 1, True), ([0, 0], 2, 16, "bf16", 1, True)])
def test_decode(lens, H, P, dtype, n_lambda, norm):
    cache, pt, q, heads, lam, w, init = decode_case(len(lens) + H, lens, H, P, dtype, n_lambda, norm)
    out = run_decode(cache, pt, q, lens, heads, max_len=max(max(lens), 1))
    assert k8.k8v4_last_device_status() == 0
    check_decode(cache, pt, q, lens, lam, w, init, out, P)
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all()


@pytest.mark.parametrize("q_gain,k_gain,v_gain,init", [(30.0, 1.0, 1.0, 0.6), (1e-3, 1.0, 1e3, 1.0), (0.0, 1.0, 1.0, -2.0),
                                                       (1.0, 1e-6, 1e-3, 0.0), (1e4, 1e-4, 30.0, 0.5)])
def test_decode_scales(q_gain, k_gain, v_gain, init):
    """Peaked and flat maps (all queries 0: both maps are the mean), small and large values, weights of 0 and below."""
    lens = [700, 65]
    cache, pt, q, heads, lam, w, init = decode_case(5, lens, 2, 64, q_gain=q_gain, k_gain=k_gain, v_gain=v_gain, init=init, n_lambda=0,
                                                    norm=False)
    out = run_decode(cache, pt, q, lens, heads)
    check_decode(cache, pt, q, lens, lam, w, init, out, 64)


def test_equal_maps_cancel():
    """The same query and key in both halves and a weight of 1: nothing is left but the roundings, and without a norm
    they stay under their bound."""
    rng = np.random.default_rng(8)
    P, n = 64, 500
    cache = k8.PagedCache(9, P)
    half = rng.standard_normal((1, 9 * P, 2, 128)).astype(np.float32)
    k = torch.from_numpy(np.concatenate([half, half], -1)).cuda()
    v = torch.from_numpy(rng.standard_normal((1, 9 * P, 2, 256)).astype(np.float32)).cuda()
    pt = np.arange(9, dtype=np.int32)[None]
    k8.kv_append_k8v4(cache, torch.from_numpy(pt).cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), k, v)
    q = torch.randn(1, 16, 128, device="cuda").bfloat16().repeat(1, 1, 2)
    out = run_decode(cache, pt, q, [n], k8.DifferentialHeads(lambda_init=1.0))
    want, bound = expected(all_cells(cache), q.double(), cells_of(pt[0], n, P), [n], None, 1.0, None, 1.0)
    check(out, want, bound)


def test_decode_bad_values_are_recorded():
    lens = [100, 130, 90]
    cache, pt, q, heads, lam, w, init = decode_case(9, lens, 2, 16)
    good = run_decode(cache, pt, q, lens, heads, max_len=130)
    # a length past the bound is clipped, a negative one counts as 0
    out = run_decode(cache, pt, q, [100, 2000, -5], heads, max_len=130)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    assert torch.equal(out[:2], good[:2]) and (out[2] == 0).all()
    # pages out of range are skipped
    bad = pt.copy()
    bad[1, 2], bad[1, 5] = cache.n_pages, -3
    out = run_decode(cache, bad, q, lens, heads, max_len=130)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    ids = cells_of(pt[1], 130, 16)
    keep = torch.tensor([c for c in range(130) if c // 16 not in (2, 5)], device="cuda")
    want, bound = expected(all_cells(cache), fp16_of(q)[1:2], ids[keep], [len(keep)], lam, init, w, 0.4)
    check(out[1:2], want, bound)
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


def test_decode_same_bits_each_time_and_on_another_stream():
    lens = [3000, 41, 1999]
    cache, pt, q, heads, lam, w, init = decode_case(10, lens, 2, 64)
    a = run_decode(cache, pt, q, lens, heads)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = run_decode(cache, pt, q, lens, heads)
    c = run_decode(cache, pt, q, lens, heads, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


# ---------------------------------------------------------------- ragged batches
def ragged(rng, n, lens, H, P, dtype, n_lambda=1, norm=True, tail=0):
    pages = sum(-(-int(x) // P) for x in lens) + 2
    cache = filled_cache(rng, pages, P, H)
    pt = tables(rng, lens, pages, P)
    HQ = 8 * H
    T = int(sum(n)) + tail
    q = queries(rng, T, HQ, dtype)
    heads, lam, w = weights(rng, HQ if n_lambda > 1 else n_lambda, norm=norm)
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return cache, pt, q, heads, lam, w, off


def run_ragged(cache, pt, q, off, lens, heads, steps=None, max_len=None, out=None, ws=None):
    max_len = int(max(lens)) if max_len is None else max_len
    out = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = k8.diff_workspace(cache, len(lens), q.shape[0], max_len) if ws is None else ws
    k8.attn_k8v4_diff(cache, q, torch.from_numpy(off).cuda(), torch.from_numpy(pt).cuda(),
                      torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len, heads, out, ws,
                      steps=None if steps is None else torch.from_numpy(np.asarray(steps, np.int32)).cuda())
    return out


def check_ragged(cache, pt, q, off, lens, lam, w, out, P, steps=None, init=0.6, only=None):
    cells = all_cells(cache)
    for b, n in enumerate(lens):
        lo, hi = int(off[b]), int(off[b + 1])
        if hi == lo:
            continue
        sees = np.maximum(n - (hi - lo) + 1 + np.arange(hi - lo), 0) if steps is None else np.asarray(steps[lo:hi])
        pick = np.arange(hi - lo) if only is None else np.unique(np.linspace(0, hi - lo - 1, only).astype(int))
        want, bound = expected(cells, fp16_of(q)[lo + pick], cells_of(pt[b], int(n), P), sees[pick], lam, init, w, 0.4)
        check(out[lo + torch.from_numpy(pick).cuda()], want, bound)


@pytest.mark.parametrize("n,lens,H,P,dtype,n_lambda,norm,tail", [
    ([1], [1], 2, 16, "bf16", 1, True, 0),                               # one token that sees itself
    ([5, 1, 0, 3], [5, 260, 30, 64], 2, 16, "bf16", 2, True, 4),          # a batch with an idle sequence, padding behind it
    ([33, 31, 1, 32], [33, 95, 129, 128], 1, 48, "f32", 1, False, 0),      # around a row tile's and a cell tile's ends
    ([17, 16, 15], [1017, 500, 15], 3, 128, "bf16", 0, True, 1),
    ([129, 7, 64], [700, 2000, 64], 2, 64, "bf16", 2, True, 0),
    ([40], [40], 8, 16, "bf16", 2, True, 0),
    ([300, 200], [301, 5000], 2, 64, "bf16", 1, True, 3)])
def test_ragged(n, lens, H, P, dtype, n_lambda, norm, tail):
    rng = np.random.default_rng(sum(n) + H)
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, H, P, dtype, n_lambda, norm, tail)
    out = run_ragged(cache, pt, q, off, lens, heads)
    assert k8.k8v4_last_device_status() == 0
    check_ragged(cache, pt, q, off, lens, lam, w, out, P)
    assert (out[int(off[-1]):] == 77.0).all()                           # rows behind the last sequence


def test_ragged_long():
    """A chunk far into a long document and single tokens of others: many cell ranges, sums over long runs."""
    n, lens = [96, 1, 2], [40011, 30000, 9]
    rng = np.random.default_rng(77)
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, 2, 64, "bf16")
    out = run_ragged(cache, pt, q, off, lens, heads)
    assert k8.k8v4_last_device_status() == 0
    check_ragged(cache, pt, q, off, lens, lam, w, out, 64, only=6)


def test_ragged_prompt():
    """A whole prompt, each token seeing one more cell."""
    n, lens = [1500], [1500]
    rng = np.random.default_rng(78)
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, 2, 16, "bf16")
    out = run_ragged(cache, pt, q, off, lens, heads)
    check_ragged(cache, pt, q, off, lens, lam, w, out, 16, only=40)


def test_steps_and_empty_rows():
    rng = np.random.default_rng(11)
    n, lens = [9, 40], [300, 1000]
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, 2, 64, "bf16", tail=2)
    steps = np.concatenate([rng.integers(0, 301, 9), rng.integers(0, 1001, 40), [0, 0]])
    steps[[0, 3, 20]] = 0
    steps[5], steps[30] = 300, 1000
    out = run_ragged(cache, pt, q, off, lens, heads, steps=steps)
    assert k8.k8v4_last_device_status() == 0
    check_ragged(cache, pt, q, off, lens, lam, w, out, 64, steps=steps)
    assert (out[[0, 3, 20]] == 0).all()
    # a step past its sequence's length is clipped to it, one below 0 counts as 0
    steps[1], steps[2] = 301, -1
    out2 = run_ragged(cache, pt, q, off, lens, heads, steps=steps)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    steps[1], steps[2] = 300, 0
    assert torch.equal(out2[:49], run_ragged(cache, pt, q, off, lens, heads, steps=steps)[:49])


def test_more_tokens_than_cells():
    """Tokens ahead of the first cell see nothing."""
    rng = np.random.default_rng(12)
    cache, pt, q, heads, lam, w, off = ragged(rng, [8], [3], 2, 16, "bf16")
    out = run_ragged(cache, pt, q, off, [3], heads)
    assert (out[:5] == 0).all()
    check_ragged(cache, pt, q, off, [3], lam, w, out, 16)


def test_bad_offsets_and_lengths_leave_their_sequence_out():
    rng = np.random.default_rng(13)
    n, lens = [6, 5, 7], [50, 60, 70]
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, 2, 16, "bf16")
    good = run_ragged(cache, pt, q, off, lens, heads)
    bad = off.copy()
    bad[3] = 19                                            # past the packed tokens
    out = run_ragged(cache, pt, q, bad, lens, heads)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    assert torch.equal(out[:11], good[:11]) and (out[11:] == 77.0).all()
    out = run_ragged(cache, pt, q, off, [50, 4000, -2], heads, max_len=70)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    assert torch.equal(out[:6], good[:6]) and (out[11:] == 0).all()


def test_ragged_equals_decode_for_single_tokens():
    """The two calls state one operator: single tokens through either agree to the sum of their bounds."""
    rng = np.random.default_rng(14)
    n, lens = [1] * 9, [int(x) for x in rng.integers(1, 3000, 9)]
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, 2, 64, "bf16")
    a, b = run_ragged(cache, pt, q, off, lens, heads), run_decode(cache, pt, q, lens, heads)
    cells = all_cells(cache)
    for i, L in enumerate(lens):
        _, bound = expected(cells, q.double()[i:i + 1], cells_of(pt[i], L, 64), [L], lam, 0.6, w, 0.4)
        assert ((a[i:i + 1].double() - b[i:i + 1].double()).norm(dim=-1) <= 2 * bound).all()


def test_captured_calls():
    """Two captured calls, each with its own workspace, replayed in turn and at the same time on two streams, after
    their inputs changed."""
    rng = np.random.default_rng(15)
    n, lens = [20, 1, 70], [400, 900, 70]
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, 2, 64, "bf16")
    ptd, offd, lensd = torch.from_numpy(pt).cuda(), torch.from_numpy(off).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    graphs, outs, qs = [], [], []
    for i in range(2):
        qi, out = torch.zeros_like(q), torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        ws = k8.diff_workspace(cache, 3, q.shape[0], 900)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            k8.attn_k8v4_diff(cache, qi, offd, ptd, lensd, 900, heads, out, ws)
        graphs.append((g, ws))
        outs.append(out)
        qs.append(qi)
    for i in range(2):
        qs[i].copy_(q if i == 0 else -q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], run_ragged(cache, pt, q, off, lens, heads))
    assert torch.equal(outs[1], run_ragged(cache, pt, -q, off, lens, heads))
    assert k8.k8v4_last_device_status() == 0
