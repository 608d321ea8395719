"""attn_k8v4_diff_decode and attn_k8v4_diff where their ways part: batches of many short sequences
(a piece of the line of tiles with several of them), ragged batches whose sequences go one token at a time, by
token tiles, or both, every box and stage size of the tile kernel, two calls at once, and waits that run out."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from test_gpu_diff import (check_decode, check_ragged, decode_case, ragged, run_decode, run_ragged)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,longest,H,P", [(120, 70, 2, 16), (400, 20, 1, 16), (60, 400, 8, 64)])
def test_many_short_sequences(seqs, longest, H, P):
    rng = np.random.default_rng(seqs)
    lens = [int(x) for x in rng.integers(0, longest + 1, seqs)]
    lens[0] = lens[-1] = 0
    lens[seqs // 2] = longest
    cache, pt, q, heads, lam, w, init = decode_case(seqs + 1, lens, H, P)
    out = run_decode(cache, pt, q, lens, heads)
    assert k8.k8v4_last_device_status() == 0
    pick = [0, 1, 2, seqs // 2 - 1, seqs // 2, seqs // 2 + 1, seqs - 2, seqs - 1] + [int(x) for x in rng.integers(0, seqs, 24)]
    check_decode(cache, pt[pick], q[pick], [lens[b] for b in pick], lam, w, init, out[pick], P)
    assert (out[0] == 0).all() and (out[-1] == 0).all()


def test_one_long_among_short():
    """A sequence of many pieces between sequences of a part of one."""
    lens = [3, 90, 1, 50001, 17, 0, 260]
    cache, pt, q, heads, lam, w, init = decode_case(5, lens, 2, 64, n_lambda=2)
    out = run_decode(cache, pt, q, lens, heads)
    check_decode(cache, pt, q, lens, lam, w, init, out, 64)


@pytest.mark.parametrize("n,lens,H,P,dtype", [
    ([1] * 30 + [0, 2, 1], [700] * 33, 2, 64, "bf16"),                    # one token each: all one at a time
    ([4, 3, 2, 1], [9000, 9000, 9000, 9000], 2, 16, "f32"),
    ([8] * 6, [3000] * 6, 2, 64, "bf16"),                                 # eight each: token tiles
    ([1] * 20 + [200, 90], [3000] * 20 + [500, 2000], 2, 64, "bf16"),      # both in a call
    ([1, 150, 2, 1, 40, 1], [4000, 150, 6000, 5000, 1000, 0], 3, 32, "bf16"),
    ([40], [700], 8, 32, "bf16"),                                         # one stage of raw tiles, boxes of 32 cells
    ([33, 1], [1500, 900], 7, 96, "f32")])
def test_ways(n, lens, H, P, dtype):
    rng = np.random.default_rng(sum(n) + H + P)
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, H, P, dtype, 2, True, 3)
    out = run_ragged(cache, pt, q, off, lens, heads)
    assert k8.k8v4_last_device_status() == 0
    check_ragged(cache, pt, q, off, lens, lam, w, out, P, only=12)
    assert (out[int(off[-1]):] == 77.0).all()


def test_steps_one_token_at_a_time():
    """Sequences of few tokens with steps of their own, some that see nothing, one past its length."""
    rng = np.random.default_rng(21)
    n, lens = [3, 1, 5, 2], [4000, 6000, 5000, 9]
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, 2, 64, "bf16")
    steps = np.array([0, 4000, 17, 5999, 1, 5000, 0, 2500, 4999, 9, 0])
    out = run_ragged(cache, pt, q, off, lens, heads, steps=steps)
    assert k8.k8v4_last_device_status() == 0
    check_ragged(cache, pt, q, off, lens, lam, w, out, 64, steps=steps)
    assert (out[[0, 6, 10]] == 0).all()
    steps[3], steps[6] = 6001, -4
    again = run_ragged(cache, pt, q, off, lens, heads, steps=steps)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    steps[3], steps[6] = 6000, 0
    assert torch.equal(again, run_ragged(cache, pt, q, off, lens, heads, steps=steps))


def test_offsets_that_overlap_stay_in_bounds():
    """Offsets that do not follow one another name tokens twice; every write stays inside the call's arrays."""
    rng = np.random.default_rng(22)
    n, lens = [2, 2, 40], [300, 300, 300]
    cache, pt, q, heads, lam, w, off = ragged(rng, n, lens, 2, 64, "bf16")
    guard = torch.full((q.shape[0] + 2, *q.shape[1:]), 77.0, dtype=torch.bfloat16, device="cuda")
    size = k8.diff_workspace(cache, 3, q.shape[0], 300).numel()
    room = torch.full((size + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    for bad in ([0, 44, 0, 44], [40, 44, 2, 44], [0, 2, 1, 44], [44, 44, 44, 0], [0, 4, 0, 8]):
        run_ragged(cache, pt, q, np.asarray(bad, np.int32), lens, heads, out=guard[1:-1], ws=room[:size])
        assert k8.k8v4_last_device_status() in (0, k8.ERANGE)
        assert (guard[0] == 77.0).all() and (guard[-1] == 77.0).all() and (room[size:] == 0x5a).all()


def test_two_calls_at_once():
    """Two streams, a workspace each, one batch of single queries and one ragged: the bits of the calls alone."""
    rng = np.random.default_rng(23)
    lens = [int(x) for x in rng.integers(1, 9000, 12)]
    cache, pt, q, heads, *_ = decode_case(24, lens, 2, 64)
    n, lens2 = [1, 70, 3, 1], [5000, 700, 4000, 20]
    cache2, pt2, q2, heads2, _, _, off2 = ragged(rng, n, lens2, 2, 64, "bf16")
    a, b = run_decode(cache, pt, q, lens, heads), run_ragged(cache2, pt2, q2, off2, lens2, heads2)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        with torch.cuda.stream(one):
            x = run_decode(cache, pt, q, lens, heads)
        with torch.cuda.stream(two):
            y = run_ragged(cache2, pt2, q2, off2, lens2, heads2)
        got.append((x, y))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, a) and torch.equal(y, b)


def test_waits_that_run_out():
    """With a bound below a microsecond a wait that is not complete at once gives up: the kernels record it, wait for
    their own copies and products and return.  The calls after it give the bits of those before."""
    rng = np.random.default_rng(25)
    lens = [20000, 300]
    cache, pt, q, heads, *_ = decode_case(26, lens, 2, 64)
    n, lens2 = [40], [700]
    cache2, pt2, q2, heads2, _, _, off2 = ragged(rng, n, lens2, 2, 64, "bf16")
    a, b = run_decode(cache, pt, q, lens, heads), run_ragged(cache2, pt2, q2, off2, lens2, heads2)
    assert k8.k8v4_last_device_status() == 0
    try:
        k8.k8v4_set_wait_limit_ns(1)
        run_decode(cache, pt, q, lens, heads)
        torch.cuda.synchronize()
        assert k8.k8v4_last_device_status() in (0, k8.ECUDA)             # its copies may have landed
        run_ragged(cache2, pt2, q2, off2, lens2, heads2)
        torch.cuda.synchronize()
        assert k8.k8v4_last_device_status() == k8.ECUDA
    finally:
        k8.k8v4_set_wait_limit_ns(0)
    assert torch.equal(run_decode(cache, pt, q, lens, heads), a)
    assert torch.equal(run_ragged(cache2, pt2, q2, off2, lens2, heads2), b)
    assert k8.k8v4_last_device_status() == 0
