"""spec_accept_k8v4 against a plain 64-bit implementation: vocabularies from one
token to odd large ones, ragged and missing drafts, drafts that were certain, exact
ties of the running sum, equal rows, rows that are refused, and the distribution of
the tokens that come out."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8

pytestmark = pytest.mark.gpu


def plain(p, q, drafts, counts, u, us):
    """float32 / bf16 values as float64 [B, n + 1, V] and [B, n, V] (or None)."""
    B, n = drafts.shape
    tokens = np.full((B, n + 1), -1, np.int32)
    accepted = np.zeros(B, np.int32)
    for b in range(B):
        a = 0
        while a < counts[b]:
            x = drafts[b, a]
            if not (0 <= x < p.shape[2]) or not (float(u[b, a]) * (1.0 if q is None else q[b, a, x]) < p[b, a, x]):
                break
            tokens[b, a] = x
            a += 1
        accepted[b] = a
        w = p[b, a]
        if a < counts[b]:
            if q is None:
                less = w.copy()
                if 0 <= drafts[b, a] < p.shape[2]:
                    less[drafts[b, a]] = 0
            else:
                less = np.maximum((w.astype(np.float32) - q[b, a].astype(np.float32)).astype(np.float64), 0)
            if less.sum() > 0:
                w = less
        c = np.cumsum(w)
        if c[-1] > 0:
            tokens[b, a] = int(np.argmax(c > float(us[b]) * c[-1]))
    return tokens, accepted


def call(p, q, drafts, counts, u, us, dtype=torch.float32):
    B, n = drafts.shape
    dev = lambda x, dt: torch.from_numpy(np.ascontiguousarray(x)).to(dt).cuda()
    tokens = torch.full((B, n + 1), -7, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    k8.spec_accept_k8v4(dev(p, dtype), None if q is None else dev(q, dtype), dev(drafts, torch.int32),
                        dev(u, torch.float32), dev(us, torch.float32), tokens, acc,
                        n_drafts=None if counts is None else dev(counts, torch.int32))
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), acc.cpu().numpy()


def inputs(seed, B, n, V, spread=2.0, noise=0.5):
    rng = np.random.default_rng(seed)

    def soft(z):
        e = np.exp(z - z.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)

    z = spread * rng.standard_normal((B, n + 1, V))
    p = soft(z)
    q = soft(z[:, :n] + noise * rng.standard_normal((B, n, V)))
    drafts = np.zeros((B, n), np.int32)
    for b in range(B):
        for i in range(n):
            drafts[b, i] = min(V - 1, int(np.searchsorted(np.cumsum(q[b, i], dtype=np.float64), rng.random())))
    return p, q, drafts, rng.integers(0, n + 1, B), rng.random((B, n), np.float32), rng.random(B, np.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (3, 2, 2), (5, 4, 31), (40, 7, 33), (9, 4, 1000), (6, 32, 777),
                                   (4, 3, 4099), (17, 5, 20011), (2, 4, 131071), (1, 1, 300001), (45, 1, 40003), (3, 2, 40004), (1, 2, 70000)])
def test_accept_against_64_bits(dtype, certain, B, n, V):
    p, q, drafts, counts, u, us = inputs(B + 7 * n + V, B, n, V)
    r = lambda x: torch.from_numpy(x).to(dtype).double().numpy()
    p64, q64 = r(p), None if certain else r(q)
    for c in (counts, None):
        got = call(p, None if certain else q, drafts, c, u, us, dtype)
        want = plain(p64, q64, drafts, np.full(B, n) if c is None else c, u, us)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert k8.k8v4_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_accept_rows_at_any_element(dtype):
    """Probabilities that begin one element behind an aligned address, beside drafts' that do not."""
    B, n, V = 2, 3, 50000
    p, q, drafts, counts, u, us = inputs(11, B, n, V)
    shift = torch.empty(B * (n + 1) * V + 1, dtype=dtype, device="cuda")[1:].view(B, n + 1, V)
    shift.copy_(torch.from_numpy(p))
    qd = torch.from_numpy(q).to(dtype).cuda()
    tokens, acc = torch.empty(B, n + 1, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    k8.spec_accept_k8v4(shift, qd, torch.from_numpy(drafts).cuda(), torch.from_numpy(u).cuda(), torch.from_numpy(us).cuda(), tokens, acc)
    want = plain(shift.double().cpu().numpy(), qd.double().cpu().numpy(), drafts, np.full(B, n), u, us)
    assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(acc.cpu().numpy(), want[1])


def test_accept_no_drafts():
    p, _, _, _, _, us = inputs(3, 6, 0, 500)
    got = call(p, None, np.zeros((6, 0), np.int32), None, np.zeros((6, 0), np.float32), us)
    want = plain(p.astype(np.float64), None, np.zeros((6, 0), np.int32), np.zeros(6, int), None, us)
    assert np.array_equal(got[0], want[0]) and not got[1].any()


@pytest.mark.parametrize("V", [64, 4096, 65536])
def test_accept_exact_ties_and_ends(V):
    """Equal probabilities 1 / V: the running sum meets u W exactly at u = j / V and the token is then j (the
    smallest index whose sum passes it); u = 0 gives the first token, u next to 1 the last."""
    us = np.array([0.0, 1 / V, 0.25, 0.5, (V - 1) / V, np.nextafter(np.float32(1), np.float32(0)), 0.5 - 2.0 ** -25], np.float32)
    B = len(us)
    p = np.full((B, 1, V), 1 / V, np.float32)
    got = call(p, None, np.zeros((B, 0), np.int32), None, np.zeros((B, 0), np.float32), us)[0][:, 0]
    assert got.tolist() == [0, 1, V // 4, V // 2, V - 1, V - 1, V // 2 - 1]


def test_accept_leading_and_trailing_zeros():
    """Zero weights ahead of and behind the only token with one are never drawn."""
    for V, at in ((5000, 0), (5000, 4999), (70000, 31337), (3, 1)):
        us = np.array([0.0, 0.3, 1 - 2.0 ** -24], np.float32)
        p = np.zeros((3, 1, V), np.float32)
        p[:, 0, at] = 0.7
        got = call(p, None, np.zeros((3, 0), np.int32), None, np.zeros((3, 0), np.float32), us)[0]
        assert (got[:, 0] == at).all(), (V, at, got)


def test_accept_equal_rows_and_zero_probability_drafts():
    """p = q: every draft with u < 1 is accepted; a draft of target probability 0 never is, at u = 0 either; where
    nothing of p - q is left, the target row is drawn from."""
    p, q, drafts, _, u, us = inputs(11, 8, 3, 300)
    q = p[:, :3].copy()
    got = call(p, q, drafts, None, u, us)
    assert (got[1] == 3).all()
    p[:, 1, :] = 0
    p[:, 1, 5] = 1
    q[:, 1, :] = 0
    q[:, 1, 5] = 1
    drafts[:, 1] = 6                                  # the target (and the draft row) give it probability 0
    u[:, 1] = 0
    got = call(p, q, drafts, None, u, us)
    want = plain(p.astype(np.float64), q.astype(np.float64), drafts, np.full(8, 3), u, us)
    assert (got[1] == 1).all() and (got[0][:, 1] == 5).all() and np.array_equal(got[0], want[0])
    assert k8.k8v4_last_device_status() == 0


def test_accept_records_and_survives_bad_values():
    """Drafts outside the vocabulary, draft counts out of range, rows of zeros, of NaN and with an infinity: recorded,
    refused (token -1 where there is nothing to draw from), the other sequences as they should be."""
    V = 1200
    p, q, drafts, _, u, us = inputs(13, 8, 3, V)
    u[:] = 0                                          # every draft of positive probability is accepted
    counts = np.array([3, 3, 9, -4, 3, 3, 3, 3])
    drafts[0, 1] = V
    drafts[1, 0] = -1
    p[4, 3] = 0
    p[5, 3] = np.nan
    p[6, 3, 77] = np.inf
    got = call(p, q, drafts, counts, u, us)
    assert k8.k8v4_last_device_status() == k8.ERANGE
    assert k8.k8v4_last_device_status() == 0
    assert got[1].tolist() == [1, 0, 3, 0, 3, 3, 3, 3]
    want = plain(np.where(np.isfinite(p), p, 0).astype(np.float64), q.astype(np.float64), drafts, counts.clip(0, 3), u, us)
    for b in (0, 1, 2, 3, 7):
        assert np.array_equal(got[0][b], want[0][b])
    assert [got[0][b, 3] for b in (4, 5, 6)] == [-1, -1, -1]


def test_accept_keeps_the_targets_distribution():
    """60,000 sequences of two drafts over 7 tokens: the first token's frequencies are the target's within 5
    standard deviations of a binomial, although the drafts come from another distribution."""
    rng = np.random.default_rng(17)
    B, V = 60000, 7
    p1 = np.array([.3, .05, .2, 0, .15, .25, .05], np.float32)
    q1 = np.array([.1, .3, .1, .2, .1, .1, .1], np.float32)
    drafts = rng.choice(V, (B, 2), p=q1.astype(np.float64) / q1.sum(dtype=np.float64)).astype(np.int32)
    got, _ = call(np.broadcast_to(p1, (B, 3, V)), np.broadcast_to(q1, (B, 2, V)), drafts, None,
                  rng.random((B, 2), np.float32), rng.random(B, np.float32))
    freq = np.bincount(got[:, 0], minlength=V) / B
    assert np.all(np.abs(freq - p1) <= 5 * np.sqrt(p1 * (1 - p1) / B) + 1e-12)


def test_accept_captured_and_replayed():
    p, q, drafts, counts, u, us = inputs(19, 5, 4, 9001)
    d = [torch.from_numpy(x).cuda() for x in (p, q, drafts, u, us)]
    tokens = torch.empty(5, 5, dtype=torch.int32, device="cuda")
    acc = torch.empty(5, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k8.spec_accept_k8v4(d[0], d[1], d[2], d[3], d[4], tokens, acc)
    for seed in (1, 2):
        us2 = np.random.default_rng(seed).random(5, np.float32)
        d[4].copy_(torch.from_numpy(us2))
        graph.replay()
        torch.cuda.synchronize()
        want = plain(p.astype(np.float64), q.astype(np.float64), drafts, np.full(5, 4), u, us2)
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(acc.cpu().numpy(), want[1])
