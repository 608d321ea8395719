"""What the differential attention's operands keep, where it shows: values far below and far above 1, cells whose values
differ by as much, a large weight beside many small ones, fp32 queries that need more than fp16's bits."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from diff_util import BF16_HALF, F16_HALF, all_cells, check, expected, weights
from test_gpu_diff import queries

pytestmark = pytest.mark.gpu


def cache_of(k, v, P=64):
    """One sequence: k, v float32 numpy [n, H, 256]."""
    n, H, _ = k.shape
    pages = -(-n // P)
    cache = k8.PagedCache(pages, P, H)
    cache.pages.zero_()
    pt = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    k8.kv_append_k8v4(cache, pt, torch.zeros(1, dtype=torch.int64, device="cuda"), torch.from_numpy(k)[None].cuda(), torch.from_numpy(v)[None].cuda())
    assert k8.k8v4_last_device_status() == 0
    return cache, pt


def attend(way, cache, pt, q, n, heads):
    """The last cells' queries through either kernel: one by one ("one"), or as the first tokens of a prompt chunk
    long enough for token tiles ("tile"), whose other tokens see as many cells."""
    if way == "one":
        out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        lens = torch.full((len(q),), n, dtype=torch.int32, device="cuda")
        ws = k8.diff_decode_workspace(cache, len(q), n)
        k8.attn_k8v4_diff_decode(cache, q, pt.expand(len(q), -1).contiguous(), lens, n, heads, out, ws)
        return out
    T = 40
    packed = q.repeat(-(-T // len(q)), 1, 1)[:T].contiguous()
    out = torch.empty(packed.shape, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    k8.attn_k8v4_diff(cache, packed, torch.tensor([0, T], **i32), pt, torch.tensor([n], **i32), n, heads, out,
                      k8.diff_workspace(cache, 1, T, n), steps=torch.full((T,), n, **i32))
    return out[:len(q)]


WAYS = pytest.mark.parametrize("way", ["one", "tile"])


@WAYS
@pytest.mark.parametrize("gain", [1e-7, 1e-6, 1e-5, 3e-4, 1.0, 3e3, 3e4])
@pytest.mark.parametrize("n", [1, 3, 200])
def test_values_of_any_size(way, gain, n):
    """V enters the products with half a step of fp16 at most, down to scales that are subnormal and up to those that
    eight times over fp16 does not hold."""
    rng = np.random.default_rng(n)
    v = (gain * np.clip(rng.standard_normal((n, 2, 256)), -1, 1)).astype(np.float32)
    if gain > 1e4:
        v[::2] = gain * np.where(rng.random((len(v[::2]), 2, 1)) < 0.5, 1, -1)         # 16 times that in one rotated element
    cache, pt = cache_of((rng.standard_normal((n, 2, 256))).astype(np.float32), v)
    q = queries(rng, 2, 16, "bf16", 2.0)
    cells = all_cells(cache)
    heads, lam, w = weights(rng, 1, norm=False)
    out = attend(way, cache, pt, q, n, heads)
    assert k8.k8v4_last_device_status() == 0
    want, bound = expected(cells, q.double(), torch.arange(n, device="cuda"), [n] * 2, lam, 0.6, w, 0.4)
    check(out, want, bound)


@WAYS
def test_cells_of_all_sizes(way):
    """Cells of small, ordinary, large and the largest values in one sequence, each kind far ahead in a row of its
    own."""
    rng = np.random.default_rng(5)
    n = 700
    kind = np.arange(n) // 64 % 4                          # (beside values of 2^16 those below 2^-11 keep 2^-22)
    k = (0.1 * rng.standard_normal((n, 2, 256))).astype(np.float32)
    k[:, :, :4] = 0
    k[:, :, :128] += 0.5 * np.eye(128, dtype=np.float32)[kind][:, None]          # lane `kind` of the first map's keys
    v = (np.array([1e-5, 1.0, 1e3, 1.0])[kind][:, None, None] * rng.standard_normal((n, 2, 256))).astype(np.float32)
    big = kind == 3
    v[big] += 3e4 * np.where(rng.random((big.sum(), 2, 1)) < 0.5, 1, -1).astype(np.float32)
    cache, pt = cache_of(k, v)
    cells = all_cells(cache)
    q = torch.zeros(4, 16, 256, device="cuda")
    for r in range(4):                                     # row r: its own kind far ahead of the others
        q[r, :, r], q[r, :, 128:] = 2000.0, 0.3
    q = q.bfloat16()
    heads = k8.DifferentialHeads(lambda_init=0.0)
    out = attend(way, cache, pt, q, n, heads)
    assert k8.k8v4_last_device_status() == 0
    want, bound = expected(cells, q.double(), torch.arange(n, device="cuda"), [n] * 4, None, 0.0, None, 1.0)
    check(out, want, bound)


@WAYS
@pytest.mark.parametrize("n", [5, 130, 200])
def test_cells_that_nobody_sees_change_no_bit(way, n):
    """Small values in front of cells whose bytes are those of the largest scales, or 0."""
    rng = np.random.default_rng(n)
    k, v = (rng.standard_normal((n, 2, 256)).astype(np.float32) for _ in range(2))
    cache, pt = cache_of(k, 1e-6 * v, P=256)
    q = queries(rng, 2, 16, "bf16", 2.0)
    heads = k8.DifferentialHeads(lambda_init=0.5)
    a = attend(way, cache, pt, q, n, heads)
    P, H = 256, 2
    run = cache.pages.view(-1)[392 * H * P:].view(P, H * 16)
    assert (run[n:] == 0).all()
    run[n:] = 0x7b
    b = attend(way, cache, pt, q, n, heads)
    assert k8.k8v4_last_device_status() == 0 and torch.equal(a, b) and (a != 0).any()


@WAYS
@pytest.mark.parametrize("n,gap", [(3000, 14.0), (30000, 20.0), (30000, 28.0)])
def test_many_small_weights_beside_a_large_one(way, n, gap):
    """A first cell that takes nearly all the weight and has no value, as the first token of a text often does: the
    result is what the many others add, each 2^-`gap` of it or so.  Weights are fp16 with at least 2^5 as the largest:
    a subnormal one is off by half of 2^-24, so by 2^-30 of the largest at most."""
    rng = np.random.default_rng(n)
    k = (0.3 * rng.standard_normal((n, 1, 256))).astype(np.float32)
    v = (1.0 + 0.5 * rng.standard_normal((n, 1, 256))).astype(np.float32)
    k[:, :, 0] = k[:, :, 128] = 0
    v[0] = 0
    q = 0.5 * rng.standard_normal((2, 8, 256)).astype(np.float32)
    q[:, :, 0] = q[:, :, 128] = 4.0
    k[0, :, 0] = k[0, :, 128] = gap * np.log(2) * 128 ** 0.5 / 4.0
    cache, pt = cache_of(k, v)
    q = torch.from_numpy(q).bfloat16().cuda()
    heads = k8.DifferentialHeads(lambda_init=-0.5)
    out = attend(way, cache, pt, q, n, heads)
    cells = all_cells(cache)
    want, bound = expected(cells, q.double(), torch.arange(n, device="cuda"), [n] * 2, None, -0.5, None, 1.0)
    lost = 2.0 ** -30 * 1.5 * cells[1][1:, 0].abs().sum(0).norm().item()
    assert lost < 0.4 * want.norm(dim=-1).min().item()   # (else it would be seen too late)
    check(out, want, bound + lost)


@WAYS
def test_fp32_queries_keep_their_bits(way):
    """Two cells that a query's bits past fp16's set apart: lanes of 1 + 2^-12 meet the one's keys, lanes of 1 - 2^-13
    the other's.  Rounded to fp16 both lanes are 1 and the cells weigh the same; their scores are 0.37 apart."""
    rng = np.random.default_rng(6)
    half = np.zeros((2, 128), np.float32)
    half[0, ::2], half[1, 1::2] = 1.0, 1.0
    k = np.tile(half[:, None], (1, 2, 2))
    v = rng.standard_normal((2, 2, 256)).astype(np.float32)
    cache, pt = cache_of(k, v)
    lanes = np.where(np.arange(256) % 2 == 0, 1 + 2.0 ** -12, 1 - 2.0 ** -13).astype(np.float32)
    size = 1000.0                                          # of a score
    q = torch.from_numpy(np.tile(lanes * np.float32(size / 64 * 128 ** 0.5), (3, 16, 1))).cuda()
    q[1, :, 128:] = 0
    q[2] *= -1
    cells = all_cells(cache)
    assert np.allclose(cells[0][:2, 0, :128].cpu().numpy(), half, rtol=1e-6)
    for lam0 in (0.0, 0.7):
        heads = k8.DifferentialHeads(lambda_init=lam0)
        out = attend(way, cache, pt, q, 2, heads)
        want, _ = expected(cells, q.double(), torch.arange(2, device="cuda"), [2] * 3, None, lam0, None, 1.0)
        # (a score is 64 equal products of each of the query's two parts in at most 32 steps, each off by a unit of 2^-23 of
        # what it has reached; the cells' weights move by a quarter of what their scores move apart, in both maps)
        apart = 2 * 32 * 2.0 ** -23 * size / 4 * (1 + lam0) * (cells[1][0] - cells[1][1]).norm(dim=-1).max().item()
        off = apart + (2 * F16_HALF + 2.0 ** -16) * (1 + lam0) * cells[1].norm(dim=-1).max().item() + BF16_HALF * want.norm(dim=-1)
        check(out, want, off)
