"""attn_k8v4_diff where a unit of the tile kernel is longer than a chain of 64 tiles: O goes into the running sum, which
is rescaled when a reference moves behind it, and is added at the end."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from diff_util import all_cells, check, expected, weights

pytestmark = pytest.mark.gpu

TILE = 128


def longest_unit(n_tok, cell_tiles, H, pairs=76):
    """The range that the schedule takes for one sequence whose token tiles all see `cell_tiles`: of the cuts into equal
    ranges the one with the least rounds x (range + 8)."""
    tiles = -(-n_tok // 32)
    base = 2 * H * (n_tok // 32 + 1)
    least = -(-2 * H * tiles * cell_tiles // max(2 * pairs, 4 * pairs - base))
    cuts = {max(least, min(cell_tiles, int(np.ceil(least * (cell_tiles / least) ** (w / 31))))) for w in range(32)}
    cost = {c: -(-2 * H * tiles * -(-cell_tiles // c) // pairs) * (c + 8) for c in cuts}
    best = max(c for c in cuts if cost[c] == min(cost.values()))
    splits = -(-cell_tiles // best)
    return -(-cell_tiles // splits)


@pytest.mark.parametrize("n_tok,tiles,H,P,dtype", [(608, 200, 2, 64, "bf16"), (128, 200, 8, 16, "bf16"), (1216, 140, 1, 128, "f32"),
                                                   (608, 65, 2, 64, "bf16")])
def test_long_units(n_tok, tiles, H, P, dtype):
    """Each token's first map meets, in one cell of one tile, a key 2^11 ahead of the thousands before it (so that both
    count), its second map in another."""
    assert longest_unit(n_tok, tiles, H) == tiles
    rng = np.random.default_rng(tiles + H)
    n, HQ = tiles * TILE, 8 * H
    at = [t for t in (10, 63, 64, 70, 127, 128, 130, 191, 192, 199) if t < tiles]
    k = (0.2 * rng.standard_normal((n, H, 256))).astype(np.float32)
    v = (0.3 + 0.5 * rng.standard_normal((n, H, 256))).astype(np.float32)
    k[:, :, :10] = k[:, :, 128:138] = 0
    ahead = 11 * np.log(2) * 128 ** 0.5 / 4
    for j, t in enumerate(at):
        k[t * TILE + 17 * (j + 1) % TILE, :, [j, 128 + j]] = ahead
    pages = -(-n // P)
    cache = k8.PagedCache(pages, P, H)
    pt = torch.from_numpy(rng.permutation(pages).astype(np.int32))[None].cuda()
    k8.kv_append_k8v4(cache, pt, torch.zeros(1, dtype=torch.int64, device="cuda"), torch.from_numpy(k)[None].cuda(), torch.from_numpy(v)[None].cuda())
    q = rng.standard_normal((n_tok, HQ, 256)).astype(np.float32)
    q[:, :, :10] = q[:, :, 128:138] = 0
    lane = np.arange(n_tok) % len(at)
    q[np.arange(n_tok), :, lane] = 4.0
    q[np.arange(n_tok), :, 128 + (lane + 3) % len(at)] = 4.0
    q = torch.from_numpy(q).cuda()
    q = q if dtype == "f32" else q.bfloat16()
    heads, lam, w = weights(rng, HQ)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    k8.attn_k8v4_diff(cache, q, torch.tensor([0, n_tok], **i32), pt, torch.tensor([n], **i32), n, heads, out,
                      k8.diff_workspace(cache, 1, n_tok, n))
    assert k8.k8v4_last_device_status() == 0
    cells = all_cells(cache)
    c = np.arange(n)
    ids = torch.from_numpy(pt[0].cpu().numpy()[c // P].astype(np.int64) * P + c % P).cuda()
    pick = np.concatenate([np.arange(n_tok - len(at), n_tok), [0, 31, 32]])
    rows = torch.from_numpy(pick).cuda()
    want, bound = expected(cells, q[rows].double(), ids, n - n_tok + pick + 1, lam, 0.6, w, 0.4)
    check(out[rows], want, bound)
