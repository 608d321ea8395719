"""Differential attention in 64 bits over a cache's bytes, with a bound of what the kernels'
stated roundings can do to each row."""
import math

import numpy as np
import torch

import quantized_paged_kv_q8_gb300 as k8

F16_HALF = torch.finfo(torch.float16).eps / 2        # 2^-11
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2      # 2^-8


def hadamard():
    i = np.arange(256)
    bits = i[:, None] & i[None, :]
    sign = np.array([bin(x).count("1") & 1 for x in range(256)])[bits]
    return torch.from_numpy((1.0 - 2.0 * sign) / 16).cuda()


HAD = None


def filled_cache(rng, n_pages, P, H, k_gain=1.0, v_gain=1.0):
    """Every cell of every page appended, keys with a few large channels."""
    cache = k8.PagedCache(n_pages, P, H)
    n = n_pages * P
    chan = np.where(rng.random((H, 256)) < 0.01, 20.0, 1.0)
    k = torch.from_numpy((k_gain * rng.standard_normal((1, n, H, 256)) * chan).astype(np.float32)).cuda()
    v = torch.from_numpy((v_gain * rng.standard_normal((1, n, H, 256))).astype(np.float32)).cuda()
    pt = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    k8.kv_append_k8v4(cache, pt, torch.zeros(1, dtype=torch.int64, device="cuda"), k, v)
    assert k8.k8v4_last_device_status() == 0
    return cache


def all_cells(cache):
    """K, and V in rotated space, of every cell, float64 [cells, H, 256], from the cache's bytes."""
    n, P, H = cache.n_pages, cache.page_size, cache.n_kv_heads
    runs = cache.pages.view(n, -1).split([256 * H * P, 8 * H * P, 128 * H * P, 16 * H * P], 1)
    kc = runs[0].contiguous().view(torch.int8).view(n * P, H, 2, 128).double()
    ks = runs[1].contiguous().view(torch.float32).view(n * P, H, 2, 1).double()
    nib = runs[2].contiguous().view(n * P, H, 8, 16)
    vs = runs[3].contiguous().view(torch.float16).view(n * P, H, 8, 1).double()
    v = (torch.cat([nib & 15, nib >> 4], -1).double() - 8) * vs
    return (kc * ks).view(n * P, H, 256), v.view(n * P, H, 256)


def weights(rng, n_lambda, init=0.6, norm=True, out_scale=0.4, spread=0.1):
    lam = [torch.from_numpy((spread * rng.standard_normal((n_lambda, 128))).astype(np.float32)).cuda() for _ in range(4)] if n_lambda else None
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(256)).astype(np.float32)).cuda() if norm else None
    return k8.DifferentialHeads(lambdas=lam, lambda_init=init, norm_weight=w, eps=1e-6, out_scale=out_scale), lam, w


def lambda_of(lam, init, HQ):
    if lam is None:
        return torch.full((HQ,), init, dtype=torch.float64, device="cuda")
    a, b, c, d = (x.double() for x in lam)
    return ((a * b).sum(-1).exp() - (c * d).sum(-1).exp() + init).expand(HQ)


def expected(cells, q, cell_ids, sees, lam, init, w, out_scale, eps=1e-6, scale=128 ** -0.5):
    """q float64 [T, HQ, 256], its sequence's cells (indices in order), cells seen by each token.
    Returns out [T, HQ, 256] and a bound of each row's error in the 2-norm.

    The bound: p and V are rounded to fp16 once each, so a map's result is off by at most 2 * 2^-11 of the sum
    of |p v| (in rotated space, where the 2-norm is that of the result); a score is a sum of 128 products accumulated
    in fp32 (each partial sum off by a unit of 2^-23 of what it has passed), which moves every p by that error
    times its size, twice with the sum below the line; 2^-16 covers the exponential, the fp32 sums over the cells
    and the joins.  The norm divides by what is left, so an error of x counts as itself and in the scale: twice.
    The result's rounding to bf16 adds 2^-8 of it."""
    global HAD
    if HAD is None:
        HAD = hadamard()
    K, V = cells[0][cell_ids], cells[1][cell_ids]
    T, HQ, _ = q.shape
    n = len(cell_ids)
    c = torch.arange(n, device="cuda")
    x = torch.zeros(T, HQ, 256, dtype=torch.float64, device="cuda")
    off = torch.zeros(T, HQ, dtype=torch.float64, device="cuda")
    lv = lambda_of(lam, init, HQ)
    sees = torch.as_tensor(sees, device="cuda")
    for h in range(HQ):
        for m in range(2):
            k = K[:, h // 8, 128 * m:128 * m + 128]
            qh = q[:, h, 128 * m:128 * m + 128]
            s = qh @ k.T * scale
            size = (qh.abs() @ k.abs().T).amax(-1) * scale if n else torch.zeros(T, dtype=torch.float64, device="cuda")
            s = s.masked_fill(c >= sees[:, None], -math.inf)
            top = s.amax(-1, keepdim=True) if n else s.sum(-1, keepdim=True)
            p = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
            p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
            o = p @ V[:, h // 8]
            absolute = (p @ V[:, h // 8].abs()).norm(dim=-1)
            f = 1.0 if m == 0 else -lv[h]
            x[:, h] += f * o
            off[:, h] += abs(f) * absolute * (2 * F16_HALF + 2.0 ** -16 + 2 * 128 * 2.0 ** -23 * size)
    x = x @ HAD
    out, bound = x, off
    if w is not None:
        norm = x.norm(dim=-1)
        # (a row near 0 is divided by sqrt(eps) at least)
        den = (norm ** 2 / 256 + eps).sqrt()
        out = x / den[..., None] * w.double()
        big = w.abs().max().item()
        bound = 2 * big * off / den
    out = out * out_scale
    return out, bound * abs(out_scale) + BF16_HALF * out.norm(dim=-1)


def check(got, want, bound):
    err = (got.double() - want).norm(dim=-1)
    assert torch.isfinite(got.double()).all()
    worst = (err - bound).max().item()
    assert worst <= 0, f"{worst:.3e} over the bound, error {err.max().item():.3e}"
