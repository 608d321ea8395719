"""block_norm_k8v4 against 64 bits: types, odd and large widths, spaced rows, gates, rows in place, parts left
out."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8

pytestmark = pytest.mark.gpu

F32_HALF = torch.finfo(torch.float32).eps / 2
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm64(x, w):
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()


def expected(y, gate, act, residual, alpha, post):
    """h in 64 bits, and what its fp32 arithmetic may be off: the mean of n squares summed in fp32 (at most n / 2 + 8
    roundings in a chain, half of it in the root; a tree of 2^5 lanes and up to 64 elements a thread leaves far fewer:
    64), four products, the gate's exponential (an argument rounded 2^-24 relative moves it by |z| of that, and 4 for the
    rest)."""
    a, rel = y.double(), 4.0
    if post is not None:
        a, rel = norm64(a, post), rel + 64
    a = a.clone()
    if gate is not None:
        z = gate.double()
        u = torch.sigmoid(z)
        a = a * {"none": z, "sigmoid": u, "silu": z * u}[act]
        rel = rel + 4 + 2 * z.abs()
    a = alpha * a
    h = a + (0 if residual is None else residual.double())
    return h, rel * F32_HALF * a.abs()


def check(y, dim, dtype, gate=None, act="none", residual=None, alpha=0.7, post=None, pre=None, in_place=False):
    n = y.shape[0]
    dt = TYPES[dtype]
    h = residual.clone() if in_place else torch.empty(n, dim, dtype=dt, device="cuda")
    normed = torch.empty(n, dim, dtype=dt, device="cuda") if pre is not None else None
    k8.block_norm_k8v4(y, h if in_place else residual, h, post_weight=post, gate=gate, gate_act=act, residual_scale=alpha,
                       pre_weight=pre, normed=normed, eps=EPS)
    want, off = expected(y, gate, act, residual, alpha, post)
    # one fp32 rounding of the sum, one to the type
    assert ((h.double() - want).abs() <= off + (half_step(dt) + 2 * F32_HALF) * (want.abs() + off) + 1e-38).all()
    if pre is not None:
        want = norm64(h.double(), pre)                     # of h as it is stored
        assert ((normed.double() - want).abs() <= (half_step(dt) + 72 * F32_HALF) * want.abs() + 1e-38).all()
    return h, normed


def rows(rng, n, dim, dtype, gain=1.0):
    return torch.from_numpy((gain * rng.standard_normal((n, dim))).astype(np.float32)).to(TYPES[dtype]).cuda()


def weight(rng, dim):
    return torch.from_numpy((1 + 0.2 * rng.standard_normal(dim)).astype(np.float32)).cuda()


@pytest.mark.parametrize("ytype,dtype", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("n,dim", [(1, 1), (3, 7), (5, 8), (9, 100), (2, 256), (130, 264), (1, 2048), (7, 4096), (33, 4099),
                                   (3, 5000), (2, 8200), (3, 16384), (2, 20001), (2, 32768)])
def test_whole(ytype, dtype, n, dim):
    rng = np.random.default_rng(n + dim)
    check(rows(rng, n, dim, ytype), dim, dtype, gate=rows(rng, n, dim, dtype, 2.0), act="sigmoid",
          residual=rows(rng, n, dim, dtype, 3.0), post=weight(rng, dim), pre=weight(rng, dim))


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("post,pre,residual,broadcast", [(0, 0, 0, 0), (1, 0, 0, 1), (0, 1, 0, 0), (0, 0, 1, 1), (1, 1, 0, 1), (0, 1, 1, 0)])
def test_parts(act, post, pre, residual, broadcast):
    rng = np.random.default_rng(3)
    n, dim = 11, 520
    gate = rows(rng, 1 if broadcast else n, dim, "bf16", 4.0)
    for g in (gate, None) + ((gate[0],) if broadcast else ()):
        check(rows(rng, n, dim, "f32"), dim, "bf16", gate=g, act=act, residual=rows(rng, n, dim, "bf16") if residual else None,
              post=weight(rng, dim) if post else None, pre=weight(rng, dim) if pre else None, alpha=-1.3)


def test_spaced_and_shifted_rows():
    """Slices of packed projections: rows of any spacing, beginning at any element."""
    rng = np.random.default_rng(4)
    for first, dim, width in ((0, 512, 1536), (8, 512, 1544), (3, 512, 1537), (1, 77, 300)):
        base, gates = rows(rng, 9, width, "bf16"), rows(rng, 9, width, "bf16")
        check(base[:, first:first + dim], dim, "bf16", gate=gates[:, width - dim:], act="silu",
              residual=rows(rng, 9, dim, "bf16"), post=weight(rng, dim), pre=weight(rng, dim))


@pytest.mark.parametrize("dim", [72, 4097, 24000])
def test_in_place(dim):
    rng = np.random.default_rng(5)
    y, res, post, pre = rows(rng, 6, dim, "bf16"), rows(rng, 6, dim, "bf16"), weight(rng, dim), weight(rng, dim)
    a = check(y, dim, "bf16", residual=res, post=post, pre=pre)
    b = check(y, dim, "bf16", residual=res, post=post, pre=pre, in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    z = y.clone()                                          # over its own input
    k8.block_norm_k8v4(z, res, z, post_weight=post, residual_scale=0.7, eps=EPS)
    assert torch.equal(z, a[0])


def test_rows_of_zeros_and_infinities():
    rng = np.random.default_rng(6)
    y, w = rows(rng, 4, 640, "f32"), weight(rng, 640)
    y[0] = 0
    y[1, 5] = float("inf")
    y[2, 7] = float("nan")
    h, normed = torch.empty(4, 640, device="cuda"), torch.empty(4, 640, device="cuda")
    k8.block_norm_k8v4(y, None, h, post_weight=w, pre_weight=w, normed=normed, eps=EPS)
    assert (h[0] == 0).all() and (normed[0] == 0).all()
    assert torch.isnan(h[1, 5]) and torch.isnan(h[2]).all() and torch.isfinite(h[3]).all()
    # a gate far below 0 closes, far above leaves the value
    g = torch.full((4, 640), -200.0, device="cuda")
    g[3] = 200.0
    y = rows(rng, 4, 640, "f32")
    for act, top in (("sigmoid", 1.0), ("silu", 200.0)):
        k8.block_norm_k8v4(y, None, h, gate=g, gate_act=act)
        assert (h[:3].abs() <= 1e-30).all() and torch.allclose(h[3], top * y[3], rtol=1e-6)


def test_many_rows():
    rng = np.random.default_rng(7)
    check(rows(rng, 70001, 64, "bf16"), 64, "bf16", residual=rows(rng, 70001, 64, "bf16"), post=weight(rng, 64), pre=weight(rng, 64))
