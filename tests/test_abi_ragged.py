"""CPU checks of the calls of a ragged batch's step: bad arguments are refused on the host,
before any device call, and the binding checks its tensors."""
import ctypes

import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8

FAKE, ODD = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x20004)
OTHER = ctypes.c_void_p(0x90000)


@pytest.fixture(scope="module")
def L():
    k8.build()
    return k8.lib()


def _desc(**kw):
    d = dict(pages=0x10000, n_pages=4, page_size=16, n_kv_heads=2, head_dim=256, format=k8.FORMAT_K8V4)
    d.update(kw)
    return ctypes.byref(k8.k8v4_cache(ctypes.c_void_p(d["pages"]), d["n_pages"], d["page_size"], d["n_kv_heads"],
                                      d["head_dim"], d["format"]))


@pytest.mark.parametrize("bad,code", [
    (dict(P=8), k8.EINVAL), (dict(P=24), k8.EINVAL), (dict(P=8192), k8.EINVAL), (dict(n_pages=0), k8.EINVAL),
    (dict(n_pages=1 << 31), k8.EINVAL), (dict(n=-1), k8.EINVAL), (dict(n=8193), k8.EINVAL), (dict(T=-1), k8.EINVAL),
    (dict(mp=0), k8.EINVAL), (dict(mp=(1 << 27) + 1), k8.EINVAL), (dict(n=8000, mp=1 << 19), k8.EINVAL),
    (dict(free=None), k8.EINVAL), (dict(nf=None), k8.EINVAL), (dict(pt=None), k8.EINVAL), (dict(lens=None), k8.EINVAL),
    (dict(new=None), k8.EINVAL), (dict(off=None), k8.EINVAL), (dict(pos=None), k8.EINVAL), (dict(slots=None), k8.EINVAL),
    (dict(granted=None), k8.EINVAL), (dict(out=None), k8.EINVAL), (dict(nfo=None), k8.EINVAL), (dict(slots=ODD), k8.EALIGN),
    (dict(pos=ODD), k8.EALIGN), (dict(pt=ctypes.c_void_p(0x20002)), k8.EALIGN), (dict(bor=ctypes.c_void_p(0x20001)), k8.EALIGN)])
def test_plan_refuses(L, bad, code):
    a = dict(P=16, n_pages=4, free=FAKE, nf=FAKE, pt=FAKE, mp=4, lens=FAKE, new=FAKE, bor=None, n=2, T=8, off=FAKE, pos=FAKE,
             slots=FAKE, granted=FAKE, out=FAKE, nfo=FAKE)
    a.update(bad)
    assert L.kv_plan_k8v4(a["P"], a["n_pages"], a["free"], a["nf"], a["pt"], a["mp"], a["lens"], a["new"], a["bor"], a["n"],
                          a["T"], a["off"], a["pos"], a["slots"], a["granted"], a["out"], a["nfo"], None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(slots=None), k8.EINVAL), (dict(slots=ODD), k8.EALIGN), (dict(n=-1), k8.EINVAL), (dict(k=None), k8.EINVAL),
    (dict(v=None), k8.EINVAL), (dict(k=ODD), k8.EALIGN), (dict(ks=511), k8.EINVAL), (dict(vs=516), k8.EALIGN),
    (dict(dtype=2), k8.EINVAL), (dict(n=1 << 29), k8.EINVAL)])
def test_slots_refuse(L, bad, code):
    a = dict(slots=FAKE, n=4, k=FAKE, ks=512, v=FAKE, vs=512, dtype=k8.BF16)
    a.update(bad)
    call = lambda d: L.kv_append_k8v4_slots(d, a["slots"], a["n"], a["k"], a["ks"], a["v"], a["vs"], a["dtype"], None)
    assert call(_desc()) == code
    assert call(_desc(head_dim=128)) == k8.EINVAL
    assert L.kv_append_k8v4_slots(_desc(), None, 0, None, 0, None, 0, k8.BF16, None) == k8.OK


def _heads(**kw):
    d = dict(q1=0x30000, k1=0x30200, q2=0x30400, k2=0x30600, n=1, init=0.8, w=0x30800, eps=1e-6, scale=0.2)
    d.update(kw)
    return ctypes.byref(k8.k8v4_diff(d["q1"], d["k1"], d["q2"], d["k2"], d["n"], d["init"], d["w"], d["eps"], d["scale"]))


def _decode(L, cache=None, q=FAKE, dtype=k8.BF16, pt=FAKE, mp=4, lens=FAKE, n=2, max_len=64, scale=0.1, heads=None, out=OTHER,
            ws=OTHER, size=1 << 24):
    return L.attn_k8v4_diff_decode(cache or _desc(), q, dtype, pt, mp, lens, n, max_len, scale, heads or _heads(), out, ws, size, None)


def _ragged(L, cache=None, q=FAKE, dtype=k8.BF16, off=FAKE, t=5, pt=FAKE, mp=4, lens=FAKE, steps=None, n=2, max_len=64, scale=0.1,
            heads=None, out=OTHER, ws=OTHER, size=1 << 28):
    return L.attn_k8v4_diff(cache or _desc(), q, dtype, off, t, pt, mp, lens, steps, n, max_len, scale, heads or _heads(), out, ws,
                            size, None)


BAD = [(dict(q=None), k8.EINVAL), (dict(q=ODD), k8.EALIGN), (dict(dtype=7), k8.EINVAL), (dict(pt=None), k8.EINVAL),
       (dict(mp=0), k8.EINVAL), (dict(lens=None), k8.EINVAL), (dict(n=-1), k8.EINVAL), (dict(n=65536), k8.EINVAL),
       (dict(max_len=65), k8.EINVAL), (dict(max_len=-1), k8.EINVAL), (dict(scale=0.0), k8.EINVAL),
       (dict(scale=float("nan")), k8.EINVAL), (dict(scale=2e30), k8.EINVAL), (dict(out=None), k8.EINVAL), (dict(out=ODD), k8.EALIGN),
       (dict(ws=None), k8.EINVAL), (dict(ws=ODD), k8.EALIGN), (dict(heads=_heads(k1=None)), k8.EINVAL),
       (dict(heads=_heads(q2=0x30408)), k8.EALIGN), (dict(heads=_heads(n=2)), k8.EINVAL), (dict(heads=_heads(n=0)), k8.EINVAL),
       (dict(heads=_heads(init=float("nan"))), k8.EINVAL), (dict(heads=_heads(init=float("inf"))), k8.EINVAL),
       (dict(heads=_heads(scale=float("inf"))), k8.EINVAL), (dict(heads=_heads(eps=-1.0)), k8.EINVAL),
       (dict(heads=_heads(w=0x30804)), k8.EALIGN)]


@pytest.mark.parametrize("bad,code", BAD)
def test_diff_refuses(L, bad, code):
    assert _decode(L, **bad) == code and _ragged(L, **bad) == code
    for fmt in (k8.FORMAT_INT8, k8.FORMAT_Q4):
        assert _decode(L, cache=_desc(format=fmt)) == k8.EINVAL and _ragged(L, cache=_desc(format=fmt)) == k8.EINVAL
    assert L.attn_k8v4_diff_decode(_desc(), FAKE, k8.BF16, FAKE, 4, FAKE, 2, 64, 0.1, None, OTHER, OTHER, 1 << 24, None) == k8.EINVAL


@pytest.mark.parametrize("bad,code", [(dict(off=None), k8.EINVAL), (dict(off=ctypes.c_void_p(0x20002)), k8.EALIGN),
                                      (dict(t=-1), k8.EINVAL), (dict(t=1 << 24), k8.EINVAL),
                                      (dict(steps=ctypes.c_void_p(0x20001)), k8.EALIGN)])
def test_ragged_refuses(L, bad, code):
    assert _ragged(L, **bad) == code


def test_nothing_to_do(L):
    assert _decode(L, n=0, q=None) == k8.OK
    assert _ragged(L, n=0, q=None) == k8.OK and _ragged(L, t=0, q=None) == k8.OK
    # heads without vectors or a norm need neither sizes nor eps
    assert _decode(L, n=0, heads=_heads(q1=None, k1=None, q2=None, k2=None, n=0, w=None, eps=-1.0)) == k8.OK
    assert L.block_norm_k8v4(None, 0, k8.F32, 0, 64, None, None, 0, 0, None, 1.0, None, 0.0, k8.F32, None, None, None) == k8.OK


def test_workspaces(L):
    d = _desc(n_pages=1 << 16, page_size=64)
    one, more = L.attn_k8v4_diff_decode_workspace_bytes(d, 1, 100), L.attn_k8v4_diff_decode_workspace_bytes(d, 40, 30000)
    assert 0 < one < more
    assert L.attn_k8v4_diff_decode_workspace_bytes(d, -1, 10) == 0 and L.attn_k8v4_diff_decode_workspace_bytes(d, 1, -1) == 0
    assert L.attn_k8v4_diff_decode_workspace_bytes(_desc(format=k8.FORMAT_Q4), 1, 10) == 0
    a, b = L.attn_k8v4_diff_workspace_bytes(d, 1, 10, 100), L.attn_k8v4_diff_workspace_bytes(d, 4, 4000, 30000)
    assert 0 < a < b
    assert L.attn_k8v4_diff_workspace_bytes(d, 1, -1, 10) == 0 and L.attn_k8v4_diff_workspace_bytes(d, 1, 1 << 24, 10) == 0
    assert L.attn_k8v4_diff_workspace_bytes(_desc(format=k8.FORMAT_INT8), 1, 10, 100) == 0


def _norm(L, y=FAKE, ys=512, yt=k8.BF16, n=4, dim=512, post=None, gate=None, gs=512, act=0, res=None, alpha=1.0, pre=None, eps=1e-6,
          dt=k8.BF16, h=OTHER, out=None):
    return L.block_norm_k8v4(y, ys, yt, n, dim, post, gate, gs, act, res, alpha, pre, eps, dt, h, out, None)


@pytest.mark.parametrize("bad,code", [
    (dict(y=None), k8.EINVAL), (dict(h=None), k8.EINVAL), (dict(yt=2), k8.EINVAL), (dict(dt=9), k8.EINVAL), (dict(n=-1), k8.EINVAL),
    (dict(dim=0), k8.EINVAL), (dict(dim=32769, ys=40000), k8.EINVAL), (dict(ys=511), k8.EINVAL), (dict(act=3), k8.EINVAL),
    (dict(gate=ctypes.c_void_p(0x50000), gs=100), k8.EINVAL), (dict(gate=ctypes.c_void_p(0x50000), gs=-1), k8.EINVAL),
    (dict(alpha=float("nan")), k8.EINVAL), (dict(alpha=float("inf")), k8.EINVAL), (dict(post=FAKE, eps=-1.0), k8.EINVAL),
    (dict(pre=FAKE, out=ctypes.c_void_p(0x70000), eps=float("nan")), k8.EINVAL), (dict(pre=FAKE), k8.EINVAL),
    (dict(pre=FAKE, out=OTHER), k8.EINVAL), (dict(pre=OTHER, out=FAKE), k8.EINVAL), (dict(y=ctypes.c_void_p(0x20001)), k8.EALIGN),
    (dict(h=FAKE, yt=k8.F32), k8.EINVAL), (dict(h=FAKE, ys=600), k8.EINVAL), (dict(gate=OTHER), k8.EINVAL),
    (dict(res=ctypes.c_void_p(0x50001)), k8.EALIGN), (dict(post=ctypes.c_void_p(0x50002)), k8.EALIGN)])
def test_block_norm_refuses(L, bad, code):
    assert _norm(L, **bad) == code


def test_binding_checks_its_tensors(L):
    cache = k8.PagedCache(4, 16, device="cpu")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    w = lambda *s: torch.zeros(*s, dtype=torch.int64)
    plan = dict(page_size=16, free_pages=i(4), n_free=i(1), page_table=i(2, 3), seq_lens=i(2), n_new=i(2), token_offsets=i(3),
                positions=w(8), slots=w(8), granted=i(2))
    for match, change in (("free_pages", dict(free_pages=w(4))), ("n_free", dict(n_free=i(2))), ("page_table", dict(page_table=i(2))),
                          ("seq_lens", dict(seq_lens=i(3))), ("n_new", dict(n_new=w(2))), ("token_offsets", dict(token_offsets=i(2))),
                          ("positions", dict(positions=i(8))), ("slots", dict(slots=w(7))), ("granted", dict(granted=i(1))),
                          ("new_lens", dict(new_lens=i(3))), ("n_free_out", dict(n_free_out=w(1))), ("n_borrowed", dict(n_borrowed=i(3))),
                          ("CUDA tensors", {})):
        with pytest.raises(ValueError, match=match):
            k8.kv_plan_k8v4(**{**plan, **change})
    kv = torch.zeros(5, 2, 256)
    for match, args in (("one shape", (w(5), kv, kv[:4])), (r"\[n_tok, 2, 256\]", (w(5), kv[:, :1], kv[:, :1])), ("slots", (w(4), kv, kv)),
                        ("slots", (i(5), kv, kv)), ("heads must be", (w(5), torch.zeros(5, 4, 256)[:, ::2], kv)), ("CUDA tensors", (w(5), kv, kv))):
        with pytest.raises(ValueError, match=match):
            k8.kv_append_k8v4_slots(cache, *args)

    heads = k8.DifferentialHeads()
    q, out, ws = torch.zeros(2, 16, 256), torch.zeros(2, 16, 256, dtype=torch.bfloat16), torch.zeros(512, dtype=torch.uint8)
    for match, args in (("q:", (q[:, :8], i(2, 3), i(2), 32, heads, out, ws)), ("out", (q, i(2, 3), i(2), 32, heads, out.float(), ws)),
                        ("page_table", (q, i(1, 3), i(2), 32, heads, out, ws)), ("seq_lens", (q, i(2, 3), w(2), 32, heads, out, ws)),
                        ("ws", (q, i(2, 3), i(2), 32, heads, out, ws.float())), ("max_seq_len", (q, i(2, 3), i(2), -1, heads, out, ws)),
                        ("bfloat16", (q.half(), i(2, 3), i(2), 32, heads, out, ws)), ("CUDA tensors", (q, i(2, 3), i(2), 32, heads, out, ws))):
        with pytest.raises(ValueError, match=match):
            k8.attn_k8v4_diff_decode(cache, *args)
    for match, args, kw in (("token_offsets", (q, i(2), i(2, 3), i(2), 32, heads, out, ws), {}), ("page_table", (q, i(3), i(2), i(2), 32, heads, out, ws), {}),
                            ("steps", (q, i(3), i(2, 3), i(2), 32, heads, out, ws), dict(steps=i(3))),
                            ("seq_lens", (q, i(3), i(2, 3), i(1), 32, heads, out, ws), {}), ("CUDA tensors", (q, i(3), i(2, 3), i(2), 32, heads, out, ws), {})):
        with pytest.raises(ValueError, match=match):
            k8.attn_k8v4_diff(cache, *args, **kw)
    for match, kw in (("four tensors", dict(lambdas=[torch.zeros(128)] * 3)), ("four tensors", dict(lambdas=[torch.zeros(64)] * 4)),
                      ("norm_weight", dict(norm_weight=torch.zeros(128))), ("float32", dict(norm_weight=torch.zeros(256).double())),
                      ("CUDA tensors", dict(norm_weight=torch.zeros(256)))):
        with pytest.raises(ValueError, match=match):
            k8.DifferentialHeads(**kw)

    y, h, wt = torch.zeros(3, 64), torch.zeros(3, 64), torch.zeros(64)
    for match, args, kw in (("y:", (y[0], None, h), {}), ("h:", (y, None, h[:2]), {}), ("h", (y, None, torch.zeros(64, 3).T), {}),
                            ("residual", (y, y.bfloat16(), h), {}), ("residual", (y, y[:2], h), {}), ("post_weight", (y, None, h), dict(post_weight=wt[:8])),
                            ("pre_weight", (y, None, h), dict(pre_weight=wt.double())), ("normed", (y, None, h), dict(pre_weight=wt)),
                            ("gate", (y, None, h), dict(gate=y.bfloat16())), ("gate", (y, None, h), dict(gate=y[:2])),
                            ("gate", (y, None, h), dict(gate=torch.zeros(64, 3).T)), ("gate_act", (y, None, h), dict(gate=y, gate_act="relu")),
                            ("y: ", (torch.zeros(64, 3).T, None, h), {}), ("CUDA tensors", (y, None, h), dict(gate=wt))):
        with pytest.raises(ValueError, match=match):
            k8.block_norm_k8v4(*args, **kw)
