"""CPU checks of the calls around the attention: bad arguments are refused on the
host, before any device call, and the binding checks its tensors."""
import ctypes

import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8

FAKE = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x20004)


@pytest.fixture(scope="module")
def L():
    k8.build()
    return k8.lib()


def _desc(**kw):
    d = dict(pages=0x10000, n_pages=4, page_size=16, n_kv_heads=2, head_dim=256, format=k8.FORMAT_K8V4)
    d.update(kw)
    return ctypes.byref(k8.k8v4_cache(ctypes.c_void_p(d["pages"]), d["n_pages"], d["page_size"], d["n_kv_heads"],
                                      d["head_dim"], d["format"]))


def _rope(table=0x40000, n_pos=64, rot=64, inter=0):
    return ctypes.byref(k8.k8v4_rope(ctypes.c_void_p(table), n_pos, rot, inter))


BAD_ROPES = [(None, k8.EINVAL), (_rope(table=0), k8.EINVAL), (_rope(n_pos=0), k8.EINVAL), (_rope(rot=0), k8.EINVAL),
             (_rope(rot=24), k8.EINVAL), (_rope(rot=272), k8.EINVAL), (_rope(table=0x40008), k8.EALIGN)]


def _norm_rope(L, q=FAKE, qs=4096, hq=16, k=FAKE, ks=512, hk=2, dtype=k8.BF16, qw=None, kw=None, eps=1e-6, pos=FAKE,
               n=1, t=1, rope=None, qo=ctypes.c_void_p(0x90000), ko=ctypes.c_void_p(0xa0000)):
    return L.qk_norm_rope_k8v4(q, qs, hq, k, ks, hk, dtype, qw, kw, eps, pos, n, t, rope or _rope(), qo, ko, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=5), k8.EINVAL), (dict(hq=-1), k8.EINVAL), (dict(hq=0, hk=0), k8.EINVAL), (dict(hq=2000), k8.EINVAL),
    (dict(qs=4095), k8.EINVAL), (dict(qs=4100), k8.EALIGN), (dict(ks=511), k8.EINVAL), (dict(q=None), k8.EINVAL),
    (dict(q=ODD), k8.EALIGN), (dict(k=None), k8.EINVAL), (dict(pos=None), k8.EINVAL), (dict(pos=ODD), k8.EALIGN),
    (dict(qo=None), k8.EINVAL), (dict(ko=None), k8.EINVAL), (dict(qo=ODD), k8.EALIGN), (dict(qw=ODD), k8.EALIGN),
    (dict(kw=FAKE, eps=-1.0), k8.EINVAL), (dict(kw=FAKE, eps=float("nan")), k8.EINVAL), (dict(n=-1), k8.EINVAL),
    (dict(t=-1), k8.EINVAL), (dict(n=1 << 20, t=1 << 20), k8.EINVAL), (dict(qs=8192, qo=FAKE), k8.EINVAL)])
def test_norm_rope_refuses(L, bad, code):
    assert _norm_rope(L, **bad) == code


@pytest.mark.parametrize("rope,code", BAD_ROPES)
def test_bad_tables_refused(L, rope, code):
    assert L.qk_norm_rope_k8v4(FAKE, 4096, 16, FAKE, 512, 2, k8.BF16, None, None, 0.0, FAKE, 1, 1, rope, FAKE, FAKE, None) == code
    assert L.kv_append_k8v4_rope(_desc(), FAKE, 4, 1, FAKE, 1, FAKE, 512, FAKE, 512, k8.BF16, None, 0.0, rope, None) == code


def test_nothing_to_do(L):
    assert _norm_rope(L, n=0) == k8.OK and _norm_rope(L, t=0) == k8.OK
    assert L.kv_append_k8v4_rope(_desc(), FAKE, 4, 1, FAKE, 0, FAKE, 512, FAKE, 512, k8.BF16, None, 0.0, _rope(), None) == k8.OK
    assert L.spec_accept_k8v4(None, None, k8.F32, None, None, None, None, 0, 4, 100, None, None, None) == k8.OK


@pytest.mark.parametrize("bad,code", [
    (dict(k=None), k8.EINVAL), (dict(v=None), k8.EINVAL), (dict(k=ODD), k8.EALIGN), (dict(ks=511), k8.EINVAL),
    (dict(vs=516), k8.EALIGN), (dict(pos=None), k8.EINVAL), (dict(pos=ODD), k8.EALIGN), (dict(dtype=2), k8.EINVAL),
    (dict(n=-1), k8.EINVAL), (dict(pt=None), k8.EINVAL), (dict(mp=0), k8.EINVAL), (dict(w=ODD), k8.EALIGN),
    (dict(w=FAKE, eps=-1.0), k8.EINVAL), (dict(n=1 << 15, t=1 << 15), k8.EINVAL)])
def test_append_rope_refuses(L, bad, code):
    a = dict(pt=FAKE, mp=4, n=1, pos=FAKE, t=1, k=FAKE, ks=512, v=FAKE, vs=512, dtype=k8.BF16, w=None, eps=1e-6)
    a.update(bad)
    assert L.kv_append_k8v4_rope(_desc(), a["pt"], a["mp"], a["n"], a["pos"], a["t"], a["k"], a["ks"], a["v"], a["vs"],
                                 a["dtype"], a["w"], a["eps"], _rope(), None) == code
    assert L.kv_append_k8v4_rope(_desc(head_dim=128), FAKE, 4, 1, FAKE, 1, FAKE, 512, FAKE, 512, k8.BF16, None, 0.0,
                                 _rope(), None) == k8.EINVAL


@pytest.mark.parametrize("bad,code", [
    (dict(p=None), k8.EINVAL), (dict(dtype=9), k8.EINVAL), (dict(drafts=None), k8.EINVAL), (dict(u=None), k8.EINVAL),
    (dict(us=None), k8.EINVAL), (dict(out=None), k8.EINVAL), (dict(acc=None), k8.EINVAL), (dict(n=33), k8.EINVAL),
    (dict(n=-1), k8.EINVAL), (dict(vocab=0), k8.EINVAL), (dict(vocab=(1 << 24) + 1), k8.EINVAL), (dict(b=-1), k8.EINVAL),
    (dict(p=ctypes.c_void_p(0x20002)), k8.EALIGN), (dict(out=ctypes.c_void_p(0x20002)), k8.EALIGN)])
def test_accept_refuses(L, bad, code):
    a = dict(p=FAKE, q=FAKE, dtype=k8.F32, drafts=FAKE, nd=None, u=FAKE, us=FAKE, b=1, n=4, vocab=100, out=FAKE, acc=FAKE)
    a.update(bad)
    assert L.spec_accept_k8v4(a["p"], a["q"], a["dtype"], a["drafts"], a["nd"], a["u"], a["us"], a["b"], a["n"],
                              a["vocab"], a["out"], a["acc"], None) == code


def test_binding_checks_its_tensors(L):
    """Shapes, types, spacing and devices are checked before the library is called (CPU tensors suffice: the last
    check refuses them)."""
    q = torch.zeros(2, 3, 16, 256, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int64)
    tab = torch.zeros(8, 64)

    def norm_rope(match, q=q, k=None, pos=pos, tab=tab, qo=None, ko=None, **kw):
        with pytest.raises(ValueError, match=match):
            k8.qk_norm_rope_k8v4(q, k, pos, tab, torch.empty(q.shape, dtype=q.dtype) if qo is None else qo, ko, **kw)

    norm_rope("256", q=q[:, :, :, :128])
    norm_rope("n_tok", q=q[0])
    norm_rope("bfloat16", q=q.half())
    norm_rope("heads must be contiguous", q=q[:, :, ::2])
    norm_rope("evenly spaced", q=q[:, :2])
    norm_rope("shape of q", qo=q[:, :2])
    norm_rope("q_out", qo=torch.empty(2, 16, 3, 256, dtype=q.dtype).transpose(1, 2))
    norm_rope("q_out", qo=torch.empty(q.shape))
    norm_rope("pos", pos=pos.int())
    norm_rope("pos", pos=pos[:1])
    norm_rope("rope_table", tab=tab.double())
    norm_rope("rope_table", tab=tab[:, ::2])
    norm_rope("tokens of q", k=q[:, :2], ko=q[:, :2])
    norm_rope("k_out", k=q, ko=q[:, :2])
    norm_rope("q_weight", q_weight=torch.zeros(255))
    norm_rope("k_weight", k_weight=torch.zeros(256, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="q: a tensor"):
        k8.qk_norm_rope_k8v4(None, None, pos, tab, q, None)
    # heads of a packed projection's tokens are fine: what is left to refuse is the CPU
    packed = torch.zeros(2, 3, 20, 256)
    norm_rope("CUDA tensors", q=packed[:, :, :16], k=packed[:, :, 16:18], ko=torch.empty(2, 3, 2, 256))

    cache = k8.PagedCache(4, 16, device="cpu")
    kv, pt = torch.zeros(2, 3, 2, 256), torch.zeros(2, 4, dtype=torch.int32)
    for match, args in (("one shape", (pt, pos, kv, kv[:1], tab)), (r"\[n_seqs, n_tok, 2, 256\]", (pt, pos, kv[:, :, :1], kv[:, :, :1], tab)),
                        ("page_table", (pt[:1], pos, kv, kv, tab)), ("page_table", (pt.long(), pos, kv, kv, tab)),
                        ("pos", (pt, pos[:1], kv, kv, tab)), ("rope_table", (pt, pos, kv, kv, tab.half())),
                        ("CUDA tensors", (pt, pos, kv, kv, tab))):
        with pytest.raises(ValueError, match=match):
            k8.kv_append_k8v4_rope(cache, *args)

    q1, out, lens, ws = torch.zeros(2, 16, 256), torch.zeros(2, 16, 256), torch.zeros(2, dtype=torch.int32), torch.zeros(512, dtype=torch.uint8)
    for match, args in (("q:", (q1[:, :8], pt, lens, 64, 64, out, ws)), ("page_table", (q1, pt[:1], lens, 64, 64, out, ws)),
                        ("seq_lens", (q1, pt, lens.long(), 64, 64, out, ws)), ("out", (q1, pt, lens, 64, 64, out[:1], ws)),
                        ("ws", (q1, pt, lens, 64, 64, out, ws.float())), ("max_seq_len", (q1, pt, lens, -1, 64, out, ws)),
                        ("CUDA tensors", (q1, pt, lens, 64, 64, out, ws))):
        with pytest.raises(ValueError, match=match):
            k8.attn_k8v4_decode_shared(cache, *args)

    p, d, tok = torch.zeros(2, 3, 50), torch.zeros(2, 2, 50), torch.zeros(2, 2, dtype=torch.int32)
    u, us, o, acc = torch.zeros(2, 2), torch.zeros(2), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for match, args in (("target_probs", (p[0], d, tok, u, us, o, acc)), ("draft_probs", (p, d[:, :, :49], tok, u, us, o, acc)),
                        ("draft_probs", (p, d.bfloat16(), tok, u, us, o, acc)), ("draft_tokens", (p, d, tok.long(), u, us, o, acc)),
                        ("u_accept", (p, d, tok, u.double(), us, o, acc)), ("u_sample", (p, d, tok, u, us[:1], o, acc)),
                        ("tokens", (p, d, tok, u, us, o[:, :2], acc)), ("n_accepted", (p, d, tok, u, us, o, acc.long())),
                        ("CUDA tensors", (p, d, tok, u, us, o, acc))):
        with pytest.raises(ValueError, match=match):
            k8.spec_accept_k8v4(*args)
    with pytest.raises(ValueError, match="n_drafts"):
        k8.spec_accept_k8v4(p, d, tok, u, us, o, acc, n_drafts=acc.long())


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), k8.EINVAL), (dict(q=ODD), k8.EALIGN), (dict(dtype=k8.F32), k8.EINVAL), (dict(pt=None), k8.EINVAL),
    (dict(mp=0), k8.EINVAL), (dict(lens=None), k8.EINVAL), (dict(n=-1), k8.EINVAL), (dict(n=65536), k8.EINVAL),
    (dict(max_len=65), k8.EINVAL), (dict(shared=-1), k8.EINVAL), (dict(scale=0.0), k8.EINVAL),
    (dict(scale=float("nan")), k8.EINVAL), (dict(out=None), k8.EINVAL), (dict(out=ODD), k8.EALIGN),
    (dict(ws=None), k8.EINVAL), (dict(ws=ODD), k8.EALIGN)])
def test_decode_shared_refuses(L, bad, code):
    a = dict(q=FAKE, dtype=k8.BF16, pt=FAKE, mp=4, lens=FAKE, n=4, max_len=64, shared=64, scale=0.0625, out=FAKE, ws=FAKE)
    a.update(bad)
    call = lambda d: L.attn_k8v4_decode_shared(d, a["q"], a["dtype"], a["pt"], a["mp"], a["lens"], a["n"], a["max_len"],
                                               a["shared"], a["scale"], a["out"], a["ws"], 1 << 24, None)
    assert call(_desc()) == code
    for fmt in (k8.FORMAT_INT8, k8.FORMAT_Q4):
        assert call(_desc(format=fmt)) == k8.EINVAL


def test_decode_shared_workspace(L):
    d = _desc(n_pages=1 << 20, page_size=64)
    size = L.attn_k8v4_shared_workspace_bytes
    assert size(d, 32, 32768, 34101) > size(d, 16, 32768, 34101) > 0
    for n, shared in ((32, 0), (3, 100000), (8, 4096), (128, 63)):     # the per-sequence decode's
        assert size(d, n, shared, shared + 1000) == L.attn_k8v4_workspace_bytes(d, n, 1, shared + 1000)
    assert size(_desc(format=k8.FORMAT_Q4), 32, 64, 64) == 0 and size(d, -1, 64, 64) == 0 and size(d, 4, -1, 64) == 0
    assert L.attn_k8v4_decode_shared(d, None, k8.BF16, FAKE, 4, None, 0, 64, 64, 0.0625, None, None, 0, None) == k8.OK
