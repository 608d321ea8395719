"""Operators of a serving step around the quantized paged KV cache, as cases that can be timed and compared:
their plain forms in elementary torch operations, the library's own calls, and their definitions in 64 bits.

    norm_rope      per-head RMS norm of queries and keys and the position rotation, in one pass
    append_rope    keys rotated by their position on the way into the paged cache (with their values)
    shared_decode  decode attention of a batch whose sequences share a long prefix, the prefix read once for all
    spec_accept    drafted tokens accepted or replaced from the target's probabilities and given random numbers

`own` says which of the two forms run() takes.  Geometry everywhere: head_dim 256, 8 query heads per KV head,
2 KV heads (the cache's own)."""
import math

import torch

own = False

D = 256            # head_dim
H = 2              # KV heads
HQ = 16            # query heads
BASE = 1.0e6       # base of the rotation's angles
EPS = 1.0e-6
FORMATS = {"int8": 1, "q4": 2, "k8v4": 3}
CELL_HEAD = {"int8": 528, "q4": 288, "k8v4": 408}       # bytes of one cell of one head


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token of one long conversation: nothing but latency
        dict(name="norm_rope 1x1", op="norm_rope", seqs=1, tok=1, start=237567, rot=64, dtype="bf16", norm=True,
             inter=False, packed=True),
        # a verify step, 8 sequences of 4 drafts + 1, whole heads rotated in adjacent pairs, no norm
        dict(name="norm_rope 8x5", op="norm_rope", seqs=8, tok=5, start=65530, rot=256, dtype="f32", norm=False,
             inter=True, packed=False),
        # a prompt chunk of 8,192 tokens at offset 229,376, taken out of the packed projection
        dict(name="norm_rope 1x8192", op="norm_rope", seqs=1, tok=8192, start=229376, rot=64, dtype="bf16", norm=True,
             inter=False, packed=True),
        # the append of a decode step of 32 sequences
        dict(name="append_rope 32x1", op="append_rope", seqs=32, tok=1, start=8192, rot=64, dtype="bf16", inter=False,
             packed=True, P=16, fmt="k8v4"),
        # 1,024 fp32 cells, 16-cell pages: the tiny round trip
        dict(name="append_rope 1x1024", op="append_rope", seqs=1, tok=1024, start=0, rot=256, dtype="f32", inter=False,
             packed=False, P=16, fmt="k8v4"),
        # a prompt of 32,768 tokens, written from the middle of a page
        dict(name="append_rope 1x32768", op="append_rope", seqs=1, tok=32768, start=1001, rot=256, dtype="bf16",
             inter=False, packed=True, P=64, fmt="k8v4"),
        # 8 short chats behind one system prompt of 1,000 cells
        dict(name="shared_decode 8x1000", op="shared_decode", seqs=8, shared=1000, own_max=40, P=16, short=False),
        # 32 requests on one document of 32,768 cells, up to 1,333 cells of their own
        dict(name="shared_decode 32x32768", op="shared_decode", seqs=32, shared=32768, own_max=1333, P=64, short=False),
        # 128 samples of one context of 118,784 cells, a few of them cut inside it
        dict(name="shared_decode 128x118784", op="shared_decode", seqs=128, shared=118784, own_max=512, P=64,
             short=True),
        # one sequence, 4 drafts
        dict(name="spec_accept 1x4", op="spec_accept", seqs=1, drafts=4, vocab=32768, dtype="f32", sure=False,
             ragged=False),
        # the verify batch (8 sequences, 4 drafts + 1), an odd vocabulary, drafts from a table rather than a model
        dict(name="spec_accept 8x4", op="spec_accept", seqs=8, drafts=4, vocab=131071, dtype="f32", sure=True,
             ragged=True),
        # 64 sequences of up to 7 drafts
        dict(name="spec_accept 64x7", op="spec_accept", seqs=64, drafts=7, vocab=262144, dtype="f32", sure=False,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append_rope", "shared_decode", "spec_accept"])
    if op == "norm_rope":
        tok = _log(rng, 1, 8192)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(64, 8192 // tok))), tok=tok, start=rng.randrange(0, 200000),
                    rot=16 * rng.randint(1, 16), dtype=rng.choice(["bf16", "f32"]), norm=rng.random() < 0.7,
                    inter=rng.random() < 0.4, packed=rng.random() < 0.6)
    if op == "append_rope":
        dtype = rng.choice(["bf16", "f32"])
        tok = _log(rng, 1, 30000)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(64, 30000 // tok))), tok=tok, start=rng.randrange(0, 200000),
                    rot=16 * rng.randint(1, 16), dtype=dtype, inter=rng.random() < 0.4, packed=rng.random() < 0.6,
                    P=rng.choice([16, 48, 64]), fmt=rng.choice(["k8v4", "k8v4", "int8", "q4"]))
    if op == "shared_decode":
        seqs = _log(rng, 1, 128)
        shared = _log(rng, 16, min(118784, 118784 * 100 // seqs))
        return dict(op=op, seqs=seqs, shared=shared, own_max=_log(rng, 1, 2000), P=rng.choice([16, 48, 64, 128]),
                    short=rng.random() < 0.5)
    return dict(op=op, seqs=_log(rng, 1, 60), drafts=rng.randint(1, 7), vocab=_log(rng, 1000, 262144),
                dtype=rng.choice(["f32", "bf16"]), sure=rng.random() < 0.3, ragged=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _channels(g, heads, share=0.01, gain=20.0):
    """Per-head channel factors: one channel in a hundred is 20 times as large, as keys have them."""
    return torch.where(torch.rand(heads, D, generator=g, device="cuda") < share, gain, 1.0)


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _rope_table(rows, rot):
    """fp32 [rows, rot]: the cosines of a position's rot / 2 angles, then their sines, each angle taken in 64 bits."""
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * BASE ** (-2.0 * j / rot)
    return torch.cat([angle.cos(), angle.sin()], -1).float()


def _rows(g, case, heads):
    """What the projection leaves: [seqs, tok, heads_i, 256] for each i, slices of one buffer where `packed`."""
    B, T, dt = case["seqs"], case["tok"], _dtype(case["dtype"])
    if case["packed"]:
        flat = _normal(g, B, T, sum(heads), D).to(dt)
        flat[:, :, heads[0]:heads[0] + H] = (flat[:, :, heads[0]:heads[0] + H] * _channels(g, H)).to(dt)
        return list(flat.split(heads, 2))
    return [(_normal(g, B, T, n, D) * (_channels(g, n) if n == H else 1.0)).to(dt).contiguous() for n in heads]


def _int8_half(x):
    """fp32 [..., 256] -> int8 codes and the two fp32 scales of the 128-lane halves."""
    x = x.unflatten(-1, (2, 128))
    s = x.abs().amax(-1) / torch.full((1,), 127.0, device=x.device)
    c = torch.where(s[..., None] > 0, x / torch.where(s > 0, s, 1.0)[..., None], 0.0).round().clamp(-127, 127)
    return c.flatten(-2), s


def _q4(y):
    """fp32 [..., 256] (rotated space) -> codes 0..15 and the eight fp16 scales of the 32-blocks."""
    y = y.unflatten(-1, (8, 32))
    m = y.gather(-1, y.abs().argmax(-1, keepdim=True))
    d = (m * -0.125).half().float()
    c = torch.where(d != 0, (y / torch.where(d != 0, d, 1.0)).round() + 8, 8.0).clamp(0, 15)
    return c.flatten(-2), d[..., 0].half()


def _nibbles(c):
    c = c.to(torch.uint8).unflatten(-1, (8, 2, 16))
    return (c[..., 0, :] | (c[..., 1, :] << 4)).flatten(-2)


def _bytes(pages, *runs):
    return torch.cat([r.contiguous().view(torch.uint8).reshape(pages, -1) for r in runs], 1).reshape(-1)


def _cache_bytes(g, fmt, pages, P):
    """A filled cache: keys with large channels, values as they are after their rotation (normal)."""
    k = _normal(g, pages, P, H, D) * _channels(g, H)
    v = _normal(g, pages, P, H, D)
    if fmt == "k8v4":
        (kc, ks), (vc, vs) = _int8_half(k), _q4(v)
        return _bytes(pages, kc.to(torch.int8), ks, _nibbles(vc), vs)
    if fmt == "int8":
        (kc, ks), (vc, vs) = _int8_half(k), _int8_half(v)
        return _bytes(pages, kc.to(torch.int8), ks, vc.to(torch.int8), vs)
    (kc, ks), (vc, vs) = _q4(k), _q4(v)
    return _bytes(pages, _nibbles(kc), ks, _nibbles(vc), vs)


def _handle(state, case, fmt, pages, P):
    """The cache descriptor a program makes once, over the bytes that the state holds."""
    import quantized_paged_kv_q8_gb300 as k8
    state["cache"] = k8.PagedCache(pages, P, H, FORMATS[fmt], pages=state["pages"])


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "norm_rope":
        q, k = _rows(g, case, [HQ, H, H])[:2] if case["packed"] else _rows(g, case, [HQ, H])
        pos = case["start"] + torch.randint(0, 50, (case["seqs"],), generator=g, device="cuda")
        s = dict(case=case, q=q, k=k, pos=pos, table=_rope_table(case["start"] + 50 + case["tok"], case["rot"]),
                 qw=1.0 + 0.2 * _normal(g, D) if case["norm"] else None,
                 kw=1.0 + 0.2 * _normal(g, D) if case["norm"] else None)
        s["q_out"] = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        s["k_out"] = torch.empty(k.shape, dtype=k.dtype, device="cuda")
        return s
    if case["op"] == "append_rope":
        B, T, P, fmt = case["seqs"], case["tok"], case["P"], case["fmt"]
        k, v = _rows(g, case, [HQ, H, H])[1:] if case["packed"] else _rows(g, case, [H, H])
        pos = case["start"] + torch.randint(0, P, (B,), generator=g, device="cuda")
        each = (2 * P - 2 + T) // P + 1                    # pages a sequence's new cells can touch
        pages = B * each
        first = case["start"] // P
        table = torch.zeros(B, first + each, dtype=torch.int32, device="cuda")
        table[:, first:] = torch.randperm(pages, generator=g, device="cuda").reshape(B, each).int()
        s = dict(case=case, k=k, v=v, pos=pos, page_table=table, pages=_cache_bytes(g, fmt, pages, P),
                 table=_rope_table(case["start"] + P + T, case["rot"]), n_pages=pages,
                 every=torch.arange(pages, dtype=torch.int32, device="cuda"),
                 k_hat=torch.empty(pages * P, H, D, device="cuda"), v_hat=torch.empty(pages * P, H, D, device="cuda"))
        if own:
            _handle(s, case, fmt, pages, P)
        return s
    if case["op"] == "shared_decode":
        B, P, shared = case["seqs"], case["P"], case["shared"]
        n_sh = -(-shared // P)
        each = -(-(shared + case["own_max"]) // P) - shared // P   # pages from the last shared one on
        pages = n_sh + B * each
        q = (_normal(g, B, HQ, D)).to(torch.bfloat16)
        ids = torch.randperm(pages, generator=g, device="cuda").int()
        table = torch.empty(B, shared // P + each, dtype=torch.int32, device="cuda")
        table[:, :shared // P] = ids[:shared // P]
        table[:, shared // P:] = ids[n_sh:].reshape(B, each)
        pages_b = _cache_bytes(g, "k8v4", pages, P)
        if shared % P:                                     # the page the prefix ends in is each sequence's own copy
            by_page = pages_b.view(pages, -1)
            by_page[table[:, shared // P].long()] = by_page[ids[n_sh - 1].long()].clone()
        lens = shared + torch.randint(1, case["own_max"] + 1, (B,), generator=g, device="cuda")
        lens[0] = shared + case["own_max"]
        if case["short"] and B > 2:                        # sequences that end inside the prefix, one of them empty
            lens[1] = torch.randint(1, shared + 1, (1,), generator=g, device="cuda")[0]
            lens[2] = 0
        s = dict(case=case, q=q, page_table=table, lens=lens.int(), pages=pages_b, n_pages=pages,
                 max_len=shared + case["own_max"], out=torch.empty(B, HQ, D, device="cuda"))
        if own:
            import quantized_paged_kv_q8_gb300 as k8
            _handle(s, case, "k8v4", pages, P)
            s["ws"] = k8.shared_workspace(s["cache"], B, shared, s["max_len"])
        return s
    B, n, V, dt = case["seqs"], case["drafts"], case["vocab"], _dtype(case["dtype"])
    logits = 3.0 * _normal(g, B, n + 1, V)
    p = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :n] + 0.7 * _normal(g, B, n, V), -1)
    cum = draft.cumsum(-1)
    at = torch.rand(B, n, 1, generator=g, device="cuda") * cum[..., -1:]
    tokens = torch.searchsorted(cum, at).clamp(max=V - 1)[..., 0].int()
    if case["sure"]:
        # a table proposes the target's likeliest token most of the time
        tokens = torch.where(torch.rand(B, n, generator=g, device="cuda") < 0.8, p[:, :n].argmax(-1).int(), tokens)
    count = torch.randint(0, n + 1, (B,), generator=g, device="cuda") if case["ragged"] else torch.full((B,), n, device="cuda")
    return dict(case=case, p=p.to(dt), q=None if case["sure"] else draft.to(dt), tokens=tokens, count=count.int(),
                u=torch.rand(B, n, generator=g, device="cuda"), us=torch.rand(B, generator=g, device="cuda"),
                out=torch.empty(B, n + 1, dtype=torch.int32, device="cuda"),
                accepted=torch.empty(B, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    import quantized_paged_kv_q8_gb300 as k8
    case = s["case"]
    if case["op"] == "norm_rope":
        k8.qk_norm_rope_k8v4(s["q"], s["k"], s["pos"], s["table"], s["q_out"], s["k_out"], q_weight=s["qw"],
                             k_weight=s["kw"], eps=EPS, interleaved=case["inter"])
        return s["q_out"], s["k_out"]
    if case["op"] == "append_rope":
        k8.kv_append_k8v4_rope(s["cache"], s["page_table"], s["pos"], s["k"], s["v"], s["table"],
                               interleaved=case["inter"])
        # the updated pages, as the values that the codes stand for
        k8.kv_dequant_k8v4(s["cache"], s["every"], 0, s["n_pages"] * case["P"], s["k_hat"], s["v_hat"])
        return s["k_hat"], s["v_hat"]
    if case["op"] == "shared_decode":
        return k8.attn_k8v4_decode_shared(s["cache"], s["q"], s["page_table"], s["lens"], s["max_len"], case["shared"],
                                          s["out"], s["ws"])
    k8.spec_accept_k8v4(s["p"], s["q"], s["tokens"], s["u"], s["us"], s["out"], s["accepted"], n_drafts=s["count"])
    return s["out"], s["accepted"]


# ---------------------------------------------------------------- the plain forms
def _rotated(x, cos, sin, rot, inter):
    """x: 64 bits [B, T, heads, 256]; cos, sin: [B, T, 1, rot / 2]."""
    a = x[..., :rot].unflatten(-1, (rot // 2, 2) if inter else (2, rot // 2)).movedim(-1 if inter else -2, 0)
    y = torch.stack([a[0] * cos - a[1] * sin, a[1] * cos + a[0] * sin], -1 if inter else -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _angles(s):
    pos = s["pos"][:, None] + torch.arange(s["case"]["tok"], device="cuda")
    return s["table"][pos].double()[:, :, None].chunk(2, -1)


def _hadamard():
    i = torch.arange(D, device="cuda")
    bits = i[:, None] & i[None, :]
    bits = bits ^ (bits >> 4)
    bits = bits ^ (bits >> 2)
    return (1 - 2 * ((bits ^ (bits >> 1)) & 1)).double() / 16


def _plain_norm_rope(s):
    case = s["case"]
    cos, sin = _angles(s)

    def one(x, w):
        y = x.double()
        if w is not None:
            y = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        return _rotated(y, cos, sin, case["rot"], case["inter"]).float().to(x.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _q4_values(nib, scales):
    """bytes [n, 128] and fp16 [n, 8] -> fp32 [n, 256]"""
    b = nib.unflatten(-1, (8, 16))
    c = torch.stack([b & 15, b >> 4], -2).flatten(-2).float() - 8
    return (c * scales.float()[..., None]).flatten(-2)


def _int8_values(codes, scales):
    return (codes.float().unflatten(-1, (2, 128)) * scales[..., None]).flatten(-2)


def _runs(pages, fmt, n, P):
    """The four runs of every page: codes and scales of K, then of V, as [n, P, H, ...]."""
    wk, wks, wv, wvs = {"k8v4": (256, 8, 128, 16), "int8": (256, 8, 256, 8), "q4": (128, 16, 128, 16)}[fmt]
    runs = pages.view(n, P * H * CELL_HEAD[fmt]).split([P * H * w for w in (wk, wks, wv, wvs)], 1)
    runs = [r.contiguous() for r in runs]
    k, v = (r.view(torch.int8 if w == 256 else torch.uint8).view(n, P, H, w) for r, w in ((runs[0], wk), (runs[2], wv)))
    ks, vs = (r.view(torch.float32 if w == 8 else torch.float16).view(n, P, H, -1) for r, w in ((runs[1], wks), (runs[3], wvs)))
    return k, ks, v, vs


def _unrotated(x):
    return (x.double() @ _hadamard()).float()


def _values(pages, fmt, n, P):
    """K (un-rotated) and V (rotated space) of every cell, fp32 [n * P, H, 256]."""
    k, ks, v, vs = _runs(pages, fmt, n, P)
    k = _unrotated(_q4_values(k, ks)) if fmt == "q4" else _int8_values(k, ks)
    v = _int8_values(v, vs) if fmt == "int8" else _q4_values(v, vs)
    return k.reshape(n * P, H, D), v.reshape(n * P, H, D)


def _plain_append_rope(s):
    case = s["case"]
    fmt, P = case["fmt"], case["P"]
    cos, sin = _angles(s)
    # rotated in 64 bits (a code next to a border goes by the last bit), rounded once to K's type
    k = _rotated(s["k"].double(), cos, sin, case["rot"], case["inter"]).float().to(s["k"].dtype).float()
    v = s["v"].float()
    if fmt == "q4":
        c, d = _q4(_unrotated(k))
        k = _unrotated((((c - 8).unflatten(-1, (8, 32))) * d.float()[..., None]).flatten(-2))
    else:
        k = _int8_values(*_int8_half(k))
    if fmt == "int8":
        v = _int8_values(*_int8_half(v))
    else:
        c, d = _q4(_unrotated(v))
        v = ((c - 8).unflatten(-1, (8, 32)) * d.float()[..., None]).flatten(-2)
    k_hat, v_hat = _values(s["pages"], fmt, s["n_pages"], P)
    cell = s["pos"][:, None] + torch.arange(case["tok"], device="cuda")
    at = s["page_table"].gather(1, cell // P).long() * P + cell % P
    k_hat[at] = k
    v_hat[at] = v
    return k_hat, v_hat


def _plain_shared_decode(s):
    case = s["case"]
    B, P, shared = case["seqs"], case["P"], case["shared"]
    lens = s["lens"].long()
    k, ks, v, vs = (r.flatten(0, 1) for r in _runs(s["pages"], "k8v4", s["n_pages"], P))

    def cells(table, idx):
        at = table.gather(-1, idx // P).long() * P + idx % P
        return _int8_values(k[at], ks[at]), _q4_values(v[at], vs[at])

    # the prefix, through the first sequence's table, for all rows; each sequence's own cells for its own
    idx = torch.arange(shared, device="cuda")
    kp, vp = cells(s["page_table"][0], idx)
    mine = shared + torch.arange(case["own_max"], device="cuda").expand(B, -1)
    ko, vo = cells(s["page_table"], mine)
    q = s["q"].float().view(B, H, 8, D)
    qg = q.movedim(1, 0).reshape(H, B * 8, D)
    sp = (qg @ kp.permute(1, 2, 0)).view(H, B, 8, shared).movedim(0, 1) * 0.0625
    so = torch.einsum("bhgd,bchd->bhgc", q, ko) * 0.0625
    sc = torch.cat([sp, so], -1)
    seen = torch.cat([idx.expand(B, -1), mine], -1) < lens[:, None]
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = (sc - torch.where(top > -math.inf, top, 0.0)).exp()
    total = p.sum(-1, keepdim=True)
    o = (p[..., :shared].movedim(1, 0).reshape(H, B * 8, shared) @ vp.movedim(1, 0)).view(H, B, 8, D).movedim(0, 1)
    o = o + torch.einsum("bhgc,bchd->bhgd", p[..., shared:], vo)
    o = torch.where(total > 0, o / total, 0.0)
    return (o @ _hadamard().float()).reshape(B, HQ, D)


def _plain_spec_accept(s):
    p, q, tokens = s["p"], s["q"], s["tokens"].long()
    B, n = tokens.shape
    i = torch.arange(n, device="cuda")
    pt = p[:, :n].gather(-1, tokens[..., None])[..., 0].double()
    qt = 1.0 if q is None else q.gather(-1, tokens[..., None])[..., 0].double()
    ok = (s["u"].double() * qt < pt) & (i < s["count"][:, None])
    acc = ok.long().cumprod(1).sum(1)
    b = torch.arange(B, device="cuda")
    target = p[b, acc].float()
    a = acc.clamp(max=n - 1)
    if q is None:
        less = target.scatter(1, tokens[b, a][:, None], 0.0)
    else:
        less = (target - q[b, a].float()).clamp(min=0)
    rejected = (acc < s["count"]) & (less.amax(-1) > 0)
    w = torch.where(rejected[:, None], less, target)
    cum = w.double().cumsum(-1)
    token = (cum > s["us"].double()[:, None] * cum[:, -1:]).int().argmax(-1).int()
    j = torch.arange(n + 1, device="cuda")
    mine = torch.cat([s["tokens"], s["tokens"][:, :1]], 1)
    out = torch.where(j < acc[:, None], mine, torch.where(j == acc[:, None], token[:, None], -1))
    return out.int(), acc.int()


def run(state):
    if own:
        return _run_own(state)
    return {"norm_rope": _plain_norm_rope, "append_rope": _plain_append_rope, "shared_decode": _plain_shared_decode,
            "spec_accept": _plain_spec_accept}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    B = case["seqs"]
    if case["op"] == "norm_rope":
        n, w = B * case["tok"], 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=n * (2 * w * (HQ + H) * D + 4 * case["rot"]), flops=n * (HQ + H) * (3 * case["rot"] + 4 * D))
    if case["op"] == "append_rope":
        n, w = B * case["tok"], 2 if case["dtype"] == "bf16" else 4
        # K and V in, the rotation's rows, the cache's bytes out; and the pages read back as fp32 values
        read = B * ((2 * case["P"] - 2 + case["tok"]) // case["P"] + 1) * case["P"]
        cell = H * CELL_HEAD[case["fmt"]]
        return dict(bytes=n * (2 * w * H * D + 4 * case["rot"] + cell) + read * (cell + 8 * H * D),
                    flops=n * H * (3 * case["rot"] + 20 * D))
    if case["op"] == "shared_decode":
        mine = B * (case["own_max"] + 1) // 2
        return dict(bytes=(case["shared"] + mine) * 816 + B * HQ * D * 6,
                    flops=4 * D * HQ * (B * case["shared"] + mine))
    w = 2 if case["dtype"] == "bf16" else 4
    return dict(bytes=B * (1 if case["sure"] else 2) * case["vocab"] * w, flops=B * 3 * case["vocab"])


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rotate(x, s):
    """Every pair as a complex number times e^(i angle), the angle's cosine and sine as the table has them."""
    case = s["case"]
    half = case["rot"] // 2
    pos = (s["pos"][:, None] + torch.arange(case["tok"], device="cuda")).reshape(-1)
    row = s["table"].double().index_select(0, pos).view(*x.shape[:2], 1, 2 * half)
    turn = torch.complex(row[..., :half].contiguous(), row[..., half:].contiguous())
    y = x.double().clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["inter"] else (slice(0, half), slice(half, 2 * half))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _walsh(x):
    """(H / 16) x by its eight stages of sums and differences."""
    y = x.double()
    for k in range(8):
        a = y.unflatten(-1, (D >> (k + 1), 2, 1 << k))
        y = torch.stack([a[..., 0, :] + a[..., 1, :], a[..., 0, :] - a[..., 1, :]], -2).flatten(-3)
    return y / 16


def _exact_int8(x):
    # the format's own roundings: the scale and the quotient are fp32 numbers
    x = x.double().view(*x.shape[:-1], 2, 128)
    s = (x.abs().max(-1, keepdim=True).values / 127).float().double()
    c = torch.round(torch.nan_to_num((x / s).float(), nan=0.0).double())
    return (c * s).view(*x.shape[:-2], D)


def _exact_q4(x):
    # the format's own roundings: the rotated value and the quotient are fp32 numbers, the scale an fp16 one
    y = _walsh(x).float().double().view(*x.shape[:-1], 8, 32)
    m = torch.gather(y, -1, y.abs().max(-1, keepdim=True).indices)
    d = (m / -8).float().half().double()
    c = (torch.round(torch.nan_to_num((y / d).float(), nan=0.0).double()) + 8).clamp(0, 15)
    return ((c - 8) * d).view(*x.shape[:-1], D)


def exact(case, seed):
    global own
    if case["op"] == "spec_accept":
        return None                                        # whole numbers
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if case["op"] == "norm_rope":
        both = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            y = x.double()
            if w is not None:
                y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / D + EPS) * w.double()
            both.append(_exact_rotate(y, s))
        return tuple(both)
    if case["op"] == "append_rope":
        P, fmt, n = case["P"], case["fmt"], s["n_pages"]
        k, ks, v, vs = (r.flatten(0, 1) for r in _runs(s["pages"], fmt, n, P))

        def values(codes, scales):
            if scales.dtype == torch.float32:
                return codes.double() * scales.double().repeat_interleave(128, -1)
            low, high = (codes & 15).view(-1, H, 8, 16), (codes >> 4).view(-1, H, 8, 16)
            return (torch.cat([low, high], -1).double() - 8).mul(scales.double()[..., None]).reshape(-1, H, D)

        old_k, old_v = values(k, ks), values(v, vs)
        if fmt == "q4":
            old_k = _walsh(old_k)
        new = _exact_rotate(s["k"], s).float().to(s["k"].dtype)
        new_k = _walsh(_exact_q4(new)) if fmt == "q4" else _exact_int8(new)
        new_v = _exact_int8(s["v"]) if fmt == "int8" else _exact_q4(s["v"])
        for b, start in enumerate(s["pos"].tolist()):
            c = torch.arange(start, start + case["tok"], device="cuda")
            at = s["page_table"][b, c // P].long() * P + c % P
            old_k[at], old_v[at] = new_k[b], new_v[b]
        return old_k, old_v
    # shared_decode: each sequence by itself over its own table, no part of it shared
    P, B = case["P"], case["seqs"]
    k, ks, v, vs = (r.flatten(0, 1) for r in _runs(s["pages"], "k8v4", s["n_pages"], P))
    out = torch.zeros(B, HQ, D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        c = torch.arange(n, device="cuda")
        at = s["page_table"][b, c // P].long() * P + c % P
        for h in range(H):
            kk = k[at, h].double() * ks[at, h].double().repeat_interleave(128, -1)
            low, high = (v[at, h] & 15).view(-1, 8, 16), (v[at, h] >> 4).view(-1, 8, 16)
            vv = ((torch.cat([low, high], -1).double() - 8) * vs[at, h].double()[..., None]).view(-1, D)
            w = torch.softmax(s["q"][b, 8 * h:8 * h + 8].double() @ kk.T / 16, -1)
            out[b, 8 * h:8 * h + 8] = _walsh(w @ vv)
    return out
