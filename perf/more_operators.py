"""Operators of a batched serving step over the quantized paged KV cache, as cases that can be timed and compared:
their plain forms in elementary torch operations, the library's own calls, and their definitions in 64 bits.

    plan         pages handed out and taken back for a step, block tables, slots and positions of its new tokens
    append       the new tokens of a ragged batch quantised and written through those slots
    diff_decode  differential attention over the cache, one query per sequence: the difference of two softmax maps
                 (one per 128-lane half of a key), its weight learned, the head normed
    diff         the same for a ragged batch: prompts, chunks and single tokens of several sequences side by side
    block_norm   a block's output normed, gated, scaled and added to the residual, the next block's norm with it

`own` says which of the two forms run() takes.  Geometry of the cache everywhere: head_dim 256, 2 KV heads, 8 query
heads per KV head; a differential head takes the 256 lanes as two maps of 128 and one value of 256."""
import math

import torch

own = False

D = 256            # head_dim
H = 2              # KV heads
HQ = 16            # query heads
EPS = 1.0e-6
SCALE = 128 ** -0.5
CELL_HEAD = 408    # bytes of one cell of one head (INT8 keys, rotated 4-bit values)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step of a small batch: one new token each, a page now and then
        dict(name="plan 32", op="plan", seqs=32, P=64, max_len=8192, prompts=0.0, done=0.0, new_max=1, tight=False),
        # a busy server's step: chats, prompts of up to 1,500 tokens, finished requests, not enough pages for all
        dict(name="plan 600", op="plan", seqs=600, P=16, max_len=16384, prompts=0.15, done=0.1, new_max=1500, tight=True),
        # the append of a decode step, one token of each of 40 sequences, some of them padding
        dict(name="append 40", op="append", tok=40, dtype="bf16", packed=True, P=16, idle=0.2),
        # prompts of a ragged batch, 20,011 tokens
        dict(name="append 20011", op="append", tok=20011, dtype="bf16", packed=True, P=64, idle=0.0),
        # one short chat: nothing but latency
        dict(name="diff_decode 1x1000", op="diff_decode", seqs=1, longest=1000, ragged=False, P=16, lam=1, norm=True),
        # a batch of 32, ragged, one of them empty
        dict(name="diff_decode 32x8192", op="diff_decode", seqs=32, longest=8192, ragged=True, P=64, lam=HQ, norm=True),
        # one long document
        dict(name="diff_decode 1x237568", op="diff_decode", seqs=1, longest=237568, ragged=False, P=64, lam=1, norm=True),
        # drafts under verification: 8 sequences of up to 5 tokens
        dict(name="diff 8x5", op="diff", seqs=8, tok=5, longest=16384, ragged=True, P=64, lam=1, norm=True),
        # chats and prompts side by side
        dict(name="diff 12x900", op="diff", seqs=12, tok=900, longest=3000, ragged=True, P=16, lam=HQ, norm=True),
        # the last chunk of a prompt of 32,768 tokens
        dict(name="diff 1x4096", op="diff", seqs=1, tok=4096, longest=32768, ragged=False, P=64, lam=1, norm=True),
        # one token between two blocks
        dict(name="block_norm 1x2048", op="block_norm", tok=1, dim=2048, y="bf16", dtype="bf16", gate="none", post=True,
             pre=True, residual=True),
        # a prompt chunk: attention's fp32 output gated by element, added to the residual, normed for the next block
        dict(name="block_norm 8192x4096", op="block_norm", tok=8192, dim=4096, y="f32", dtype="bf16", gate="sigmoid",
             post=True, pre=True, residual=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "diff_decode", "diff", "block_norm"])
    if op == "plan":
        return dict(op=op, seqs=_log(rng, 1, 600), P=rng.choice([16, 48, 64]), max_len=_log(rng, 64, 16384),
                    prompts=rng.choice([0.0, 0.1, 0.3]), done=rng.choice([0.0, 0.05, 0.2]), new_max=_log(rng, 1, 700),
                    tight=rng.random() < 0.4)
    if op == "append":
        return dict(op=op, tok=_log(rng, 1, 19000), dtype=rng.choice(["bf16", "f32"]), packed=rng.random() < 0.6,
                    P=rng.choice([16, 48, 64]), idle=rng.choice([0.0, 0.2]))
    lam, norm, P = rng.choice([0, 1, HQ]), rng.random() < 0.8, rng.choice([16, 48, 64, 128])
    if op == "diff_decode":
        seqs = _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, longest=_log(rng, 1, 230000 // seqs), ragged=rng.random() < 0.6, P=P, lam=lam, norm=norm)
    if op == "diff":
        seqs, tok = _log(rng, 1, 16), _log(rng, 1, 4000)
        tok = min(tok, 4000 // seqs + 1)
        longest = max(tok, _log(rng, 16, max(16, min(32000, 4000 * 32000 // (seqs * max(tok, 32) * 2)))))
        return dict(op=op, seqs=seqs, tok=tok, longest=longest, ragged=rng.random() < 0.6, P=P, lam=lam, norm=norm)
    dim = _log(rng, 100, 12000)
    return dict(op=op, tok=_log(rng, 1, max(1, min(8000, 30000000 // dim))), dim=dim - dim % rng.choice([1, 8, 64]),
                y=rng.choice(["bf16", "f32"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                gate=rng.choice(["none", "raw", "sigmoid", "silu", "row"]), post=rng.random() < 0.7,
                pre=rng.random() < 0.8, residual=rng.random() < 0.8)


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _keys(g, n):
    """One channel in a hundred is 20 times as large, as keys have them."""
    return _normal(g, n, H, D) * torch.where(_uniform(g, H, D) < 0.01, 20.0, 1.0)


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


def _cache_bytes(g, pages, P):
    """A filled cache: per page the runs of K codes, K scales, V nibbles, V scales."""
    kc, ks = _int8_half(_keys(g, pages * P))
    vc, vs = _q4(_normal(g, pages * P, H, D))
    runs = (kc.to(torch.int8), ks, _nibbles(vc), vs)
    return torch.cat([r.contiguous().view(torch.uint8).reshape(pages, -1) for r in runs], 1).reshape(-1)


def _handle(s, P):
    """The cache descriptor a program makes once, over the bytes that the state holds."""
    import quantized_paged_kv_q8_gb300 as k8
    s["cache"] = k8.PagedCache(s["n_pages"], P, H, k8.FORMAT_K8V4, pages=s["pages"])
    return k8


def _shape(case):
    """What the sizes of a case's batch are drawn from: the case alone, other values fill it with each seed."""
    return _generator(1000 * case["seqs"] + 7 * case.get("tok", 0) + 1)


def _prepare_plan(case, g):
    B, P = case["seqs"], case["P"]
    max_pages = -(-(case["max_len"] + case["new_max"]) // P)
    n_pages = B * max_pages + 64
    shape = _shape(case)
    u = _uniform(shape, B)
    new = torch.where(u < case["prompts"], (case["new_max"] ** _uniform(shape, B)).long(), 1)
    new = torch.where((u >= case["prompts"]) & (u < case["prompts"] + case["done"]), -1, new)
    new = torch.where(u > 0.97, 0, new) if B > 8 else new                           # waits for its caller
    lens = torch.randint(0, case["max_len"] + 1, (B,), generator=g, device="cuda")
    lens = torch.where(u < case["prompts"] * 0.5, 0, lens)                           # a prompt's first tokens
    have = (lens + P - 1) // P
    used = int(have.sum())
    want = int(((lens + new.clamp(min=0) + P - 1) // P - have).clamp(min=0).sum())
    back = int(torch.where(new < 0, have, 0).sum())
    spare = min(n_pages - used, max(0, want - back) * 3 // 4 if case["tight"] else want + 50)
    ids = torch.randperm(n_pages, generator=g, device="cuda").int()
    j = torch.arange(max_pages, device="cuda")
    rank = (have.cumsum(0) - have)[:, None] + j
    table = torch.where(j < have[:, None], ids[rank.clamp(max=n_pages - 1)], -1).int()
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:spare] = ids[used:used + spare]
    T = max(1, int(new.clamp(min=0).sum())) + 17                                    # a padded batch
    new_i = dict(dtype=torch.int32, device="cuda")
    return dict(case=case, page_table=table, free=free, n_free=torch.tensor([spare], **new_i), lens=lens.int(), new=new.int(),
                tokens=T, new_lens=torch.empty(B, **new_i), n_free_out=torch.empty(1, **new_i),
                offsets=torch.empty(B + 1, **new_i), granted=torch.empty(B, **new_i),
                positions=torch.empty(T, dtype=torch.int64, device="cuda"),
                slots=torch.empty(T, dtype=torch.int64, device="cuda"))


def _prepare_append(case, g):
    T, P, dt = case["tok"], case["P"], _dtype(case["dtype"])
    pages = -(-T // P) + 3
    if case["packed"]:
        flat = _normal(g, T, HQ + 2 * H, D)
        flat[:, HQ:HQ + H] = _keys(g, T)
        k, v = flat.to(dt).split([HQ, H, H], 1)[1:]
    else:
        k, v = _keys(g, T).to(dt), _normal(g, T, H, D).to(dt)
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:T]
    # runs of cells, as a plan gives them: whole pages in a random order
    order = torch.randperm(pages, generator=g, device="cuda")
    run = torch.arange(T, device="cuda")
    slots = torch.where(torch.tensor(T > 2 * P, device="cuda"), order[run // P] * P + run % P, slots)
    slots = torch.where(_uniform(g, T) < case["idle"], -1, slots)
    s = dict(case=case, k=k, v=v, slots=slots, pages=_cache_bytes(g, pages, P), n_pages=pages,
             every=torch.arange(pages, dtype=torch.int32, device="cuda"),
             k_hat=torch.empty(pages * P, H, D, device="cuda"), v_hat=torch.empty(pages * P, H, D, device="cuda"))
    if own:
        _handle(s, P)
    return s


def _heads(case, g, s):
    """The learned weights of the differential heads of one layer."""
    s["lam"] = [0.1 * _normal(g, case["lam"], 128) for _ in range(4)] if case["lam"] else None
    s["init"] = 0.8 - 0.6 * math.exp(-0.3 * (1 + int(torch.randint(0, 30, (1,), generator=g, device="cuda"))))
    s["w"] = 1.0 + 0.2 * _normal(g, D) if case["norm"] else None


def _prepare_diff(case, g):
    B, P, longest = case["seqs"], case["P"], case["longest"]
    single = case["op"] == "diff_decode"
    lens = torch.full((B,), longest, device="cuda")
    if case["ragged"] and B > 1:
        lens[1:] = (1 + (longest - 1) * _uniform(g, B - 1)).long()
        if B > 3:
            lens[2] = 0
    n = torch.ones(B, dtype=torch.int64, device="cuda") if single else torch.full((B,), case["tok"], device="cuda")
    if not single:
        if case["ragged"] and B > 1:
            n[1:] = (case["tok"] ** _uniform(_shape(case), B - 1)).long()
            if B > 3:
                n[2] = 0                                   # in the batch, with nothing to do in this step
        lens = torch.maximum(n, lens)
    each = -(-longest // P)
    pages = B * each
    T = int(n.sum())
    s = dict(case=case, n_pages=pages, pages=_cache_bytes(g, pages, P), lens=lens.int(), max_len=longest,
             page_table=torch.randperm(pages, generator=g, device="cuda").int().view(B, each), q=_normal(g, T, HQ, D).bfloat16(),
             out=torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda"))
    _heads(case, g, s)
    if not single:
        s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
        s["most"] = int(n.max())
    if own:
        k8 = _handle(s, P)
        s["heads"] = k8.DifferentialHeads(lambdas=s["lam"], lambda_init=s["init"], norm_weight=s["w"], eps=EPS,
                                          out_scale=1.0 - s["init"])
        s["ws"] = k8.diff_decode_workspace(s["cache"], B, longest) if single else k8.diff_workspace(s["cache"], B, T, longest)
    return s


def _prepare_block_norm(case, g):
    n, dim, dt = case["tok"], case["dim"], _dtype(case["dtype"])
    gate = None
    if case["gate"] != "none":
        gate = _normal(g, 1 if case["gate"] == "row" else n, dim).to(dt)
    return dict(case=case, y=_normal(g, n, dim).to(_dtype(case["y"])), gate=gate,
                residual=(2.0 * _normal(g, n, dim)).to(dt) if case["residual"] else None,
                post=1.0 + 0.2 * _normal(g, dim) if case["post"] else None,
                pre=1.0 + 0.2 * _normal(g, dim) if case["pre"] else None,
                h=torch.empty(n, dim, dtype=dt, device="cuda"),
                normed=torch.empty(n, dim, dtype=dt, device="cuda") if case["pre"] else None)


ALPHA = 0.7        # the residual scale of a block
ACTS = {"none": "none", "raw": "none", "row": "none", "sigmoid": "sigmoid", "silu": "silu"}


def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "diff_decode": _prepare_diff, "diff": _prepare_diff,
            "block_norm": _prepare_block_norm}[case["op"]](case, _generator(seed))


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    import quantized_paged_kv_q8_gb300 as k8
    case = s["case"]
    if case["op"] == "plan":
        k8.kv_plan_k8v4(case["P"], s["free"], s["n_free"], s["page_table"], s["lens"], s["new"], s["offsets"], s["positions"],
                        s["slots"], s["granted"], new_lens=s["new_lens"], n_free_out=s["n_free_out"])
        return s["page_table"], s["free"], s["n_free_out"], s["new_lens"], s["offsets"], s["positions"], s["slots"], s["granted"]
    if case["op"] == "append":
        k8.kv_append_k8v4_slots(s["cache"], s["slots"], s["k"], s["v"])
        # the updated pages, as the values that the codes stand for
        k8.kv_dequant_k8v4(s["cache"], s["every"], 0, s["n_pages"] * case["P"], s["k_hat"], s["v_hat"])
        return s["k_hat"], s["v_hat"]
    if case["op"] == "diff_decode":
        return k8.attn_k8v4_diff_decode(s["cache"], s["q"], s["page_table"], s["lens"], s["max_len"], s["heads"], s["out"],
                                        s["ws"], sm_scale=SCALE)
    if case["op"] == "diff":
        return k8.attn_k8v4_diff(s["cache"], s["q"], s["offsets"], s["page_table"], s["lens"], s["max_len"], s["heads"],
                                 s["out"], s["ws"], sm_scale=SCALE)
    k8.block_norm_k8v4(s["y"], s["residual"], s["h"], post_weight=s["post"], gate=s["gate"], gate_act=ACTS[case["gate"]],
                       residual_scale=ALPHA, pre_weight=s["pre"], normed=s["normed"], eps=EPS)
    return (s["h"], s["normed"]) if case["pre"] else s["h"]


# ---------------------------------------------------------------- the plain forms
def _plain_plan(s):
    case, P, T = s["case"], s["case"]["P"], s["tokens"]
    table, free, lens, new = s["page_table"].long(), s["free"].long(), s["lens"].long(), s["new"].long()
    B, max_pages = table.shape
    n_pages, n_free = free.shape[0], s["n_free"].long()
    want = new.clamp(min=0)
    ends = want.cumsum(0)
    have = (lens + P - 1) // P
    fits = (new >= 0) & (lens + want <= max_pages * P) & (ends <= T)
    need = torch.where(fits, (lens + want + P - 1) // P - have, 0)
    asked = need.cumsum(0)
    # what finished sequences give back goes on the stack first, in order
    back = torch.where(new == -1, have, 0)
    back_ends = back.cumsum(0)
    j = torch.arange(n_pages, device="cuda")
    giver = torch.searchsorted(back_ends, j, right=True).clamp(max=B - 1)
    given = table[giver, (j - (back_ends - back)[giver]).clamp(0, max_pages - 1)]
    total = n_free + back_ends[-1:]
    stack = torch.where(j < n_free, free, given[(j - n_free).clamp(min=0)])
    ok = fits & ((need == 0) | (asked <= total))
    got = torch.where(ok, need, 0)
    taken = got.sum()
    # entry k of the pages handed out is k below the top of the stack
    col = torch.arange(max_pages, device="cuda")
    k = (asked - need)[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + got)[:, None])
    table = torch.where(fresh, stack[(total - 1 - k).clamp(0, n_pages - 1)], table)
    left = total - taken
    free = torch.where((j >= n_free) & (j < left), stack, free)
    # the new tokens
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    cell = lens[b] + t - (ends - want)[b]
    page = table[b, (cell // P).clamp(0, max_pages - 1)]
    written = live & ok[b]
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return (table.int(), free.int(), left.int(), torch.where(new == -1, 0, torch.where(ok, lens + want, lens)).int(),
            torch.cat([zero, ends]).clamp(max=T).int(), torch.where(written, cell, 0),
            torch.where(written, page * P + cell % P, -1), torch.where(ok, want, 0).int())


def _hadamard():
    i = torch.arange(D, device="cuda")
    bits = i[:, None] & i[None, :]
    bits = bits ^ (bits >> 4)
    bits = bits ^ (bits >> 2)
    return (1 - 2 * ((bits ^ (bits >> 1)) & 1)).double() / 16


def _q4_values(nib, scales):
    """bytes [..., 128] and fp16 [..., 8] -> fp32 [..., 256]"""
    b = nib.unflatten(-1, (8, 16))
    c = torch.stack([b & 15, b >> 4], -2).flatten(-2).float() - 8
    return (c * scales.float()[..., None]).flatten(-2)


def _int8_values(codes, scales):
    return (codes.float().unflatten(-1, (2, 128)) * scales[..., None]).flatten(-2)


def _runs(s):
    """The four runs of every page as [cells, H, ...]: K codes and scales, V nibbles and scales."""
    n, P = s["n_pages"], s["case"]["P"]
    runs = [r.contiguous() for r in s["pages"].view(n, P * H * CELL_HEAD).split([P * H * w for w in (256, 8, 128, 16)], 1)]
    types = (torch.int8, torch.float32, torch.uint8, torch.float16)
    return [r.view(t).view(n * P, H, -1) for r, t in zip(runs, types)]


def _plain_append(s):
    k = _int8_values(*_int8_half(s["k"].float()))
    # the rotation in 64 bits (a code next to a border goes by the last bit), rounded once
    c, d = _q4((s["v"].double() @ _hadamard()).float())
    v = ((c - 8).unflatten(-1, (8, 32)) * d.float()[..., None]).flatten(-2)
    kc, ks, vn, vs = _runs(s)
    k_hat, v_hat = _int8_values(kc, ks), _q4_values(vn, vs)
    live = s["slots"] >= 0
    at = s["slots"][live]
    k_hat[at] = k[live]
    v_hat[at] = v[live]
    return k_hat, v_hat


def _weight(s):
    """lambda of every query head, [HQ] or one for all."""
    if s["lam"] is None:
        return torch.full((1,), s["init"], device="cuda")
    a, b, c, d = s["lam"]
    return (a * b).sum(-1).exp() - (c * d).sum(-1).exp() + s["init"]


def _differential(s, q, seen):
    """q fp32 [B, T, HQ, 256], seen: the cells that each query sees, [B, T] -> fp32 [B, T, HQ, 256]."""
    P, L = s["case"]["P"], s["max_len"]
    idx = torch.arange(L, device="cuda")
    at = s["page_table"].long()[:, idx // P] * P + idx % P
    kc, ks, vn, vs = _runs(s)
    K, V = _int8_values(kc[at], ks[at]), _q4_values(vn[at], vs[at])                  # [B, L, H, 256]
    B, T = q.shape[:2]
    rows = q.view(B, T, H, 8, 2, 128).permute(0, 2, 4, 1, 3, 5).reshape(B, H, 2, T * 8, 128)
    K = K.view(B, L, H, 2, 128).permute(0, 2, 3, 4, 1)                               # [B, H, map, 128, L]
    sc = (rows @ K).view(B, H, 2, T, 8, L) * SCALE
    sc.masked_fill_((idx >= seen[..., None])[:, None, None, :, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(B, H, 2, T * 8, L) @ V.permute(0, 2, 1, 3)[:, :, None]
    o = torch.where(total > 0, o.view(B, H, 2, T, 8, D) / total, 0.0) @ _hadamard().float()
    o = o.permute(0, 3, 1, 4, 2, 5).reshape(B, T, HQ, 2, D)
    x = o[..., 0, :] - _weight(s)[:, None] * o[..., 1, :]
    if s["w"] is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w"]
    return x * (1.0 - s["init"])


def _plain_diff_decode(s):
    return _differential(s, s["q"].float()[:, None], s["lens"].long()[:, None])[:, 0].bfloat16()


def _plain_diff(s):
    off = s["offsets"].long()
    n = off[1:] - off[:-1]
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(off[1:], t, right=True)
    i = t - off[b]
    B, T = n.shape[0], s["most"]
    q = torch.zeros(B, T, HQ, D, device="cuda")
    q[b, i] = s["q"].float()
    j = torch.arange(T, device="cuda")
    seen = torch.where(j < n[:, None], (s["lens"].long() - n)[:, None] + j + 1, 0)
    return _differential(s, q, seen)[b, i].bfloat16()


def _normed(x, w):
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w


def _plain_block_norm(s):
    case = s["case"]
    a = s["y"].float()
    if s["post"] is not None:
        a = _normed(a, s["post"])
    if s["gate"] is not None:
        z = s["gate"].float()
        u = 1.0 / (1.0 + (-z).exp())
        a = a * {"none": z, "sigmoid": u, "silu": z * u}[ACTS[case["gate"]]]
    a = ALPHA * a
    h = (a if s["residual"] is None else s["residual"].float() + a).to(s["h"].dtype)
    if s["pre"] is None:
        return h
    return h, _normed(h.float(), s["pre"]).to(h.dtype)


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "append": _plain_append, "diff_decode": _plain_diff_decode, "diff": _plain_diff,
            "block_norm": _plain_block_norm}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    if case["op"] == "plan":
        B = case["seqs"]
        tok = B * (1 + case["prompts"] * case["new_max"] / max(1.0, math.log(case["new_max"] + 1.0)))
        back = case["done"] * B * case["max_len"] / 2 / case["P"]
        # lengths and requests in and out; each new token's page, slot and position; pages handed out and given back
        return dict(bytes=int(20 * B + 20 * tok + 8 * tok / case["P"] + 8 * back), flops=int(4 * (B + tok)))
    if case["op"] == "append":
        n, w, P = case["tok"], 2 if case["dtype"] == "bf16" else 4, case["P"]
        read = (-(-n // P) + 3) * P
        return dict(bytes=n * (2 * w * H * D + 8 + H * CELL_HEAD) + read * H * (CELL_HEAD + 8 * D), flops=n * H * 20 * D)
    if case["op"] in ("diff_decode", "diff"):
        B, L = case["seqs"], case["longest"]
        T = 1 if case["op"] == "diff_decode" else case["tok"]
        cells, tok = B * L, B * T
        if case["ragged"] and B > 1:
            cells = L + (B - 1) * L // 2
            tok = T + (B - 1) * max(1, int((T - 1) / max(1.0, math.log(T)))) if T > 1 else B
        seen = tok * max(1, L - T // 2) if not case["ragged"] else tok * max(1, cells // B)
        # q1 k1 and q2 k2 over 128 lanes each, p1 v and p2 v over 256
        return dict(bytes=cells * H * CELL_HEAD + tok * HQ * D * 4, flops=1536 * HQ * seen)
    n, dim, w = case["tok"], case["dim"], 2 if case["dtype"] == "bf16" else 4
    gate = 0 if case["gate"] == "none" else 1 if case["gate"] == "row" else n
    return dict(bytes=dim * (n * (2 if case["y"] == "bf16" else 4) + w * (gate + n * (case["residual"] + 1 + case["pre"]))),
                flops=10 * n * dim)


# ---------------------------------------------------------------- the definitions in 64 bits
def _walsh(x):
    """(H / 16) x by its eight stages of sums and differences."""
    y = x.double()
    for k in range(8):
        a = y.unflatten(-1, (D >> (k + 1), 2, 1 << k))
        y = torch.stack([a[..., 0, :] + a[..., 1, :], a[..., 0, :] - a[..., 1, :]], -2).flatten(-3)
    return y / 16


def _exact_append(s):
    """The stored values by their definition, in which scales and quotients are fp32."""
    kc, ks, vn, vs = _runs(s)
    k_hat = kc.double() * ks.double().repeat_interleave(128, -1)
    codes = torch.cat([(vn & 15).view(-1, H, 8, 16), (vn >> 4).view(-1, H, 8, 16)], -1).double() - 8
    v_hat = (codes * vs.double()[..., None]).reshape(-1, H, D)
    live = s["slots"] >= 0
    at = s["slots"][live]
    for half in range(2):
        x = s["k"][..., 128 * half:128 * half + 128]
        scale = (x.abs().amax(-1).float() / torch.full((1,), 127.0, device="cuda")).double()
        code = torch.where(scale[..., None] > 0, x.double() / scale.clamp(min=1e-300)[..., None], 0.0).float().double()
        k_hat[at, :, 128 * half:128 * half + 128] = (code.round().clamp(-127, 127) * scale[..., None])[live]
    y = _walsh(s["v"]).float()                                                       # the stored rotation is fp32
    for block in range(8):
        x = y[..., 32 * block:32 * block + 32]
        most = x.abs().max(-1, keepdim=True).indices
        d = (x.gather(-1, most) / -8).half().double()
        code = torch.where(d != 0, (x.double() / torch.where(d != 0, d, 1.0)).float().double().round().clamp(-8, 7), 0.0)
        v_hat[at, :, 32 * block:32 * block + 32] = (code * d)[live]
    return k_hat, v_hat


def _exact_diff(s):
    """Sequence by sequence and map by map over the sequence's own cells."""
    case, P = s["case"], s["case"]["P"]
    kc, ks, vn, vs = _runs(s)
    T = s["q"].shape[0]
    maps = torch.zeros(2, T, HQ, D, dtype=torch.float64, device="cuda")
    off = list(range(T + 1)) if case["op"] == "diff_decode" else s["offsets"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        lo, hi = off[b], off[b + 1]
        if n == 0 or hi == lo:
            continue
        c = torch.arange(n, device="cuda")
        at = s["page_table"][b, c // P].long() * P + c % P
        sees = n - (hi - lo) + 1 + torch.arange(hi - lo, device="cuda")
        for g in range(H):
            codes = torch.cat([(vn[at, g] & 15).view(-1, 8, 16), (vn[at, g] >> 4).view(-1, 8, 16)], -1).double() - 8
            v = _walsh((codes * vs[at, g].double()[..., None]).reshape(-1, D))
            for m in range(2):
                k = kc[at, g, 128 * m:128 * m + 128].double() * ks[at, g, m].double()[:, None]
                for h in range(8 * g, 8 * g + 8):
                    sc = s["q"][lo:hi, h, 128 * m:128 * m + 128].double() @ k.T / math.sqrt(128.0)
                    sc[c >= sees[:, None]] = -math.inf
                    maps[m, lo:hi, h] = torch.softmax(sc, -1) @ v
    lam = torch.tensor(s["init"], dtype=torch.float64, device="cuda").expand(HQ)
    if s["lam"] is not None:
        a, b, c, d = (x.double() for x in s["lam"])
        lam = lam + torch.exp(torch.einsum("hd,hd->h", a, b)) - torch.exp(torch.einsum("hd,hd->h", c, d))
    x = maps[0] - lam.view(1, HQ, 1) * maps[1]
    if s["w"] is not None:
        x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / D + EPS) * s["w"].double()
    return x * (1.0 - s["init"])


def _exact_block_norm(s):
    case = s["case"]

    def norm(x, w):
        return x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()

    a = s["y"].double()
    if s["post"] is not None:
        a = norm(a, s["post"])
    if s["gate"] is not None:
        z = s["gate"].double()
        act = ACTS[case["gate"]]
        a = a * (z if act == "none" else torch.sigmoid(z) * (z if act == "silu" else 1.0))
    h = ALPHA * a + (0.0 if s["residual"] is None else s["residual"].double())
    if s["pre"] is None:
        return h
    # the next block norms what it finds: the sum as it is stored
    return h, norm(h.to(s["h"].dtype).double(), s["pre"])


def exact(case, seed):
    global own
    if case["op"] == "plan":
        return None                                        # whole numbers
    was, own = own, False
    s = prepare(case, seed)
    own = was
    return {"append": _exact_append, "diff_decode": _exact_diff, "diff": _exact_diff, "block_norm": _exact_block_norm}[case["op"]](s)
