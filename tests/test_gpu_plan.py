"""kv_plan_k8v4 against a sequence-by-sequence simulation, and kv_append_k8v4_slots against
the oracle's appends: batches of every size, pages given back and handed out in one call, refusals, bad values,
padded batches, in place and captured."""
import numpy as np
import pytest
import torch

import oracle
import quantized_paged_kv_q8_gb300 as k8
from gpu_util import CANARY

pytestmark = pytest.mark.gpu


def simulate(P, n_pages, free, n_free, table, lens, new, borrowed, T):
    """The rule, one sequence after the other."""
    free, table, B, width = free.copy(), table.copy(), len(lens), table.shape[1]
    borrowed = np.zeros(B, int) if borrowed is None else borrowed
    status = 0
    top = int(np.clip(n_free, 0, n_pages))
    status = status or (k8.ERANGE if top != n_free else 0)
    stack = list(free[:top])
    out_len, granted, ok_len = lens.copy(), np.zeros(B, np.int32), (lens >= 0) & (lens <= width * P)
    done = np.zeros(B, bool)
    for b in range(B):
        if new[b] == -1 and ok_len[b]:
            have = -(-int(lens[b]) // P)
            row = table[b, max(borrowed[b], 0):have]
            if borrowed[b] < 0 or borrowed[b] > have or (len(row) and ((row < 0) | (row >= n_pages)).any()):
                status = status or k8.ERANGE
                continue
            stack += list(row)
            out_len[b], done[b] = 0, True
    given = list(stack)
    off, pos, slots = np.zeros(B + 1, np.int64), np.zeros(T, np.int64), np.full(T, -1, np.int64)
    full = False
    at = 0
    for b in range(B):
        want = max(int(new[b]), 0)
        start, at = at, at + want
        off[b + 1] = at
        if not ok_len[b] or new[b] < -1:
            status = status or k8.ERANGE
            continue
        if new[b] == -1:
            continue
        if lens[b] + want > width * P:
            status = status or k8.ERANGE
            if at > T and want:
                status = status or k8.ENOSPACE
            continue
        if at > T and want:
            status = status or k8.ENOSPACE
            continue
        have, need = -(-int(lens[b]) // P), -(-(int(lens[b]) + want) // P)
        if need > have:
            if full or need - have > len(stack):
                full = True                                # every later one that needs a page is refused too
                status = status or k8.ENOSPACE
                continue
            for j in range(have, need):
                table[b, j] = stack.pop()
        out_len[b], granted[b] = lens[b] + want, want
        for i in range(want):
            c = int(lens[b]) + i
            pos[start + i] = c
            slots[start + i] = int(table[b, c // P]) * P + c % P
    left = len(stack)
    if left > top:
        free[top:left] = given[top:left]
    return dict(free=free, n_free=left, table=table, lens=out_len, off=np.minimum(off, T), pos=pos, slots=slots,
                granted=granted, status=status)


def batch(rng, B, P, longest, n_pages_extra, prompts=0.3, done=0.2, most=50, borrow=False):
    lens = rng.integers(0, longest + 1, B).astype(np.int32)
    new = np.where(rng.random(B) < prompts, rng.integers(0, most + 1, B), 1).astype(np.int32)
    new[rng.random(B) < done] = -1
    width = -(-(longest + most) // P) + 1
    have = -(-lens // P)
    n_pages = int(have.sum()) + n_pages_extra
    ids = rng.permutation(n_pages).astype(np.int32)
    table = rng.integers(-5, n_pages + 5, (B, width)).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = np.full(max(n_pages, 1), -1, np.int32)
    free[:n_pages_extra] = ids[at:]
    borrowed = None
    if borrow:
        borrowed = np.array([rng.integers(0, h + 1) for h in have], np.int32)
    return dict(P=P, n_pages=max(n_pages, 1), free=free, n_free=n_pages_extra, table=table, lens=lens, new=new,
                borrowed=borrowed, T=int(np.maximum(new, 0).sum()) + 5)


def dev(a, dtype=torch.int32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def run(s, in_place=False):
    free, table, lens = dev(s["free"]), dev(s["table"]), dev(s["lens"])
    n_free = torch.tensor([s["n_free"]], dtype=torch.int32, device="cuda")
    B, T = len(s["lens"]), s["T"]
    i32 = dict(dtype=torch.int32, device="cuda")
    off, granted = torch.full((B + 1,), -9, **i32), torch.full((B,), -9, **i32)
    pos, slots = (torch.full((T,), -9, dtype=torch.int64, device="cuda") for _ in range(2))
    new_lens = lens if in_place else torch.full((B,), -9, **i32)
    n_free_out = n_free if in_place else torch.full((1,), -9, **i32)
    k8.kv_plan_k8v4(s["P"], free, n_free, table, lens, dev(s["new"]), off, pos, slots, granted,
                    new_lens=None if in_place else new_lens, n_free_out=None if in_place else n_free_out,
                    n_borrowed=dev(s["borrowed"]))
    got = dict(free=free, n_free=n_free_out, table=table, lens=new_lens, off=off, pos=pos, slots=slots, granted=granted)
    return {k: v.cpu().numpy() for k, v in got.items()}


def check(s, in_place=False):
    want = simulate(s["P"], s["n_pages"], s["free"], s["n_free"], s["table"], s["lens"], s["new"], s["borrowed"], s["T"])
    got = run(s, in_place)
    status = k8.k8v4_last_device_status()
    for k in got:
        assert np.array_equal(np.asarray(got[k]).ravel(), np.asarray(want[k]).ravel()), k
    assert (status != 0) == (want["status"] != 0)
    return want, got, status


@pytest.mark.parametrize("B,P,longest,extra,most", [
    (1, 16, 0, 4, 3), (1, 64, 1000, 0, 20), (7, 16, 40, 3, 50), (32, 64, 3000, 100, 1), (33, 48, 500, 10, 300),
    (600, 16, 700, 100, 90), (1025, 16, 60, 300, 5), (3000, 32, 100, 5000, 40), (8192, 16, 30, 700, 3)])
@pytest.mark.parametrize("borrow,in_place", [(False, False), (True, True)])
def test_plan(B, P, longest, extra, most, borrow, in_place):
    rng = np.random.default_rng(B + P + longest + borrow)
    check(batch(rng, B, P, longest, extra, most=most, borrow=borrow), in_place)


@pytest.mark.parametrize("extra", [0, 1, 5, 17, 1000])
def test_scarce_pages(extra):
    """Refused sequences, and later ones that need no page still served; with and without pages given back."""
    for done in (0.0, 0.3):
        rng = np.random.default_rng(extra)
        s = batch(rng, 90, 16, 200, extra, prompts=0.5, done=done, most=40)
        want, _, status = check(s)
        assert status in (0, k8.ENOSPACE)


def test_too_many_tokens():
    """The packed tokens end at max_tokens: sequences that pass it are refused, offsets stop there."""
    rng = np.random.default_rng(3)
    for T in (0, 1, 40, 100):
        s = batch(rng, 40, 16, 100, 400, prompts=0.8, done=0.1, most=20)
        s["T"] = T
        _, _, status = check(s)
        assert status == k8.ENOSPACE


def test_nothing_in_the_batch():
    s = dict(P=16, n_pages=4, free=np.array([3, 1, -1, -1], np.int32), n_free=2, table=np.zeros((0, 2), np.int32),
             lens=np.zeros(0, np.int32), new=np.zeros(0, np.int32), borrowed=None, T=3)
    got = run(s)
    assert got["off"].tolist() == [0] and got["slots"].tolist() == [-1] * 3 and got["n_free"].tolist() == [2]


def test_bad_values():
    """Lengths, counts, borrowed pages, stack heights and page ids out of range refuse their sequence and are
    recorded; the others are served."""
    rng = np.random.default_rng(4)
    base = batch(rng, 20, 16, 100, 60, done=0.3)
    width = base["table"].shape[1]
    for change in ("len", "neg", "count", "past", "borrow", "row", "low", "high"):
        s = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in base.items()}
        if change == "len":
            s["lens"][3] = width * 16 + 1
        elif change == "neg":
            s["lens"][5] = -4
        elif change == "count":
            s["new"][2] = -3
        elif change == "past":
            s["new"][6], s["lens"][6] = 5, width * 16 - 2
            s["T"] += 5
        elif change == "borrow":
            s["borrowed"] = np.zeros(20, np.int32)
            s["new"][4], s["borrowed"][4] = -1, 99
        elif change == "row":
            b = int(np.argmax(s["lens"]))
            s["new"][b] = -1
            s["table"][b, 1] = s["n_pages"]
        elif change == "low":
            s["n_free"] = -3
        elif change == "high":
            s["free"] = np.arange(s["n_pages"], dtype=np.int32)
            s["n_free"] = s["n_pages"] + 7
            s["new"][s["new"] == -1] = 1
        if change == "past":                               # the row's pages up to the length are named
            s["table"][6] = s["table"][6] % s["n_pages"]
        _, _, status = check(s)
        assert status == k8.ERANGE, change


def test_pages_are_neither_lost_nor_doubled():
    """A server's life: steps of a changing batch in place on the device, captured once; every page is in the stack or
    in one row at all times."""
    rng = np.random.default_rng(5)
    B, P, width, n_pages = 48, 16, 20, 400
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.full((B, width), -1, **i32), torch.zeros(B, **i32)
    free, n_free = dev(rng.permutation(n_pages).astype(np.int32)), torch.tensor([n_pages], **i32)
    new, off, granted = torch.zeros(B, **i32), torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
    pos, slots = (torch.zeros(900, dtype=torch.int64, device="cuda") for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k8.kv_plan_k8v4(P, free, n_free, table, lens, new, off, pos, slots, granted)
    held = np.zeros(B, int)
    for _ in range(60):
        want = rng.integers(0, 30, B).astype(np.int32)
        want[rng.random(B) < 0.15] = -1
        new.copy_(dev(want))
        g.replay()
        t, ln, f, nf = table.cpu().numpy(), lens.cpu().numpy(), free.cpu().numpy(), int(n_free)
        got = granted.cpu().numpy()
        held = np.where(want == -1, 0, held + got)
        assert np.array_equal(ln, held)
        owned = np.concatenate([t[b, :-(-ln[b] // P)] for b in range(B)] + [f[:nf]])
        assert np.array_equal(np.sort(owned), np.arange(n_pages))
    k8.k8v4_last_device_status()


# ---------------------------------------------------------------- appends through slots
@pytest.mark.parametrize("fmt", [k8.FORMAT_K8V4, k8.FORMAT_INT8, k8.FORMAT_Q4])
@pytest.mark.parametrize("n,H,P,dtype,packed", [(1, 2, 16, "bf16", False), (37, 3, 48, "f32", True), (200, 2, 64, "bf16", True),
                                                (2600, 2, 16, "bf16", True), (5001, 1, 32, "bf16", False), (2700, 2, 16, "f32", False)])
def test_slots_write_the_append_s_bytes(fmt, n, H, P, dtype, packed):
    rng = np.random.default_rng(n + H)
    pages = -(-n // P) + 2
    gpu, ref = k8.PagedCache(pages, P, H, fmt), oracle.Cache(pages, P, H, fmt, fill=CANARY)
    gpu.pages.fill_(CANARY)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    flat = torch.from_numpy(rng.standard_normal((n, 2 * H + 3, 256)).astype(np.float32)).to(dt).cuda()
    k, v = flat[:, :H], flat[:, H:2 * H]
    if not packed:
        k, v = k.contiguous(), v.contiguous()
    slots = rng.permutation(pages * P)[:n].astype(np.int64)
    idle = rng.random(n) < 0.1
    slots[idle] = -1
    k8.kv_append_k8v4_slots(gpu, torch.from_numpy(slots).cuda(), k, v)
    assert k8.k8v4_last_device_status() == 0
    # the oracle writes token t as a sequence of its own, its one page the slot's
    live = np.flatnonzero(~idle)
    kn, vn = (np.ascontiguousarray(x.float().cpu().numpy()[live][:, None]) for x in (k, v))
    ref.append((slots[live] // P).astype(np.int32)[:, None], slots[live] % P, kn, vn)
    assert np.array_equal(gpu.pages.cpu().numpy(), ref.buf)


@pytest.mark.parametrize("n", [3, 3000])
def test_slots_out_of_range_are_skipped(n):
    rng = np.random.default_rng(n)
    pages, P = -(-n // 16) + 1, 16
    caches = [k8.PagedCache(pages, P) for _ in range(2)]
    k, v = (torch.from_numpy(rng.standard_normal((n, 2, 256)).astype(np.float32)).bfloat16().cuda() for _ in range(2))
    slots = torch.from_numpy(rng.permutation(pages * P)[:n].astype(np.int64)).cuda()
    for bad in (-2, pages * P, 1 << 40, -(1 << 62)):
        s, t = slots.clone(), slots.clone()
        s[1], t[1] = bad, -1
        for c, at in zip(caches, (s, t)):
            c.pages.fill_(CANARY)
            k8.kv_append_k8v4_slots(c, at, k, v)
            assert k8.k8v4_last_device_status() == (k8.ERANGE if at is s else 0)
        assert torch.equal(caches[0].pages, caches[1].pages)
