"""What orders the reuse of each buffer of the ragged tile kernel (csrc/k8v4_diff_tc.cu): its roles, their waits and
arrivals as a graph, in which every use of a place has to come behind all uses of the tile that had it before.  On the CPU:
a missing wait shows here, not as a run that goes wrong once in a while."""
import os
import re

import pytest

import quantized_paged_kv_q8_gb300 as k8

SOURCE = open(os.path.join(os.path.dirname(k8.__file__), "csrc", "k8v4_diff_tc.cu")).read()


def constant(name):
    return int(re.search(rf"constexpr int {name} = (\d+)", SOURCE).group(1))


class Graph:
    """Events, what each comes behind (bitsets), barriers as (name, use) with their arrivals and waits, and places in
    memory with their (tile, event, writes)."""

    def __init__(self):
        self.before, self.last, self.bars, self.waits, self.uses = [], {}, {}, [], {}

    def event(self, actor, *behind):
        i = len(self.before)
        self.before.append([x for x in (self.last.get(actor), *behind) if x is not None])
        self.last[actor] = i
        return i

    def bar(self, name, use):
        if (name, use) not in self.bars:
            self.bars[name, use] = self.event(("bar", name, use))
        return self.bars[name, use]

    def wait(self, actor, name, use):
        self.waits.append((name, use, self.event(actor, self.bar(name, use))))

    def arrive(self, actor, name, use):
        self.before[self.bar(name, use)].append(self.event(actor))

    def use(self, actor, place, tile, writes):
        self.uses.setdefault(place, []).append((tile, self.event(actor), writes))

    def closure(self):
        left = [len(x) for x in self.before]
        behind_me = [[] for _ in self.before]
        for i, xs in enumerate(self.before):
            for x in xs:
                behind_me[x].append(i)
        out, ready, seen = [0] * len(left), [i for i, n in enumerate(left) if n == 0], 0
        while ready:
            i = ready.pop()
            seen += 1
            for j in behind_me[i]:
                out[j] |= out[i] | 1 << i
                left[j] -= 1
                if left[j] == 0:
                    ready.append(j)
        assert seen == len(left), "the waits go round in a circle"
        return out

    def faults(self, phases):
        """Places used by a tile while an earlier one may still use them, and barrier phases that a later one may pass
        before a waiter has seen them (phases: uses after which a barrier comes round)."""
        behind, bad = self.closure(), set()
        for place, uses in self.uses.items():
            for ta, a, wa in uses:
                for tb, b, wb in uses:
                    if ta < tb and (wa or wb) and not behind[b] >> a & 1:
                        bad.add(place if isinstance(place, str) else place[0])
        for name, use, at in self.waits:
            later = self.bars.get((name, use + phases.get(name[0], 2)))
            if later is not None and not behind[later] >> at & 1:
                bad.add("phase of " + name[0])
        return bad


def kernel(tiles, stages, ring, moves=True):
    g = Graph()
    for i in range(tiles):
        buf = i & 1
        for c in (0, 1):
            for w in range(3):                              # copies: V rows and the valid groups, V scales, K rows and scales
                who = ("load", c, w)
                if i >= stages:
                    g.wait(who, ("raw empty", c, i % stages), i - stages)
                if w == 0:
                    g.use(who, ("valid groups", c, i % stages), i, True)
                g.use(who, ("raw", c, w, i % stages), i, True)
                g.arrive(who, ("raw full", c, i % stages), i)
            for kind in "kv":
                for w in range(4):
                    who = (kind, c, w)
                    g.wait(who, ("raw full", c, i % stages), i)
                    g.use(who, ("valid groups", c, i % stages), i, False)
                    for part in range(3):
                        g.use(who, ("raw", c, part, i % stages), i, False)
                    if i >= 2:
                        g.wait(who, ("S full", buf) if kind == "k" else ("O done", buf), i - 2)
                    g.arrive(who, ("raw empty", c, i % stages), i)
                    g.use(who, (f"{kind} tile", c, w, buf), i, True)
                    if kind == "k":
                        g.use(who, ("K scales", c, w, i % ring), i, True)
                        g.arrive(who, ("K scales full", c, i % 4), i)
                    g.arrive(who, (f"{kind} full", buf), i)
        # the issuing warp: S(i) and O(i) in either order beyond what their operands ask for
        if i:
            g.wait("issue S", ("S free",), i - 1)
        g.wait("issue S", ("k full", buf), i)
        for c in (0, 1):
            for w in range(4):
                g.use("issue S", ("k tile", c, w, buf), i, False)
                g.use("issue S", ("S", c, w), i, True)
        g.arrive("issue S", ("S full", buf), i)
        for c in (0, 1):
            for w in range(4):
                who = ("row", c, w, buf)
                g.wait(who, ("S full", buf), i)
                g.wait(who, ("K scales full", c, i % 4), i)
                g.use(who, ("S", c, w), i, False)
                g.arrive(who, ("S free",), i)
                for k in range(4):
                    g.use(who, ("K scales", c, k, i % ring), i, False)
                if i:
                    g.wait(who, ("reference", c, w, buf ^ 1), i - 1)
                g.use(who, ("reference of the rows", c, w), i, True)
                g.arrive(who, ("reference", c, w, buf), i)
                if i >= 2:
                    g.wait(who, ("O done", buf), i - 2)
                g.use(who, ("P", c, w, buf), i, True)
                if i and moves:                             # a reference that moved, or a fold: any tile may, or none
                    g.wait(who, ("O done", buf ^ 1), i - 1)
                    g.use(who, ("O", c, w), i - 0.5, True)
                    g.use(who, ("running sum", c, w), i, True)
                g.arrive(who, ("P full", buf), i)
        g.wait("issue O", ("v full", buf), i)
        g.wait("issue O", ("P full", buf), i)
        for c in (0, 1):
            for w in range(4):
                g.use("issue O", ("v tile", c, w, buf), i, False)
                g.use("issue O", ("P", c, w, buf), i, False)
                g.use("issue O", ("O", c, w), i, True)
        g.arrive("issue O", ("O done", buf), i)
    # the rows' way out lies over Q and the operand tiles
    for c in (0, 1):
        for grp in (0, 1):
            for w in range(4):
                g.wait(("row", c, w, grp), ("O done", (tiles - 1) & 1), tiles - 1)
                g.arrive(("row", c, w, grp), ("all rows", c), 0)
    for c in (0, 1):
        for grp in (0, 1):
            for w in range(4):
                g.wait(("row", c, w, grp), ("all rows", c), 0)
        for kind in "kv":
            for w in range(4):
                for buf in (0, 1):
                    g.use(("row", c, 0, 0), (f"{kind} tile", c, w, buf), tiles, True)
        for w in range(4):
            g.use(("row", c, 0, 0), ("running sum", c, w), tiles, True)
            g.use(("row", c, 0, 0), ("O", c, w), tiles, False)
    # a barrier's next use: its name holds its place, `use` counts tiles
    phases = {"raw empty": stages, "raw full": stages, "K scales full": 4, "S free": 1, "all rows": 1}
    return g.faults(phases)


@pytest.mark.parametrize("moves", [False, True])
@pytest.mark.parametrize("stages", [1, 2, 3])
@pytest.mark.parametrize("tiles", [1, 2, 3, 13])
def test_every_place_is_free_when_it_is_written(tiles, stages, moves):
    assert kernel(tiles, stages, constant("kKsRing"), moves) == set()


def test_the_graph_sees_a_ring_that_is_too_short():
    """Rows free S before they read its cells' scales: with places for four tiles the conversion of tile i could write
    over what tile i - 4's rows have yet to read, where three raw tiles let it run that far ahead."""
    for moves in (False, True):
        assert kernel(13, 3, 4, moves) == {"K scales"} and kernel(13, 2, 4, moves) == set()
