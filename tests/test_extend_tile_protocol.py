"""The orderings inside the prompt kernel of favor_decode_extend (csrc/k_decode_extend_tc.cu), checked on
the CPU as a graph of what must happen before what (no GPU code runs).

Its warps tell each other about a tile (D_r, whether it changed, the values' scale) through rings in shared
memory of ``kExtRing`` tiles, and wait on barriers by the parity of their phase. Two things have to hold for
any speed of any warp: a ring's entry is read by everyone before the tile that takes its place writes it, and
a wait is reached before its barrier completes the following phase (or the wait would never end).
The walk below follows the kernel's roles step by step; ring and stage counts are read from the source."""

import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_positive_b200",
                   "csrc", "k_decode_extend_tc.cu")
TILES = 40


def source_constants(d):
    text = open(SRC).read()
    ring = int(re.search(r"constexpr int kExtRing = (\d+);", text).group(1))
    four, two = re.search(r"NS = D == 64 \? (\d+) : (\d+);", text).groups()
    stages = int(four if d == 64 else two)
    wide, narrow, other = re.search(r"lead = NS >= (\d+) \? (\d+) : (\d+);", text).groups()
    return ring, stages, int(narrow if stages >= int(wide) else other)


class Walk:
    """Events in program order per warp; a barrier's phase completes after all its arrivals."""

    def __init__(self, d, stages, lead, flush):
        self.before = []       # per event: the events it directly follows
        self.at = {}           # warp -> its last event
        self.arrivals = {}     # (barrier, phase) -> arriving events
        self.waits = []        # (event, barrier, phase)
        self.touched = []      # (event, ring, tile, "r" or "w")
        self.flush = flush     # tiles the accumulator is taken before
        n, NS = TILES, stages
        self.blocks = d // 64
        self.scales = ("sScale6", "sScale7") if self.blocks == 2 else ("sScale",)
        self.bs = ("sB6", "sB7") if self.blocks == 2 else ("sB",)
        self.E(n)
        for w in (4, 5):
            self.keys(w, n, NS)
        for w in (6, 7):
            self.values(w, n, lead, NS)
        self.issue_p(n, NS)
        self.issue_s(n, NS)
        self.close()

    def event(self, warp):
        e = len(self.before)
        self.before.append([self.at[warp]] if warp in self.at else [])
        self.at[warp] = e
        return e

    def wait(self, warp, bar, phase):
        self.waits.append((self.event(warp), bar, phase))

    def arrive(self, warp, bar, phase):
        self.arrivals.setdefault((bar, phase), []).append(self.event(warp))

    def touch(self, warp, ring, tile, how):
        self.touched.append((self.event(warp), ring, tile, how))

    def E(self, n):  # the exponent warps (each follows the same steps)
        for g in range(n):
            self.wait("E", ("p_full", g & 1), g >> 1)
            self.touch("E", "sD", g, "w")
            self.touch("E", "sRaise", g, "w")
            self.arrive("E", ("d_full", g & 3), g >> 2)
            self.arrive("E", ("phi_full", g & 1), g >> 1)

    def take(self, warp, g):  # what warps 4-7 do at tile g
        self.wait(warp, ("d_full", g & 3), g >> 2)
        for ring in ("sRaise", "sD") + self.scales:
            self.touch(warp, ring, g, "r")
        if g in self.flush:
            k = sorted(self.flush).index(g)
            self.wait(warp, ("acc_full", 0), k)
            for ring in self.bs:
                self.touch(warp, ring, g - 1, "r")
            self.arrive(warp, ("acc_free", 0), k)

    def keys(self, w, n, NS):
        def conv(g):
            self.wait(w, ("k_full", g % NS), g // NS)
            self.arrive(w, ("k_conv", g % NS), g // NS)

        for g in range(min(2, n)):
            conv(g)
        for g in range(n):
            if g + 2 < n:
                conv(g + 2)
            self.take(w, g)

    def values(self, w, n, lead, NS):
        halves = self.blocks == 2  # each warp takes its half of every tile, else every second tile
        scale, b = (f"sScale{w}", f"sB{w}") if halves else ("sScale", "sB")

        def mine(g):
            return halves or (g & 1) == (w & 1)

        def conv(g):
            self.wait(w, ("v_full", g % NS), g // NS)
            if g > 0:
                if not halves:
                    self.wait(w, ("b_set", (g - 1) & 3), (g - 1) >> 2)
                self.touch(w, b, g - 1, "r")
            self.touch(w, b, g, "w")
            self.touch(w, scale, g, "w")
            if not halves:
                self.arrive(w, ("b_set", g & 3), g >> 2)
            self.arrive(w, ("d_full", g & 3), g >> 2)
            self.arrive(w, ("v_conv", g % NS), g // NS)

        for g in range(lead):
            if mine(g):
                conv(g)
        for g in range(n):
            if g + lead < n and mine(g + lead):
                conv(g + lead)
            self.take(w, g)

    def issue_p(self, n, NS):
        def load():
            self.arrive(8, ("k_full", self.nk % NS), self.nk // NS)
            self.nk += 1

        self.nk = 0
        while self.nk < min(NS, n):
            load()
        for i in range(n):
            self.wait(8, ("k_conv", i % NS), i // NS)
            if i >= 2:
                self.wait(8, ("s_done", i & 1), (i >> 1) - 1)
            self.arrive(8, ("p_full", i & 1), i >> 1)
            if i >= 1 and self.nk < n:
                self.wait(8, ("p_full", (i - 1) & 1), (i - 1) >> 1)
                load()

    def issue_s(self, n, NS):
        def load():
            self.arrive(9, ("v_full", self.nv % NS), self.nv // NS)
            self.nv += 1

        self.nv = 0
        while self.nv < min(NS, n):
            load()
        taken = 0
        for j in range(n):
            if j >= 1 and self.nv < n:
                self.wait(9, ("s_done", (j - 1) & 1), (j - 1) >> 1)
                load()
            self.wait(9, ("v_conv", j % NS), j // NS)
            self.wait(9, ("phi_full", j & 1), j >> 1)
            self.touch(9, "sRaise", j, "r")
            for ring in self.scales:
                self.touch(9, ring, j, "r")
            if j in self.flush:
                self.arrive(9, ("acc_full", 0), taken)
                self.wait(9, ("acc_free", 0), taken)
                taken += 1
            self.arrive(9, ("s_done", j & 1), j >> 1)

    def close(self):
        """Each event's set of predecessors (a bit mask)."""
        for e, bar, phase in self.waits:
            self.before[e] += self.arrivals[(bar, phase)]
        self.past = [None] * len(self.before)
        for root in range(len(self.before)):
            stack = [root]
            while stack:
                e = stack[-1]
                todo = [b for b in self.before[e] if self.past[b] is None]
                if self.past[e] is not None:
                    stack.pop()
                elif todo:
                    assert len(stack) < 4 * len(self.before), "the waits form a circle"
                    stack += todo
                else:
                    mask = 1 << e
                    for b in self.before[e]:
                        mask |= self.past[b]
                    self.past[e] = mask
                    stack.pop()

    def ordered(self, a, b):
        return (self.past[b] >> a) & 1 == 1

    def overwritten(self, ring):
        """(ring, tile) entries that the tile ``ring`` later may overwrite before everyone has read them."""
        writes = {(name, t): e for e, name, t, how in self.touched if how == "w"}
        bad = set()
        for e, name, t, how in self.touched:
            if how == "r":
                assert self.ordered(writes[(name, t)], e), (name, t)
                late = writes.get((name, t + ring))
                if late is not None and not self.ordered(e, late):
                    bad.add((name, t))
        return bad

    def overrun(self):
        """Waits that some barrier's next phase may pass."""
        bad = set()
        for e, bar, phase in self.waits:
            nxt = self.arrivals.get((bar, phase + 1))
            if nxt is not None and not any(self.ordered(e, a) for a in nxt):
                bad.add((bar, phase))
        return bad


FLUSHES = [set(), {16, 32}, set(range(1, TILES)), {3, 4, 5, 16, 17, 32}] + \
          [set(random.Random(s).sample(range(1, TILES), 8)) for s in range(6)]


@pytest.mark.parametrize("flush", FLUSHES)
@pytest.mark.parametrize("d", [64, 128])
def test_ring_entries_are_read_before_they_are_written_again(d, flush):
    ring, stages, lead = source_constants(d)
    walk = Walk(d, stages, lead, flush)
    assert not walk.overwritten(ring)
    assert not walk.overrun()


def test_four_entries_would_not_do():
    """The walk sees the fault that rings of four tiles had: between flushes the exponent warps come round
    to a tile's entry while a value warp still has to read it."""
    bad = Walk(64, 4, 2, set()).overwritten(4)
    assert {name for name, _ in bad} >= {"sD", "sRaise"}
