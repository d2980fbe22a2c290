"""A barrier-level model of the tensor-core tree kernel (csrc/tree_tc.cu): producers, MMA issuer, the
in-order tensor pipe and the softmax groups as coroutines under random schedules.  Every run has to
end, every operand has to be the one that the step means, and nothing may be overwritten while a
reader still needs it."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def done(self, parity):
        return (self.phase & 1) != (parity & 1)


class Model:
    """One CTA.  segs: tiles of each list in its run, the first runs[i] of them copied by TMA (they
    land by themselves), the others by the producers' own copies.  Roles are generators that yield a condition to
    wait for, or None for a step."""

    def __init__(self, halves, segs, used=None, runs=0, slots=None, metas=4):
        self.H, self.segs = halves, segs
        self.run_tiles = {x + i for _, x, end in self.tiles() for i in range(min(runs, end - x))}
        self.flying, self.loaders = [], 4    # TMA copies in flight, producers at work
        self.NS = slots or (4 if halves == 2 else 5)
        self.used = [True] * halves if used is None else used
        n = self.NS
        self.full, self.empty = [Bar(4) for _ in range(n)], [Bar(1) for _ in range(n)]
        self.qfull, self.ofree = [Bar(1) for _ in range(halves)], [Bar(1) for _ in range(halves)]
        self.sfull, self.pfull = [Bar(2), Bar(2)], [Bar(1) for _ in range(halves)]
        self.pvdone = [Bar(1) for _ in range(halves)]
        self.slot = [None] * n               # (what, tile) that has landed
        self.meta = [None] * metas
        self.q = [None] * halves             # list whose queries are in shared memory
        self.s = [None, None]                # score buffers: ("S" | "P", half, tile)
        self.o = [None] * halves             # last tile added to O, and its list
        self.pipe = []                       # tensor pipe, in order
        self.out = []

    def tiles(self):
        x = 0
        for seg, n in enumerate(self.segs):
            yield seg, x, x + n
            x += n

    def producer(self, w):
        total, NS, held = sum(self.segs), self.NS, None

        def land(p):
            slot, what = p
            if w == 0:
                self.slot[slot] = what
            self.full[slot].arrive()

        for u in range(2 * total):
            x, slot = u >> 1, u % NS
            what, runs = ("V" if u & 1 else "K", x), x in self.run_tiles
            ready = lambda: self.empty[slot].done((u // NS & 1) ^ 1)  # noqa: E731,B023
            if held is not None and (runs or not ready()):
                yield None
                land(held)
                held = None
            yield ready
            if w == 0:
                self.slot[slot] = "loading"
                if not u & 1:
                    self.meta[x % len(self.meta)] = x
            yield None
            if runs:
                self.flying.append(lambda p=(slot, what): land(p))
                continue
            if held is not None:
                land(held)
            held = (slot, what)
        if held is not None:
            yield None
            land(held)
        self.loaders -= 1

    def tma(self, rng):
        while self.loaders or self.flying:
            yield lambda: bool(self.flying) or not self.loaders
            if self.flying:
                self.flying.pop(rng.randrange(len(self.flying)))()

    def issue(self, *op):
        self.pipe.append(op)

    def pipe_role(self):
        while True:
            yield lambda: bool(self.pipe)
            op = self.pipe.pop(0)
            if op[0] == "S":
                _, h, t, buf, ks, seg = op
                assert self.slot[ks] == ("K", t) and self.q[h] == seg
                self.s[buf] = "writing"
                yield None
                assert self.slot[ks] == ("K", t) and self.q[h] == seg
                self.s[buf] = ("S", h, t)
            elif op[0] == "PV":
                _, h, t, buf, vs, first = op
                assert self.s[buf] == ("P", h, t) and self.slot[vs] == ("V", t)
                yield None
                assert self.s[buf] == ("P", h, t) and self.slot[vs] == ("V", t)
                assert self.o[h] == ("free" if first else t - 1), (self.o, op)
                self.o[h] = t
            elif op[0] == "commit":
                op[1].arrive()
            elif op[0] == "end":
                return

    def mma(self):
        H, NS = self.H, self.NS
        pcount = 0
        for seg, x0, end in self.tiles():
            if H == 2:
                u = 2 * x0
                for h in range(2):
                    if not self.used[h]:
                        continue
                    yield lambda: self.qfull[h].done(seg)  # noqa: B023
                    yield lambda: self.full[u % NS].done(u // NS)  # noqa: B023
                    self.issue("S", h, x0, h, u % NS, seg)
                    self.issue("commit", self.sfull[h])
                    self.sfull[h].arrive()
                self.issue("commit", self.empty[u % NS])
                for t in range(x0, end):
                    v = 2 * t + 1
                    yield lambda: self.full[v % NS].done(v // NS)  # noqa: B023
                    for h in range(2):
                        if not self.used[h]:
                            continue
                        yield lambda: self.pfull[h].done(pcount)  # noqa: B023
                        if t == x0:
                            yield lambda: self.ofree[h].done(seg + 1)  # noqa: B023
                            self.issue_first(h)
                        self.issue("PV", h, t, h, v % NS, t == x0)
                        if t + 1 < end:
                            yield lambda: self.full[(v + 1) % NS].done((v + 1) // NS)  # noqa: B023
                            self.issue("S", h, t + 1, h, (v + 1) % NS, seg)
                            self.issue("commit", self.sfull[h])
                            self.sfull[h].arrive()
                        else:
                            self.issue("commit", self.pvdone[h])
                    self.issue("commit", self.empty[v % NS])
                    if t + 1 < end:
                        self.issue("commit", self.empty[(v + 1) % NS])
                    pcount += 1
            else:
                yield lambda: self.qfull[0].done(seg)  # noqa: B023
                for t in range(x0, end + 1):
                    if t < end:
                        u = 2 * t
                        yield lambda: self.full[u % NS].done(u // NS)  # noqa: B023
                        self.issue("S", 0, t, t & 1, u % NS, seg)
                        self.issue("commit", self.sfull[t & 1])
                        self.sfull[t & 1].arrive()
                        self.issue("commit", self.empty[u % NS])
                    if t == x0:
                        continue
                    v = 2 * (t - 1) + 1
                    yield lambda: self.full[v % NS].done(v // NS)  # noqa: B023
                    yield lambda: self.pfull[0].done(pcount)  # noqa: B023
                    if t - 1 == x0:
                        yield lambda: self.ofree[0].done(seg + 1)  # noqa: B023
                        self.issue_first(0)
                    self.issue("PV", 0, t - 1, (t - 1) & 1, v % NS, t - 1 == x0)
                    self.issue("commit", self.pvdone[0])
                    self.issue("commit", self.empty[v % NS])
                    pcount += 1
        self.issue("end")

    def issue_first(self, h):
        # the output of the list before has been read
        assert self.o[h] in (None, "read")
        self.o[h] = "free"

    def softmax(self, h):
        NS, n_s = self.NS, 0
        segs = list(self.tiles())
        self.q[h] = 0
        self.qfull[h].arrive()
        for seg, x0, end in segs:
            for t in range(x0, end):
                buf = h if self.H == 2 else t & 1
                v = 2 * t + 1
                yield lambda: self.sfull[buf].done(n_s if self.H == 2 else n_s >> 1)  # noqa: B023
                if t not in self.run_tiles:
                    yield lambda: self.full[v % NS].done(v // NS)  # noqa: B023
                    assert self.slot[v % NS] == ("V", t)
                assert self.s[buf] == ("S", h, t) and self.meta[t % len(self.meta)] == t
                if t + 1 == end and seg + 1 < len(segs):
                    self.q[h] = seg + 1      # the next list's queries, handed over after this tile
                yield None
                if self.H == 1 and n_s > 0 and t > x0 and random.random() < 0.5:   # a rescale of O
                    yield lambda: self.pvdone[0].done(n_s + 1)  # noqa: B023
                    assert self.o[0] == t - 1
                elif self.H == 2 and t > x0:
                    assert self.o[h] == t - 1
                assert self.s[buf] == ("S", h, t) and self.meta[t % len(self.meta)] == t
                self.s[buf] = ("P", h, t)
                if self.H == 1 and n_s > 0:
                    yield lambda: self.pvdone[0].done(n_s + 1)  # noqa: B023
                self.pfull[h].arrive()
                n_s += 1
                yield None
            if seg + 1 < len(segs):
                self.qfull[h].arrive()
            yield lambda: self.pvdone[h].done(seg if self.H == 2 else n_s + 1)  # noqa: B023
            assert self.o[h] == end - 1
            self.out.append((h, seg))
            self.o[h] = "read"
            self.ofree[h].arrive()

    def run(self, rng):
        roles = [self.producer(w) for w in range(4)] + [self.mma(), self.pipe_role(), self.tma(rng)]
        roles += [self.softmax(h) for h in range(self.H) if self.used[h]]
        state = {i: (r, next(r, "end")) for i, r in enumerate(roles)}
        while True:
            live = {i: s for i, s in state.items() if s[1] != "end"}
            if not live:
                break
            ready = [i for i, (r, c) in live.items() if c is None or c()]
            assert ready, f"every role waits: {sorted(live)} of {len(roles)}"
            i = rng.choice(ready)
            state[i] = (roles[i], next(roles[i], "end"))
        assert sorted(self.out) == sorted((h, s) for h in range(self.H) if self.used[h] for s in range(len(self.segs)))


@pytest.mark.parametrize("runs", [0, 1, 4, 100])
@pytest.mark.parametrize("halves,used", [(1, None), (2, None), (2, [True, False])])
@pytest.mark.parametrize("segs", [[1], [2], [3, 1], [9], [1, 1, 1, 1], [2, 7, 1, 5], [30, 3], [1, 2, 3, 4, 5, 6]])
def test_every_schedule_ends(halves, used, segs, runs):
    for seed in range(30):
        random.seed(seed)
        Model(halves, segs, used, runs).run(random.Random(seed))


@pytest.mark.parametrize("halves", [1, 2])
@pytest.mark.parametrize("slots", [4, 5, 8])
@pytest.mark.parametrize("segs", [[1], [9], [3, 1], [2, 7, 1, 5], [30, 3], [1, 2, 3, 4, 5, 6]])
def test_every_ring_depth_ends(halves, segs, slots):
    """Eight sets of a tile's bits are enough for a ring of four tiles, as d = 64 has it."""
    for runs in (0, 2, 100):
        for seed in range(15):
            random.seed(seed)
            Model(halves, segs, None, runs, slots, 8).run(random.Random(seed))
