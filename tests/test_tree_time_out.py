"""Time-outs of the tensor-core tree kernel (csrc/tree_tc.cu), on the CPU: a model of a CTA in which any
wait may run out, each warp for itself.  Whatever gives up when, every warp has to come to the CTA's last
barrier."""
import os
import random
import re

import pytest

from sparse_long_context_cca_gb300 import build as cbuild


class Bar:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def done(self, parity):
        return (self.phase & 1) != (parity & 1)


class Cta:
    """Roles are generators, one per warp.  `yield cond` is a bounded wait: True once the condition holds;
    False when it does not and a wait has run out somewhere, or this one runs out.  `yield None` is a step.
    A wait looks at its condition first, then at the flag, as the kernel's does.
    joint: the warps of a half meet at an unbounded barrier before a list's parents are read.
    drain: after a time-out the producers wait for their copies behind the CTA's last barrier ("last"), or
    where they end, if they see it there ("own")."""

    def __init__(self, halves, segs, runs, joint, drain="last"):
        self.H, self.segs, self.runs, self.joint, self.drain = halves, segs, runs, joint, drain
        self.NS = n = 4 if halves == 2 else 5
        self.total = sum(segs)
        self.full, self.empty = [Bar(4) for _ in range(n)], [Bar(1) for _ in range(n)]
        self.qfull, self.ofree, self.pfull = ([Bar(4) for _ in range(halves)] for _ in range(3))
        self.sfull, self.pvdone = [Bar(2), Bar(2)], [Bar(1) for _ in range(halves)]
        self.meet = [Bar(4) for _ in range(halves)]
        self.pipe, self.flying, self.abort = [], [], False

    def tiles(self):
        x = 0
        for seg, n in enumerate(self.segs):
            yield seg, x, x + n
            x += n

    def by_tma(self, x):
        return any(x0 <= x < min(x0 + self.runs, end) for _, x0, end in self.tiles())

    def producer(self, w):
        held = None
        for u in range(2 * self.total):
            slot, bulk = u % self.NS, self.by_tma(u >> 1)
            room = lambda: self.empty[slot].done((u // self.NS & 1) ^ 1)  # noqa: E731,B023
            if held is not None and (bulk or not room()):
                yield None
                self.full[held].arrive()
                held = None
            if not (yield room):
                held = None
                break
            if bulk:
                self.flying.append(self.full[slot])
                continue
            if held is not None:
                self.full[held].arrive()
            held = slot
            yield None
        if held is not None:
            self.full[held].arrive()
        while self.drain == "own" and self.abort and self.flying:
            yield None

    def mma(self):
        H, NS, pcount = self.H, self.NS, 0
        full = lambda u: self.full[u % NS].done(u // NS)  # noqa: E731

        def scores(buf):
            self.pipe.append(self.sfull[buf])
            self.sfull[buf].arrive()

        for seg, x0, end in self.tiles():
            if H == 2:
                for h in range(2):
                    if not ((yield lambda: self.qfull[h].done(seg)) and (yield lambda: full(2 * x0))):  # noqa: B023
                        return
                    scores(h)
                self.pipe.append(self.empty[2 * x0 % NS])
                for t in range(x0, end):
                    v = 2 * t + 1
                    if not (yield lambda: full(v)):  # noqa: B023
                        return
                    for h in range(2):
                        if not (yield lambda: self.pfull[h].done(pcount)):  # noqa: B023
                            return
                        if t == x0 and not (yield lambda: self.ofree[h].done(seg + 1)):  # noqa: B023
                            return
                        if t + 1 < end:
                            if not (yield lambda: full(v + 1)):  # noqa: B023
                                return
                            scores(h)
                        else:
                            self.pipe.append(self.pvdone[h])
                    self.pipe.append(self.empty[v % NS])
                    if t + 1 < end:
                        self.pipe.append(self.empty[(v + 1) % NS])
                    pcount += 1
            else:
                if not (yield lambda: self.qfull[0].done(seg)):  # noqa: B023
                    return
                for t in range(x0, end + 1):
                    if t < end:
                        if not (yield lambda: full(2 * t)):  # noqa: B023
                            return
                        scores(t & 1)
                        self.pipe.append(self.empty[2 * t % NS])
                    if t == x0:
                        continue
                    v = 2 * t - 1
                    if not ((yield lambda: full(v)) and (yield lambda: self.pfull[0].done(pcount))):  # noqa: B023
                        return
                    if t - 1 == x0 and not (yield lambda: self.ofree[0].done(seg + 1)):  # noqa: B023
                        return
                    self.pipe += [self.pvdone[0], self.empty[v % NS]]
                    pcount += 1

    def parents(self, h, n):
        """Before the n-th list's tree is read."""
        if self.joint:
            self.meet[h].arrive()
            while not self.meet[h].done(n):
                yield "unbounded"

    def softmax(self, h):
        n_s, NS, segs = 0, self.NS, list(self.tiles())
        self.qfull[h].arrive()
        yield from self.parents(h, 0)
        for seg, x0, end in segs:
            for t in range(x0, end):
                buf, v = (h, 2 * t + 1) if self.H == 2 else (t & 1, 2 * t + 1)
                if not (yield lambda: self.sfull[buf].done(n_s if self.H == 2 else n_s >> 1)):  # noqa: B023
                    return
                if not self.by_tma(t) and not (yield lambda: self.full[v % NS].done(v // NS)):  # noqa: B023
                    return
                if self.H == 1 and n_s > 0 and not (yield lambda: self.pvdone[0].done(n_s + 1)):  # noqa: B023
                    return
                self.pfull[h].arrive()
                n_s += 1
                yield None
            if seg + 1 < len(segs):
                self.qfull[h].arrive()
            if not (yield lambda: self.pvdone[h].done(seg if self.H == 2 else n_s + 1)):  # noqa: B023
                return
            yield None
            self.ofree[h].arrive()
            if seg + 1 < len(segs):
                yield from self.parents(h, seg + 1)

    def run(self, rng, patience):
        """True when every warp has come to the end.  patience: how rarely a wait runs out."""
        warps = [self.producer(w) for w in range(4)] + [self.mma()] + [self.softmax(h) for h in range(self.H) for _ in range(4)]
        state = {i: (w, next(w, "end")) for i, w in enumerate(warps)}
        for _ in range(200000):
            if self.pipe and rng.random() < 0.3:
                self.pipe.pop(0).arrive()
            if self.flying and rng.random() < 0.3:
                self.flying.pop(rng.randrange(len(self.flying))).arrive()
            live = [i for i, s in state.items() if s[1] != "end"]
            if not live:
                # the CTA's last barrier; behind it the producers that gave up wait for what still flies
                self.left = 0 if self.abort and self.drain == "last" else len(self.flying)
                return True
            # unbounded barriers that nothing can complete any more: the CTA hangs
            if all(state[i][1] == "unbounded" for i in live) and not self.pipe and not self.flying:
                for i in live:
                    state[i] = (state[i][0], next(state[i][0], "end"))
                if all(state[i][1] == "unbounded" for i in live if state[i][1] != "end"):
                    return not [i for i in live if state[i][1] != "end"]
                continue
            i = rng.choice(live)
            warp, cond = state[i]
            try:
                if cond is None or cond == "unbounded":
                    state[i] = (warp, warp.send(None))
                elif cond():
                    state[i] = (warp, warp.send(True))
                elif self.abort:
                    state[i] = (warp, warp.send(False))
                elif rng.random() < patience:
                    self.abort = True
                    state[i] = (warp, warp.send(False))
            except StopIteration:
                state[i] = (warp, "end")
        return False


SEGS = [[1], [2, 1], [1, 1, 1, 1], [2, 7, 1, 5], [1, 2, 3, 4, 5, 6]]


@pytest.mark.parametrize("halves", [1, 2])
@pytest.mark.parametrize("segs", SEGS)
@pytest.mark.parametrize("runs", [0, 2, 100])
def test_every_warp_ends_whatever_runs_out(halves, segs, runs):
    for seed in range(60):
        rng = random.Random(seed)
        assert Cta(halves, segs, runs, joint=False).run(rng, 10.0 ** -(1 + seed % 3)), seed
    assert Cta(halves, segs, runs, joint=False).run(random.Random(0), 0.0)     # and where nothing does


def test_a_barrier_among_warps_that_may_disagree_hangs():
    """What the kernel must not have: some schedule leaves one warp at the barrier for good."""
    assert all(Cta(1, [1, 1, 1, 1], 0, joint=True).run(random.Random(s), 0.0) for s in range(20))
    assert not all(Cta(1, [1, 1, 1, 1], 0, joint=True).run(random.Random(s), 10.0 ** -(1 + s % 3)) for s in range(400))


def test_no_copy_outlives_the_cta():
    def left(drain, patience):
        out = []
        for seed in range(300):
            cta = Cta(1 + seed % 2, SEGS[seed % len(SEGS)], 100, False, drain)
            assert cta.run(random.Random(seed), patience)
            out.append(cta.left)
        return out

    assert not any(left("last", 0.03)) and not any(left("last", 0.0)) and any(left("own", 0.03))
    source = open(os.path.join(cbuild.CSRC, "tree_tc.cu")).read()
    code = re.sub(r"//[^\n]*", "", source)
    # the wait for the copies stands behind the last barrier
    assert code.rindex("__syncthreads()") < code.index("last_bulk >= NS")


def test_the_kernel_has_no_such_barrier():
    source = open(os.path.join(cbuild.CSRC, "tree_tc.cu")).read()
    code = re.sub(r"//[^\n]*", "", source)
    assert not re.search(r"named_bar|bar\.sync|barrier\.sync|__syncthreads_|__barrier", code)
    assert len(re.findall(r"__syncthreads\(\)", code)) == 2          # after the set-up, and at the end
    waits = re.findall(r"mbar_\w*wait\w*|wait_bounded", code)
    assert waits.count("mbar_try_wait") == 1                         # a look, not a wait
    assert all(w in ("mbar_try_wait", "wait_bounded") for w in waits)
