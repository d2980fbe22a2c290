"""Barrier-level models of the packed gradient kernels (packed_bwd_tc.cu), run on the CPU.

The models follow the kernels' schedules: the producer's rings, the issuer's order of products and commits,
the element-wise warps, and a tensor pipe that executes what was issued in order, some time later.  Every wait
names the phase that it expects; buffers remember what was put into them, and each reader checks that it finds
what it expects.  The processes are interleaved in seeded random order; a state in which none can move is a
deadlock.  With one barrier for dS and two buffers, for instance, a warp that is ahead can arrive for one that
is not, and the product reads a tile that is not finished."""
import os
import random
import re

import pytest

WARPS = 3  # of the kernel's eight
SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_long_context_cca_gb300", "csrc", "packed_bwd_tc.cu")


def test_model_constants_match_the_kernel():
    found = dict(re.findall(r"(LONG_ST|SHORT_ST) = (\d+)", open(SRC).read()))
    assert found == {"LONG_ST": str(LONG), "SHORT_ST": str(SHORT)}


LONG, SHORT = 3, 2


class Bar:
    def __init__(self, name, count=1):
        self.name, self.count, self.left, self.phases = name, count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phases = self.count, self.phases + 1


def simulate(procs, seed):
    """procs: {name: generator of waits (bar, phases) or predicates}; returns what is stuck, or None."""
    rng, waiting = random.Random(seed), dict.fromkeys(procs)
    while any(n != "pipe" for n in procs):
        moved = False
        for name in rng.sample(sorted(procs), len(procs)):
            for _ in range(rng.randint(1, 4)):
                w = waiting[name]
                if callable(w):
                    if not w():
                        break
                elif w is not None:
                    bar, phase = w
                    if bar.phases < phase:
                        break
                    assert bar.phases == phase, (name, bar.name, bar.phases, phase)   # a wait sees a parity alone
                waiting[name] = None
                moved = True
                try:
                    waiting[name] = next(procs[name])
                except StopIteration:
                    del procs[name]
                    break
        if not moved:
            return {n: getattr(waiting[n][0], "name", "?") if isinstance(waiting[n], tuple) else "poll" for n in procs}
    return None


class Pipe:
    """Executes in order; a commit arrives once everything before it is done."""

    def __init__(self):
        self.queue = []

    def issue(self, what):
        self.queue.append(what)

    def commit(self, bar):
        self.queue.append(bar.arrive)

    def run(self):
        while True:
            yield lambda: bool(self.queue)
            self.queue.pop(0)()


def run_dq(tiles, seed):
    """tiles[i]: key tiles of item i."""
    B = {n: Bar(n, WARPS if n in ("read", "ds", "accfree", "qt") else 1)
         for n in ("res", "resfree", "read", "dp", "ds", "dsfree", "done", "accfree", "q", "qt")}
    lfull, lempty = [Bar(f"lfull{s}") for s in range(LONG)], [Bar(f"lempty{s}") for s in range(LONG)]
    sfull, sempty = [Bar(f"sfull{s}") for s in range(SHORT)], [Bar(f"sempty{s}") for s in range(SHORT)]
    smem = {"q": None, "do": None, "k": [None] * LONG, "v": [None] * SHORT}
    tmem = {"s": None, "dp": None, "dq": None, "ds": [None] * WARPS, "q": [None] * WARPS}
    out = []
    pipe = Pipe()

    def expect(got, want):
        def check():
            assert got() == want, (got(), want)
        return check

    def producer():
        g = 0
        for it, T in enumerate(tiles):
            yield B["qt"], it
            smem["q"] = it
            B["q"].arrive()
            yield B["resfree"], it
            smem["do"] = it
            B["res"].arrive()
            for _ in range(T):
                yield lempty[g % LONG], g // LONG
                smem["k"][g % LONG] = g
                lfull[g % LONG].arrive()
                yield sempty[g % SHORT], g // SHORT
                smem["v"][g % SHORT] = g
                sfull[g % SHORT].arrive()
                g += 1

    def issuer():
        g = 0

        def products(g, it, first):
            yield lfull[g % LONG], g // LONG + 1
            if first:
                yield B["qt"], it + 1
            if g > 0:
                yield B["read"], g

            def s():
                assert smem["k"][g % LONG] == g and tmem["q"] == [it] * WARPS
                tmem["s"] = g
            pipe.issue(s)
            yield sfull[g % SHORT], g // SHORT + 1
            if first:
                yield B["res"], it + 1

            def dp():
                assert smem["v"][g % SHORT] == g and smem["do"] == it
                tmem["dp"] = g
            pipe.issue(dp)
            pipe.commit(B["dp"])
            pipe.commit(sempty[g % SHORT])

        for it, T in enumerate(tiles):
            yield from products(g, it, True)
            for x in range(T):
                if x + 1 < T:
                    yield from products(g + 1, it, False)
                else:
                    pipe.commit(B["resfree"])
                yield B["ds"], g + 1
                if x == 0:
                    yield B["accfree"], it

                def dq(g=g, it=it, x=x):
                    assert tmem["ds"] == [g] * WARPS and smem["k"][g % LONG] == g
                    if x == 0:
                        tmem["dq"] = (it, 0)
                    assert tmem["dq"] == (it, x)
                    tmem["dq"] = (it, x + 1)
                pipe.issue(dq)
                pipe.commit(B["dsfree"])
                pipe.commit(lempty[g % LONG])
                g += 1
            pipe.commit(B["done"])

    def warp(w):
        g = 0

        def copy_q(it):
            yield B["q"], it + 1
            assert smem["q"] == it
            tmem["q"][w] = it
            B["qt"].arrive()
        if tiles:
            yield from copy_q(0)
        for it, T in enumerate(tiles):
            for _ in range(T):
                yield B["dp"], g + 1
                assert tmem["s"] == g and tmem["dp"] == g
                B["read"].arrive()
                if g > 0:
                    yield B["dsfree"], g
                tmem["ds"][w] = g
                B["ds"].arrive()
                g += 1
            if it + 1 < len(tiles):
                yield from copy_q(it + 1)
            yield B["done"], it + 1
            assert tmem["dq"] == (it, T)
            out.append((it, w))
            B["accfree"].arrive()

    procs = {"producer": producer(), "issuer": issuer(), "pipe": pipe.run(), **{f"warp{w}": warp(w) for w in range(WARPS)}}
    stuck = simulate(procs, seed)
    if stuck is None:
        assert sorted(out) == [(it, w) for it in range(len(tiles)) for w in range(WARPS)]
    return stuck


def run_dkv(tiles, seed, by_need=False):
    """tiles[i]: (query tile, head) pairs of item i; there may be none.  by_need: the producer hands the items' numbers on, and
    None is an item that all pass over."""
    END = len(tiles)
    item, itemfree = [Bar("item0"), Bar("item1")], [Bar("itemfree0", 2), Bar("itemfree1", 2)]
    number, cur = [None, None], [None]

    B = {n: Bar(n, WARPS if n in ("p", "ds", "accfree", "named") else 1)
         for n in ("res", "resfree", "s", "p", "dp", "ds", "done", "accfree", "named")}
    lfull, lempty = [Bar(f"lfull{s}") for s in range(LONG)], [Bar(f"lempty{s}") for s in range(LONG)]
    sfull, sempty = [Bar(f"sfull{s}") for s in range(SHORT)], [Bar(f"sempty{s}") for s in range(SHORT)]
    smem = {"kv": None, "q": [None] * LONG, "do": [None] * SHORT, "slot": [None] * WARPS}
    tmem = {"s": [None] * WARPS, "dp": [None] * WARPS, "dk": None, "dv": None}   # per warp: ("s" or "p", tile)
    out, pipe = [], Pipe()

    def producer():
        g = nr = 0
        for it in range(END + 1):
            if by_need:
                yield itemfree[it & 1], it // 2
                number[it & 1] = it
                item[it & 1].arrive()
            n = tiles[it] if it < END else None
            if not n:
                continue
            yield B["resfree"], nr
            smem["kv"] = it
            B["res"].arrive()
            nr += 1
            for _ in range(n):
                yield lempty[g % LONG], g // LONG
                smem["q"][g % LONG] = g
                lfull[g % LONG].arrive()
                yield sempty[g % SHORT], g // SHORT
                smem["do"][g % SHORT] = g
                sfull[g % SHORT].arrive()
                g += 1

    def issuer():
        g = nr = 0

        def issue_s(g, it):
            yield lfull[g % LONG], g // LONG + 1

            def s():
                assert smem["kv"] == it and smem["q"][g % LONG] == g
                tmem["s"] = [("s", g)] * WARPS
            pipe.issue(s)
            pipe.commit(B["s"])

        def issue_dp(g, it):
            yield sfull[g % SHORT], g // SHORT + 1

            def dp():
                assert smem["kv"] == it and smem["do"][g % SHORT] == g
                tmem["dp"] = [("dp", g)] * WARPS
            pipe.issue(dp)
            pipe.commit(B["dp"])

        done = 0
        for it in range(END + 1):
            if by_need:
                yield item[it & 1], it // 2 + 1
                assert number[it & 1] == it
                itemfree[it & 1].arrive()
            n = tiles[it] if it < END else None
            if n is None:
                continue
            if n > 0:
                yield B["res"], nr + 1
                yield from issue_s(g, it)
                yield from issue_dp(g, it)
                nr += 1
                if n == 1:
                    pipe.commit(B["resfree"])
            else:
                yield B["accfree"], done
            for x in range(n):
                yield B["p"], g + 1
                if x == 0:
                    yield B["accfree"], done

                def dv(g=g, it=it, x=x):
                    assert tmem["s"] == [("p", g)] * WARPS and smem["do"][g % SHORT] == g
                    assert x == 0 or tmem["dv"] == (it, x)
                    tmem["dv"] = (it, x + 1)
                pipe.issue(dv)
                pipe.commit(sempty[g % SHORT])
                if x + 1 < n:
                    yield from issue_s(g + 1, it)
                yield B["ds"], g + 1

                def dk(g=g, it=it, x=x):
                    assert tmem["dp"] == [("ds", g)] * WARPS and smem["q"][g % LONG] == g
                    assert x == 0 or tmem["dk"] == (it, x)
                    tmem["dk"] = (it, x + 1)
                pipe.issue(dk)
                pipe.commit(lempty[g % LONG])
                if x + 1 < n:
                    yield from issue_dp(g + 1, it)
                    if x + 2 == n:
                        pipe.commit(B["resfree"])
                g += 1
            pipe.commit(B["done"])
            done += 1

    def warp(w):
        g = named = done = 0
        for it in range(END + 1):
            if by_need:
                if w == 0:
                    yield item[it & 1], it // 2 + 1
                    cur[0] = number[it & 1]
                    itemfree[it & 1].arrive()
                for read in (True, False):      # the second barrier: every warp has read it
                    B["named"].arrive()
                    named += 1
                    yield B["named"], named
                    assert not read or cur[0] == it
            n = tiles[it] if it < END else None
            if n is None:
                continue
            if n > 0:
                smem["slot"][w] = g
            B["named"].arrive()
            named += 1
            yield B["named"], named
            for x in range(n):
                yield B["s"], g + 1
                assert tmem["s"][w] == ("s", g) and smem["slot"] == [g] * WARPS
                tmem["s"][w] = ("p", g)
                B["p"].arrive()
                yield B["dp"], g + 1
                assert tmem["dp"][w] == ("dp", g) and smem["slot"] == [g] * WARPS
                tmem["dp"][w] = ("ds", g)
                B["ds"].arrive()
                for move in (True, False):
                    B["named"].arrive()
                    named += 1
                    yield B["named"], named
                    if move:
                        smem["slot"][w] = g + 1 if x + 1 < n else None
                g += 1
            yield B["done"], done + 1
            done += 1
            assert n == 0 or tmem["dk"] == tmem["dv"] == (it, n)
            out.append((it, w))
            B["accfree"].arrive()

    procs = {"producer": producer(), "issuer": issuer(), "pipe": pipe.run(), **{f"warp{w}": warp(w) for w in range(WARPS)}}
    stuck = simulate(procs, seed)
    if stuck is None:
        assert sorted(out) == [(it, w) for it in range(len(tiles)) if tiles[it] is not None for w in range(WARPS)]
    return stuck


ITEMS = [[1], [2], [1, 1, 1, 1], [5, 4, 3, 2, 1], [7, 1, 6, 1, 2, 9], [3] * 6]


@pytest.mark.parametrize("tiles", ITEMS, ids=str)
def test_dq(tiles):
    for seed in range(60):
        assert run_dq(tiles, seed) is None


@pytest.mark.parametrize("tiles", ITEMS + [[0], [0, 2, 0, 0, 1], [4, 0, 3, 0]], ids=str)
def test_dkv(tiles):
    for seed in range(60):
        assert run_dkv(tiles, seed) is None
        assert run_dkv(tiles, seed, True) is None


@pytest.mark.parametrize("tiles", [[], [None], [3, None, 1, None, None, 0, 2], [None, None, 4, 0, None]], ids=str)
def test_dkv_items_handed_on(tiles):
    for seed in range(60):
        assert run_dkv(tiles, seed, True) is None
