"""Barrier-level models of the packed kernels' producers (attn_packed_tc.cu, packed_bwd_tc.cu), run on the CPU: tiles that
end behind their sequence, which the producer waits for, clears and hands over by an arrival of its own, and the copies
that are under way when a wait runs out.

Copies are posted and land later, in any order; a barrier completes a phase once its arrivals and its copies' bytes are
there; a wait sees a parity alone, and gives up once the CTA's abort flag is set, unless it is one that only time ends.  The
tensor pipe executes in order, some time later.  Checked: every product finds the tile that it expects, cleared where
its sequence ends inside; no state in which nobody can move; and, whenever the flag is set, a CTA that
ends with no copy and no product under way."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_long_context_cca_gb300", "csrc")
BN, NS, LONG, SHORT = 128, 5, 3, 2


def source(name):
    return open(os.path.join(CSRC, name)).read()


def test_the_models_are_of_these_kernels():
    attn, bwd = source("attn_packed_tc.cu"), source("packed_bwd_tc.cu")
    assert dict(re.findall(r"constexpr int (BM|BN|NS) = (\d+);", attn)) == {"BM": "128", "BN": "128", "NS": str(NS)}
    assert dict(re.findall(r"(LONG_ST|SHORT_ST) = (\d+)", bwd)) == {"LONG_ST": str(LONG), "SHORT_ST": str(SHORT)}
    # the producers wait for their copies whether or not the flag is set when they look
    for text in (attn, bwd):
        for line in re.findall(r"if \(\*[a-z.]*abort_flag.*", text):
            assert "report(" in line, line


def test_the_contiguous_kernel_waits_for_its_copies_at_its_end():
    # behind the barrier that all warps come to, so that the flag is what it will be
    text = source("attn_tc.cu")
    at = text.index("The copies already issued land before the CTA exits")
    assert "__syncthreads();\n    if (*abort_flag && threadIdx.x == 0) {" in text[at - 200:at] and text.count("if (*abort_flag") == 1


class Bar:
    def __init__(self, name, count=1):
        self.name, self.count, self.left, self.bytes, self.phases = name, count, count, 0, 0

    def check(self):
        if self.left == 0 and self.bytes == 0:
            self.left, self.phases = self.count, self.phases + 1

    def arrive(self, expect=0):
        self.bytes += expect
        self.left -= 1
        assert self.left >= 0, self.name
        self.check()

    def land(self, n):
        self.bytes -= n
        self.check()

    def passed(self, parity):
        return (self.phases & 1) != parity


class Cta:
    """The processes of a CTA, its copies and its tensor pipe, interleaved at random."""

    def __init__(self, seed, abort_at=None):
        self.rng, self.copies, self.pipe, self.aborted, self.abort_at, self.steps = random.Random(seed), [], [], False, abort_at, 0

    def copy(self, bar, effect, n=1):
        self.copies.append((bar, effect, n))

    def issue(self, what):
        self.pipe.append(what)

    def commit(self, bar):
        self.pipe.append(bar.arrive)

    def expect(self, got, want):
        assert self.aborted or got == want, (got, want)

    def run(self, procs):
        waiting, answer = dict.fromkeys(procs), dict.fromkeys(procs)
        while procs:
            moved = False
            self.steps += 1
            if self.abort_at is not None and self.steps >= self.abort_at:
                self.aborted = True
            for name in self.rng.sample(sorted(procs), len(procs)):
                for _ in range(self.rng.randint(1, 4)):
                    w = waiting[name]
                    if w is not None:
                        bar, parity, gives_up = w
                        if bar.passed(parity):
                            answer[name] = True
                        elif self.aborted and gives_up:
                            answer[name] = False
                        else:
                            break
                    try:
                        waiting[name] = procs[name].send(answer[name] if w is not None else None)
                        moved = True
                    except StopIteration:
                        del procs[name]
                        moved = True
                        break
            for _ in range(self.rng.randint(0, 2)):
                if self.copies:
                    bar, effect, n = self.copies.pop(self.rng.randrange(len(self.copies)))
                    effect()
                    bar.land(n)
                    moved = True
            for _ in range(self.rng.randint(0, 2)):
                if self.pipe:
                    self.pipe.pop(0)()
                    moved = True
            if not moved and not self.copies and not self.pipe:
                late = [n for n in procs if not waiting[n][2]]
                if not late:
                    return {n: waiting[n][0].name for n in procs}
                assert self.aborted, late      # a wait that only time ends, for something that never comes: only after an abort
                for n in late:
                    try:
                        waiting[n] = procs[n].send(False)
                    except StopIteration:
                        del procs[n]
        # the CTA ends here
        assert not self.copies and not self.pipe, (len(self.copies), len(self.pipe))
        return None


# ---------------------------------------------------------------- attention

class Item:
    """256 rows of a sequence of n (or fewer of each of several heads), as make_item cuts them."""

    def __init__(self, n, pair, g, w, mode, lr):
        lo = lambda i: max(0, i - w + 1)                          # noqa: E731
        start = lambda i: lo(i) // g * g if mode else lo(i)       # noqa: E731
        rows, i0 = 1 << lr, pair * 256
        self.n, self.groups, self.lo0 = n, n // g, start(i0)
        self.valid, self.tc, self.kl, self.kh, last = [], [], [], [], i0
        for a in (i0, i0 + rows):
            b = min(a + rows, n) - 1
            self.valid.append(a < n)
            if a < n:
                last = b
            self.tc.append(-(-(lo(b) // g) // BN) if a < n else 0)
            self.kl.append((start(a) - self.lo0) // BN if a < n else 0)
            self.kh.append((b - self.lo0) // BN + 1 if a < n else 0)
        self.Tc = max(self.tc)
        self.T = self.Tc + (last - self.lo0) // BN + 1

    def uses(self, h, t):
        return self.valid[h] and (t < self.tc[h] if t < self.Tc else self.kl[h] <= t - self.Tc < self.kh[h])

    def first(self, h):
        return 0 if self.tc[h] > 0 else self.Tc + self.kl[h]

    def next(self, h, t):
        if t < self.Tc:
            return t + 1 if t + 1 < self.tc[h] else self.Tc + self.kl[h]
        return t + 1 if t + 1 < self.Tc + self.kh[h] else -1

    def left(self, t):
        """Keys of the sequence from the tile's first one on."""
        return self.groups - t * BN if t < self.Tc else self.n - self.lo0 - (t - self.Tc) * BN


def items_of(lens, g, w, mode, heads=2, share=0):
    out = []
    for p in range(max(-(-n // 256) for n in lens) - 1, -1, -1):
        for n in sorted(lens, reverse=True):
            if n > p * 256:
                lr = next((7 - c for c in range(share, 0, -1) if n <= 256 >> c), 7)
                out += [Item(n, p, g, w, mode, lr) for _ in range(max(1, heads >> (7 - lr)))]
    return out


def run_attention(items, seed, abort_at=None, drain="always"):
    c = Cta(seed, abort_at)
    qfull, qfree, cut_bar, drained = Bar("qfull"), Bar("qfree"), Bar("cut"), Bar("drain")
    full, empty = [Bar(f"full{s}") for s in range(NS)], [Bar(f"empty{s}") for s in range(NS)]
    sfull, pfull, pvdone, ofree = ([Bar(n + h) for h in "AB"] for n in ("sfull", "pfull", "pvdone", "ofree"))
    slot, q_item = [None] * NS, [None]
    s_tile = [None, None]

    def put(at, what):
        return lambda: slot.__setitem__(at, what)

    def producer():
        u = cut = n_iter = 0
        ok = True
        for n, it in enumerate(items):
            if not (yield qfree, (n_iter & 1) ^ 1, True):
                break
            qfull.arrive(2)
            for _ in range(2):
                c.copy(qfull, lambda n=n: q_item.__setitem__(0, n))
            n_iter += 1        # (the kernel's loop counts on whether or not the tiles' loop was left)
            for t in range(it.T):
                ks, vs, left = u % NS, (u + 1) % NS, it.left(t)
                ok = (yield empty[ks], ((u // NS) & 1) ^ 1, True) and (yield empty[vs], (((u + 1) // NS) & 1) ^ 1, True)
                if not ok:
                    break
                here = cut_bar if left < BN else full[ks]
                here.arrive(2)
                c.copy(here, put(ks, ("K", u // 2)))
                c.copy(here, put(vs, ("V", u // 2, "clear" if left >= BN else "as copied")))
                if left < BN:
                    ok = yield cut_bar, cut & 1, True
                    if not ok:
                        yield cut_bar, cut & 1, False
                        break
                    cut += 1
                    c.expect(slot[vs], ("V", u // 2, "as copied"))
                    slot[vs] = ("V", u // 2, "clear")
                    full[ks].arrive()
                u += 2
            if not ok:
                break
        if drain == "always" or c.aborted:
            for v in range(max(u - 2 * NS, 0), u, 2):
                yield full[v % NS], (v // (2 * NS)) & 1, False
            if n_iter > 0:
                yield qfull, (n_iter - 1) & 1, False

    def issuer():
        ubase, pend, pf, nh = 0, [0] * NS, [0, 0], [0, 0]

        def issue_s(n, it, h, t, s_left):
            uk = ubase + 2 * t
            s = uk % NS
            if pend[s] == 0:
                if not (yield full[s], (uk // (2 * NS)) & 1, True):
                    return False
                pend[s] = int(it.uses(0, t)) + int(it.uses(1, t))

            def product():
                c.expect((slot[s], q_item[0]), (("K", uk // 2), n))
                s_tile[h] = (n, t)
            c.issue(product)
            c.commit(sfull[h])
            pend[s] -= 1
            if pend[s] == 0:
                c.commit(empty[s])
            s_left[0] -= 1
            if s_left[0] == 0:
                c.commit(qfree)
            return True

        def work():
            nonlocal ubase
            for n, it in enumerate(items):
                if not (yield qfull, n & 1, True):
                    return
                s_left = [sum(it.uses(h, t) for h in range(2) for t in range(it.T))]
                order = (1, 0) if it.valid[1] and it.first(1) < it.first(0) else (0, 1)
                for h in order:
                    if it.valid[h] and not (yield from issue_s(n, it, h, it.first(h), s_left)):
                        return
                first_pv, defer = [True, True], [-1, -1]
                for t in range(it.T):
                    vs = (ubase + 2 * t + 1) % NS
                    for h in range(2):
                        if 0 <= defer[h] <= t + 2:
                            if not (yield from issue_s(n, it, h, defer[h], s_left)):
                                return
                            defer[h] = -1
                    for h in range(2):
                        if not it.uses(h, t):
                            continue
                        if not (yield pfull[h], pf[h] & 1, True):
                            return
                        pf[h] += 1
                        if first_pv[h] and not (yield ofree[h], (nh[h] & 1) ^ 1, True):
                            return
                        first_pv[h] = False
                        c.issue(lambda vs=vs, u=ubase // 2 + t: c.expect(slot[vs], ("V", u, "clear")))
                        tn = it.next(h, t)
                        if tn > t + 2:
                            defer[h] = tn
                        elif tn >= 0:
                            if not (yield from issue_s(n, it, h, tn, s_left)):
                                return
                        else:
                            c.commit(pvdone[h])
                    c.commit(empty[vs])
                ubase += 2 * it.T
                for h in range(2):
                    nh[h] += int(it.valid[h])
        yield from work()
        c.commit(drained)
        yield drained, 0, False

    def softmax(h):
        seen = done = 0
        for n, it in enumerate(items):
            if not it.valid[h]:
                continue
            t = it.first(h)
            while t >= 0:
                if not (yield sfull[h], seen & 1, True):
                    return
                c.expect(s_tile[h], (n, t))
                seen += 1
                pfull[h].arrive()
                t = it.next(h, t)
            if not (yield pvdone[h], done & 1, True):
                return
            ofree[h].arrive()
            done += 1

    return c.run({"producer": producer(), "issuer": issuer(), "softmaxA": softmax(0), "softmaxB": softmax(1)})


BATCHES = [([300], 16, 64, 0, 0), ([1, 2, 128, 129, 500], 16, 48, 0, 0), ([31, 33, 64, 65, 127, 5], 4, 24, 1, 2), ([1500, 700, 2], 4, 200, 0, 0),
           ([2500, 90], 512, 4, 1, 0), ([900, 257], 1, 1, 0, 0), ([40] * 6, 16, 10 ** 6, 0, 3)]


@pytest.mark.parametrize("batch", BATCHES, ids=lambda b: "-".join(map(str, b[0])))
def test_attention(batch):
    items = items_of(*batch[:4], share=batch[4])
    assert any(it.left(t) < BN for it in items for t in range(it.T))
    for seed in range(25):
        assert run_attention(items, seed) is None


@pytest.mark.parametrize("batch", BATCHES[:4], ids=lambda b: "-".join(map(str, b[0])))
def test_attention_that_is_given_up(batch):
    items = items_of(*batch[:4], share=batch[4])
    for seed in range(120):
        assert run_attention(items, seed, abort_at=1 + 3 * seed) is None


def test_the_model_sees_copies_that_nobody_waits_for():
    # a producer that waits for its copies only if the flag is set when it looks: an abort right behind that
    items = items_of([128], 16, 64, 0, heads=1)

    def ends(seed, at):
        try:
            return run_attention(items, seed, at, drain="if aborted") is None
        except AssertionError:
            return False
    assert not all(ends(seed, at) for seed in range(40) for at in range(2, 14))
    assert all(run_attention(items, seed, at) is None for seed in range(40) for at in range(2, 14))


# ---------------------------------------------------------------- gradients

def run_rings(items, seed, kind, abort_at=None):
    """items[i]: keys or rows that are left of each tile of item i.  dq: only the long ring's tiles are cut (keys), the
    queries have a barrier of their own; dkv: both rings' are (rows)."""
    c = Cta(seed, abort_at)
    lfull, lempty = [Bar(f"lfull{s}") for s in range(LONG)], [Bar(f"lempty{s}") for s in range(LONG)]
    sfull, sempty = [Bar(f"sfull{s}") for s in range(SHORT)], [Bar(f"sempty{s}") for s in range(SHORT)]
    res, resfree, qbar, qt, cut_bar, drained = (Bar(n) for n in ("res", "resfree", "q", "qt", "cut", "drain"))
    held = {"l": [None] * LONG, "s": [None] * SHORT, "res": None, "q": None}

    def producer():
        g = nl = ns = nq = nr = 0
        cut = [0]

        def load(full, ring, at, tile, left):
            if left >= BN:
                full.arrive(1)
                c.copy(full, lambda: held[ring].__setitem__(at, (tile, "clear")))
                return True
            cut_bar.arrive(1)
            c.copy(cut_bar, lambda: held[ring].__setitem__(at, (tile, "as copied")))
            if not (yield cut_bar, cut[0] & 1, True):
                yield cut_bar, cut[0] & 1, False
                return False
            cut[0] += 1
            c.expect(held[ring][at], (tile, "as copied"))
            held[ring][at] = (tile, "clear")
            full.arrive()
            return True

        def work():
            nonlocal g, nl, ns, nq, nr
            for it, tiles in enumerate(items):
                if kind == "dq":
                    if not (yield qt, (it & 1) ^ 1, True):
                        return
                    qbar.arrive(1)
                    c.copy(qbar, lambda it=it: held.__setitem__("q", it))
                    nq = it + 1
                if not (yield resfree, (it & 1) ^ 1, True):
                    return
                res.arrive(1)
                c.copy(res, lambda it=it: held.__setitem__("res", it))
                nr = it + 1
                for left in tiles:
                    if not (yield lempty[g % LONG], ((g // LONG) & 1) ^ 1, True):
                        return
                    if not (yield from load(lfull[g % LONG], "l", g % LONG, g, left)):
                        return
                    nl = g + 1
                    if not (yield sempty[g % SHORT], ((g // SHORT) & 1) ^ 1, True):
                        return
                    if not (yield from load(sfull[g % SHORT], "s", g % SHORT, g, left if kind == "dkv" else BN)):
                        return
                    ns = g + 1
                    g += 1
        yield from work()
        if nr > 0:
            yield res, (nr - 1) & 1, False
        for x in range(max(nl - LONG, 0), nl):
            yield lfull[x % LONG], (x // LONG) & 1, False
        for x in range(max(ns - SHORT, 0), ns):
            yield sfull[x % SHORT], (x // SHORT) & 1, False
        if nq > 0:
            yield qbar, (nq - 1) & 1, False

    def issuer():
        def work():
            g = 0
            for it, tiles in enumerate(items):
                if kind == "dq":
                    if not (yield qbar, it & 1, True):
                        return
                    c.expect(held["q"], it)
                    qt.arrive()
                if not (yield res, it & 1, True):
                    return
                for x in range(len(tiles)):
                    if not (yield lfull[g % LONG], (g // LONG) & 1, True) or not (yield sfull[g % SHORT], (g // SHORT) & 1, True):
                        return

                    def product(g=g, it=it):
                        c.expect((held["l"][g % LONG], held["s"][g % SHORT], held["res"]), ((g, "clear"), (g, "clear"), it))
                    c.issue(product)
                    c.commit(sempty[g % SHORT])
                    c.commit(lempty[g % LONG])
                    g += 1
                c.commit(resfree)
        yield from work()
        c.commit(drained)
        yield drained, 0, False

    return c.run({"producer": producer(), "issuer": issuer()})


TILES = [[[5]], [[128, 128, 40]] * 3, [[300, 172, 44], [44], [128], [7, 135, 7, 1]], [[500, 372, 244, 116]] * 2]


@pytest.mark.parametrize("kind", ["dq", "dkv"])
@pytest.mark.parametrize("items", TILES, ids=str)
def test_gradients(items, kind):
    for seed in range(60):
        assert run_rings(items, seed, kind) is None
        assert run_rings(items, seed, kind, abort_at=1 + seed) is None
