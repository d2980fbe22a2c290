"""A run of the paged operators as a serving loop uses them: a prompt goes into pages, then steps of
drafted trees are appended, attended, verified, compacted, pooled, and pages are reserved, shared,
copied and freed, all from device data.  Every step's attention equals the 64-bit oracle's rows of
the whole sequence so far."""
import numpy as np
import pytest
import torch

import oracle
from paged_ref import chain, rotate, t64
from sparse_long_context_cca_gb300 import api

pytestmark = pytest.mark.gpu

CASES = [  # dtype, Hq, Hkv, d, g, w, rows, core rows, T
    (torch.bfloat16, 8, 2, 128, 8, 48, 16, 8, 7),
    (torch.bfloat16, 2, 2, 64, 4, 40, 8, 16, 5),
    (torch.float32, 4, 2, 128, 8, 32, 24, 4, 6),
    (torch.bfloat16, 16, 1, 128, 16, 64, 32, 32, 20),   # 320 rows per KV head
]


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


class Cache:
    """One layer's pages and their two books (raw tokens, core tokens)."""

    def __init__(self, B, Hkv, d, g, w, rows, crows, cap, dtype):
        self.B, self.g, self.w, self.rows, self.crows = B, g, w, rows, crows
        cols, ccols = cap // rows + 2, cap // g // crows + 2
        mk = lambda n, r: torch.full((n, Hkv, r, d), float("nan"), dtype=dtype, device="cuda")  # noqa: E731
        n, nc = B * (w // rows + 6) + B * (cap // rows + 2), B * ccols + 2
        self.K, self.V, self.Kc, self.Vc = mk(n, rows), mk(n, rows), mk(nc, crows), mk(nc, crows)
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.refs, self.crefs, self.table, self.ctable = z(n), z(nc), z(B, cols) - 1, z(B, ccols) - 1
        self.status = z(1)

    def room(self, lens, extra):
        kw = dict(dev_status=self.status)
        pairs = api.cca_pages_reserve(self.refs, self.table, lens, extra, self.rows, **kw)
        api.cca_pages_copy(self.K, self.V, pairs, **kw)
        cores = lens // self.g
        more = (lens + extra) // self.g - cores
        pairs = api.cca_pages_reserve(self.crefs, self.ctable, cores, more.to(torch.int32), self.crows, **kw)
        api.cca_pages_copy(self.Kc, self.Vc, pairs, **kw)

    def drop_behind(self, lens):
        """Raw pages that no later window reaches, and those past the last token."""
        cols = torch.full_like(lens, self.table.shape[1])
        behind = (lens - self.w + 1).clamp(min=0) // self.g * self.g // self.rows
        api.cca_pages_free(self.refs, self.table, torch.zeros_like(lens), behind.to(torch.int32), dev_status=self.status)
        api.cca_pages_free(self.refs, self.table, (-(-lens // self.rows)).to(torch.int32), cols, dev_status=self.status)

    def fork(self, src, dst, lens):
        api.cca_pages_fork(self.refs, self.table, src, dst, lens, self.rows, dev_status=self.status)
        api.cca_pages_fork(self.crefs, self.ctable, src, dst, (lens // self.g).to(torch.int32), self.crows, dev_status=self.status)

    def drop(self, rows):
        for refs, table in ((self.refs, self.table), (self.crefs, self.ctable)):
            last = torch.zeros(self.B, dtype=torch.int32, device="cuda")
            last[rows] = table.shape[1]
            api.cca_pages_free(refs, table, torch.zeros_like(last), last, dev_status=self.status)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_serving_loop(case):
    dtype, Hq, Hkv, d, g, w, rows, crows, T = CASES[case]
    rng, gen = np.random.default_rng(case), torch.Generator().manual_seed(case)
    B, cap, prompt = 3, 400, [61, 17, 130]
    scale = 1.0 if dtype == torch.float32 else d ** -0.25
    mk = lambda *s: (torch.randn(s, generator=gen) * scale).to(dtype)  # noqa: E731
    f, _ = api.rope_frequencies(d, 10000.0)
    cache = Cache(B, Hkv, d, g, w, rows, crows, cap, dtype)
    # the sequences in 64 bits: rotated queries and keys as the device holds them, values
    seq = [dict(Q=np.zeros((Hq, 0, d)), K=np.zeros((Hkv, 0, d)), V=np.zeros((Hkv, 0, d))) for _ in range(B)]

    def commit(b, q, k, v):
        for n, x in (("Q", q), ("K", k), ("V", v)):
            seq[b][n] = np.concatenate([seq[b][n], x], 1)

    # prompts of different lengths, right-padded to one batch
    N = max(prompt)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    Q, K, V = (mk(B, N, h, d).cuda().transpose(1, 2) for h in (Hq, Hkv, Hkv))
    cache.room(lens, i32(prompt))
    q = api.cca_rope_append(Q, K, V, cache.K, cache.V, cache.table, lens, f, counts=i32(prompt), dev_status=cache.status)
    api.cca_pool_pages(q, cache.K, cache.V, cache.table, cache.Kc, cache.Vc, cache.ctable, lens, i32(prompt), g,
                       dev_status=cache.status)
    k, _ = api.cca_rope(K, None, f)
    want, bound = rotate(K, np.broadcast_to(np.arange(N), (B, N)), f.cpu(), "half")
    assert (np.abs(t64(k) - want) <= bound).all()
    for b in range(B):
        commit(b, t64(q)[b, :, :prompt[b]], t64(k)[b, :, :prompt[b]], t64(V)[b, :, :prompt[b]])
    lens = i32(prompt)
    cache.drop_behind(lens)
    assert cache.status.item() == 0

    for step in range(6):
        if step == 3:   # sequence 2 ends, and branches off sequence 0
            cache.drop([2])
            cache.fork(i32([0]), i32([2]), lens)
            lens[2] = lens[0]
            seq[2] = {n: x.copy() for n, x in seq[0].items()}
        extra = torch.full_like(lens, T)
        cache.room(lens, extra)
        parents = np.array([[int(rng.integers(max(-1, t - 3), t)) for t in range(T)] for _ in range(B)])
        if T > 5:
            parents[1, -2:] = -2
        if step == 4:
            parents = np.broadcast_to(np.arange(-1, T - 1), (B, T)).copy()
        par = None if step == 4 else i32(parents)
        Q, K, V = (mk(B, T, h, d).cuda().transpose(1, 2) for h in (Hq, Hkv, Hkv))
        q = api.cca_rope_append(Q, K, V, cache.K, cache.V, cache.table, lens, f, parents=par, dev_status=cache.status)
        O, LSE = api.cca_tree_fwd(q, cache.K, cache.V, cache.table, cache.Kc, cache.Vc, cache.ctable, lens, g, w, parents=par,
                                  dev_status=cache.status)
        depth = np.array([[len(chain(p, t) or [0]) - 1 for t in range(T)] for p in parents.tolist()])
        pos = lens.cpu().numpy()[:, None] + depth
        k = np.zeros((B, Hkv, T, d))
        for b in range(B):   # what the pages hold of the new tokens
            for t in range(T):
                if chain(parents[b].tolist(), t) is not None:
                    x = int(lens[b]) + t
                    k[b, :, t] = t64(cache.K[int(cache.table[b, x // rows]), :, x % rows])
        # each node's row against the oracle: the whole sequence, the node's chain at its end
        qn, vn = t64(q), t64(V)
        accepted, paths = [], np.zeros((B, T), int)
        for b in range(B):
            leaf = int(rng.integers(0, T - 2))
            for t in sorted({0, leaf, T - 1}):
                ch = chain(parents[b].tolist(), t)
                if ch is None:
                    assert not O[b, :, t].any()
                    continue
                ch = ch[::-1]
                n = seq[b]["Q"].shape[1] + len(ch)
                pad = -n % g
                grow = lambda x, y: np.concatenate([x, y, np.zeros((x.shape[0], pad, d))], 1)[None]  # noqa: E731,B023
                Qs, Ks, Vs = grow(seq[b]["Q"], qn[b][:, ch]), grow(seq[b]["K"], k[b][:, ch]), grow(seq[b]["V"], vn[b][:, ch])
                Kc, Vc = oracle.pool(Qs, Ks, Vs, g)
                Oe, Le = oracle.attn_rows(Qs, Ks, Vs, Kc, Vc, g, w, [(0, h, n - 1) for h in range(Hq)])
                # core rows are rounded to the cache's type before they are attended (half a step of their
                # size in K moves a score by at most that times sum |q k| tau), and so are weights and output
                tau = d ** -0.5
                eps = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
                move = 2 * eps * tau * np.abs(Qs[0, :, n - 1]).sum(-1).max() * np.abs(Ks).max() + 1e-5
                size = np.abs(Vs).max()
                assert np.abs(t64(O[b, :, t]) - Oe).max() <= (2 * move + 4 * eps + 1e-6) * size
                assert np.abs(t64(LSE[b, :, t]) - Le).max() <= move + 1e-5
            ch = chain(parents[b].tolist(), leaf)[::-1]
            accepted.append(len(ch) if step != 2 else 0)
            paths[b, :len(ch)] = ch
            if accepted[-1]:
                commit(b, qn[b][:, ch], k[b][:, ch], vn[b][:, ch])
        acc, path = i32(accepted), i32(paths)
        # padding past the accepted nodes is never looked at
        api.cca_pages_compact(cache.K, cache.V, cache.table, lens, path, acc, dev_status=cache.status)
        api.cca_pool_pages(q, cache.K, cache.V, cache.table, cache.Kc, cache.Vc, cache.ctable, lens, acc, g, path=path,
                           dev_status=cache.status)
        lens = lens + acc
        cache.drop_behind(lens)
        assert cache.status.item() == 0 and pos.shape == (B, T)
        # the books balance: every page is held as often as tables name it
        for refs, table in ((cache.refs, cache.table), (cache.crefs, cache.ctable)):
            held = torch.bincount(table[table >= 0].long(), minlength=refs.numel())
            assert torch.equal(held.int(), refs)
    # the raw pages held reach back one window and no further
    n = (cache.table >= 0).sum(1)
    assert int(n.max()) <= (w + g) // rows + 2


def test_step_in_one_graph():
    """A whole step captured once and replayed for later lengths, trees and tables."""
    dtype, Hq, Hkv, d, g, w, rows, crows, T = torch.bfloat16, 8, 2, 128, 8, 48, 16, 8, 6
    B, cap = 2, 300
    gen = torch.Generator(device="cuda").manual_seed(0)
    mk = lambda *s: (torch.randn(s, generator=gen, device="cuda") * 0.3).to(dtype)  # noqa: E731
    f, _ = api.rope_frequencies(d)
    parents, path, acc = i32([[-1, 0, 0, 1, 2, 3]] * B), i32([[0, 2, 4]] * B), i32([3, 2])
    steps = [(mk(B, Hq, T, d), mk(B, Hkv, T, d), mk(B, Hkv, T, d)) for _ in range(14)]

    def step(c, lens, Q, K, V, ws):
        c.room(lens, torch.full_like(lens, T))
        q = api.cca_rope_append(Q, K, V, c.K, c.V, c.table, lens, f, parents=parents, dev_status=c.status)
        out = api.cca_tree_fwd(q, c.K, c.V, c.table, c.Kc, c.Vc, c.ctable, lens, g, w, parents=parents, dev_status=c.status,
                               workspace=ws)
        api.cca_pages_compact(c.K, c.V, c.table, lens, path, acc, dev_status=c.status)
        api.cca_pool_pages(q, c.K, c.V, c.table, c.Kc, c.Vc, c.ctable, lens, acc, g, path=path, dev_status=c.status)
        lens += acc
        c.drop_behind(lens)
        return out

    ws = torch.empty(api.tree_workspace_size(B, Hq, Hkv, T, d, g, w, dtype), dtype=torch.uint8, device="cuda")
    results = []
    for captured in (False, True):
        c, lens = Cache(B, Hkv, d, g, w, rows, crows, cap, dtype), i32([0, 0])
        got = []
        if not captured:
            for x in steps:
                got.append([t.clone() for t in step(c, lens, *x, ws)])
        else:
            buf = [t.clone() for t in steps[0]]
            got.append([t.clone() for t in step(c, lens, *buf, ws)])     # warm-up: the first step
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = step(c, lens, *buf, ws)
            for x in steps[1:]:
                for t, s in zip(buf, x):
                    t.copy_(s)
                graph.replay()
                got.append([t.clone() for t in out])
        torch.cuda.synchronize()
        assert c.status.item() == 0 and lens.tolist() == [42, 28]
        results.append(got)
    for a, b in zip(*results):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def branch(refs, table, K, V, lens, extra, src, dst, last, gate):
    """Forked rows get room, their shared pages are copied, the old rows end; `gate` makes the lengths."""
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    side.wait_stream(here)
    with torch.cuda.stream(side):
        late = lens + gate.sum(dtype=torch.int32)      # a kernel on another stream, still running
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    here.wait_stream(side)
    api.cca_pages_fork(refs, table, src, dst, late, K.shape[-2], dev_status=status)
    pairs = api.cca_pages_reserve(refs, table, late, extra, K.shape[-2], dev_status=status)
    api.cca_pages_copy(K, V, pairs, dev_status=status)
    kept = pairs.clone()                               # a copy between two of the calls
    api.cca_pages_free(refs, table, torch.zeros_like(lens), last, dev_status=status)
    return kept, status


def test_calls_behind_copies_and_other_streams():
    """The page calls may be scheduled while the work before them drains; they wait for it, also
    where it is a copy or another stream's, eager and captured."""
    B, cols, rows, n = 6, 9, 16, 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    K0, V0 = (torch.randn(n, 2, rows, 64, generator=gen, device="cuda").bfloat16() for _ in range(2))
    lens, grown = i32([70, 33, 70, 33, 9, 0]), [75, 38]  # the forked rows are as long as their sources
    held, extra = i32([75, 38, 0, 0, 14, 0]), i32([0, 0, 20, 20, 0, 0])
    src, dst, last = i32([0, 1]), i32([2, 3]), i32([cols, cols, 0, 0, 0, 0])
    gate = torch.zeros(64 << 20, dtype=torch.int8, device="cuda")
    gate[:5] = 1                                       # lengths grow by 5
    results = []
    for captured in (False, True):
        refs, table = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
        api.cca_pages_reserve(refs, table, torch.zeros_like(lens), held, rows)
        K, V = K0.clone(), V0.clone()
        start = refs.clone(), table.clone()
        args = refs, table, K, V, lens, extra, src, dst, last, gate
        branch(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.graph(graph):
                kept, status = branch(*args)
        refs.copy_(start[0]), table.copy_(start[1]), K.copy_(K0), V.copy_(V0)
        if captured:
            graph.replay()
        else:
            kept, status = branch(*args)
        torch.cuda.synchronize()
        assert status.item() == 0
        results.append([t.clone() for t in (refs, table, K, V, kept)])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    refs, table, K, V, kept = results[0]
    for b, s in ((2, 0), (3, 1)):
        old, new = kept[b].tolist()
        assert old >= 0 and new == table[b][grown[s] // rows].item() and refs[new].item() == 1
        assert torch.equal(K[new], K0[old]) and torch.equal(V[new], V0[old])
    assert (table[:2] == -1).all() and kept[4].tolist() == [-1, -1]
