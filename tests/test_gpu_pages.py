"""Pages of a cache: reserving, forking, copying, compacting, freeing; storing new tokens and
pooling groups through pages.  Against plain sequential code on the CPU."""
import numpy as np
import pytest
import torch

from paged_ref import close, paged, pool_groups, rotate
from sparse_long_context_cca_gb300 import api

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Book:
    """The rules, one entry after the other."""

    def __init__(self, n, B, cols, rows):
        self.refs, self.table, self.rows = [0] * n, [[-1] * cols for _ in range(B)], rows

    def gpu(self):
        return i32(self.refs), i32(self.table)

    def same(self, refs, table):
        assert refs.tolist() == self.refs
        assert table.tolist() == self.table

    def reserve(self, lens, extra):
        cols, refs, wanted, pairs = len(self.table[0]), list(self.refs), [], [[-1, -1] for _ in lens]
        for b, (n, e) in enumerate(zip(lens, extra)):
            if e <= 0 or n < 0 or -(-(n + e) // self.rows) > cols:
                continue
            for c in range(n // self.rows, -(-(n + e) // self.rows)):
                p = self.table[b][c]
                if p < 0 or refs[p] > 1:
                    wanted.append((b, c, p))
                    if p >= 0:
                        refs[p] -= 1
        free = [p for p, r in enumerate(self.refs) if r == 0]
        if len(wanted) > len(free):
            return pairs
        for (b, c, p), new in zip(wanted, free):
            self.table[b][c] = new
            refs[new] = 1
            if p >= 0 and c == lens[b] // self.rows and lens[b] % self.rows:
                pairs[b] = [p, new]
        self.refs = refs
        return pairs

    def fork(self, src, dst, lens):
        for s, d in zip(src, dst):
            for c in range(min(-(-lens[s] // self.rows), len(self.table[0]))):
                p = self.table[s][c]
                self.table[d][c] = p
                if p >= 0:
                    self.refs[p] += 1

    def free(self, first, last):
        for b, (x, y) in enumerate(zip(first, last)):
            for c in range(max(x, 0), min(y, len(self.table[0]))):
                p = self.table[b][c]
                if p >= 0:
                    self.refs[p] -= 1
                    self.table[b][c] = -1


@pytest.mark.parametrize("n,B,cols,rows", [(64, 5, 9, 16), (9000, 70, 40, 7), (3, 1, 2, 1), (5000, 1100, 4, 64)])
def test_book_through_random_steps(n, B, cols, rows):
    rng = np.random.default_rng(n)
    book = Book(n, B, cols, rows)
    refs, table = book.gpu()
    lens = [0] * B
    for step in range(12):
        extra = rng.integers(-1, 2 * rows + 2, B).tolist()
        extra = [min(e, cols * rows - x) for e, x in zip(extra, lens)]
        st = status()
        pairs = api.cca_pages_reserve(refs, table, i32(lens), i32(extra), rows, dev_status=st)
        before = [r[:] for r in book.table]
        want = book.reserve(lens, extra)
        book.same(refs, table)
        assert pairs.tolist() == want
        full = book.table == before and any(e > 0 and before[b][x // rows:-(-(x + e) // rows)].count(-1) for b, (x, e) in enumerate(zip(lens, extra)))
        assert st.item() == (api.CCA_ERR_NO_PAGES if full else 0)
        if not full:
            lens = [x + max(int(rng.integers(0, e + 1)) if e > 0 else 0, 0) for x, e in zip(lens, extra)]
        if B > 1:
            order = rng.permutation(B)
            dst, src = order[:B // 3], order[B // 3:]
            src = rng.choice(src, len(dst))
            last = [cols if b in dst else 0 for b in range(B)]
            first = [0] * B
            api.cca_pages_free(refs, table, i32(first), i32(last))
            book.free(first, last)
            st = status()
            api.cca_pages_fork(refs, table, i32(src), i32(dst), i32(lens), rows, dev_status=st)
            book.fork(src, dst, lens)
            for s, d in zip(src, dst):
                lens[d] = lens[s]
            book.same(refs, table)
            assert st.item() == 0
        behind = [int(rng.integers(0, x // rows + 1)) for x in lens]
        api.cca_pages_free(refs, table, i32([-3] * B), i32([b // 2 for b in behind]))
        book.free([-3] * B, [b // 2 for b in behind])
        book.same(refs, table)


def test_reserve_last_holder_keeps_the_page():
    book = Book(10, 4, 3, 16)
    book.table = [[2, -1, -1], [2, -1, -1], [2, -1, -1], [-1, -1, -1]]
    book.refs[2] = 3
    refs, table = book.gpu()
    pairs = api.cca_pages_reserve(refs, table, i32([5, 5, 5, 0]), i32([1, 20, 1, 0]), 16)
    assert pairs.tolist() == [[2, 0], [2, 1], [-1, -1], [-1, -1]]
    assert table.tolist() == [[0, -1, -1], [1, 3, -1], [2, -1, -1], [-1, -1, -1]]
    assert refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0, 0, 0]


def test_reserve_too_few_pages_changes_nothing():
    refs, table = i32([1, 0, 1]), i32([[0, -1, -1], [2, -1, -1]])
    st = status()
    pairs = api.cca_pages_reserve(refs, table, i32([4, 4]), i32([4, 4]), 4, dev_status=st)
    assert st.item() == api.CCA_ERR_NO_PAGES and (pairs == -1).all()
    assert refs.tolist() == [1, 0, 1] and table.tolist() == [[0, -1, -1], [2, -1, -1]]
    # a row outside the table is reported and the others are served
    st = status()
    api.cca_pages_reserve(refs, table, i32([4, 4]), i32([4, 100]), 4, dev_status=st)
    assert st.item() == api.CCA_ERR_INVALID_ARG and table.tolist() == [[0, 1, -1], [2, -1, -1]]
    st = status()
    api.cca_pages_reserve(refs, table, i32([2 ** 31 - 1, -5]), i32([2 ** 31 - 1, 3]), 4, dev_status=st)
    assert st.item() == api.CCA_ERR_INVALID_ARG and refs.tolist() == [1, 1, 1]


def test_fork_refuses_clashes():
    table0 = [[0, 1], [-1, -1], [-1, -1], [2, -1]]
    for src, dst, done in (([0, 0], [1, 1], [1]), ([0, 1], [1, 2], [2]), ([0], [0], []), ([0], [3], []), ([0], [9], []),
                           ([-1], [1], []), ([0, 0], [1, 2], [1, 2])):
        refs, table, st = i32([1, 1, 1, 0]), i32(table0), status()
        api.cca_pages_fork(refs, table, i32(src), i32(dst), i32([3, 0, 0, 1]), 2, dev_status=st)
        want = [list(r) for r in table0]
        for d in done:
            want[d] = [0, 1] if src[dst.index(d)] == 0 else [-1, -1]
        held = sum(want[d][0] == 0 for d in done)
        assert table.tolist() == want and refs.tolist() == [1 + held, 1 + held, 1, 0]
        assert st.item() == (0 if len(done) == len(dst) else api.CCA_ERR_INVALID_ARG)
    api.cca_pages_fork(refs, table, i32([]), i32([]), i32([3, 0, 0, 1]), 2)   # no pairs


def test_free_twice_is_reported():
    refs, table, st = i32([1, 0]), i32([[0, 0, 1, 99]]), status()
    api.cca_pages_free(refs, table, i32([0]), i32([2 ** 31 - 1]), dev_status=st)
    assert refs.tolist() == [0, 0] and table.tolist() == [[-1, -1, -1, 99]] and st.item() == api.CCA_ERR_INVALID_ARG


@DTYPES
@pytest.mark.parametrize("shape", [(7, 2, 3, 64), (3, 9, 4, 24, 128), (40, 1, 1, 64), (2, 300, 1, 16, 64)])
def test_copy(shape, dtype):
    gen = torch.Generator(device="cuda").manual_seed(0)
    Kp = torch.randn(shape, generator=gen, device="cuda").to(dtype)
    Vp = torch.randn(shape, generator=gen, device="cuda").to(dtype)
    n = shape[-4]
    rng = np.random.default_rng(n)
    order = rng.permutation(n)
    k = n // 3
    pairs = np.stack([rng.choice(order[k:], k), order[:k]], 1)
    pairs = np.concatenate([pairs, [[-1, -1], [0, -1]]])
    wk, wv = Kp.clone(), Vp.clone()
    for a, z in pairs[:k]:
        wk[..., z, :, :, :], wv[..., z, :, :, :] = Kp[..., a, :, :, :], Vp[..., a, :, :, :]
    st = status()
    api.cca_pages_copy(Kp, Vp, i32(pairs), dev_status=st)
    assert torch.equal(Kp, wk) and torch.equal(Vp, wv) and st.item() == 0
    # clashes: a destination that is a source, the same destination twice, a page out of range
    api.cca_pages_copy(Kp, Vp, i32([[0, 1], [1, 2], [0, n], [n + 5, 0]]), dev_status=st)
    wk[..., 2, :, :, :], wv[..., 2, :, :, :] = wk[..., 1, :, :, :].clone(), wv[..., 1, :, :, :].clone()
    assert torch.equal(Kp, wk) and torch.equal(Vp, wv) and st.item() == api.CCA_ERR_INVALID_ARG
    if n > 4:
        api.cca_pages_copy(Kp, Vp, i32([[0, 4], [1, 4]]))
        wk[..., 4, :, :, :], wv[..., 4, :, :, :] = wk[..., 0, :, :, :].clone(), wv[..., 0, :, :, :].clone()
        assert torch.equal(Kp, wk) and torch.equal(Vp, wv)
    api.cca_pages_copy(Kp, Vp, torch.empty(0, 2, dtype=torch.int32, device="cuda"))


def test_copy_many_pairs():
    n = 6000
    Kp = torch.arange(n * 16 * 64, device="cuda").reshape(n, 1, 16, 64).float()
    Vp = -Kp
    wk = Kp.clone()
    wk[n // 2:] = wk[:n // 2].flip(0)
    pairs = torch.stack([torch.arange(n // 2 - 1, -1, -1), torch.arange(n // 2, n)], 1).int().cuda()
    api.cca_pages_copy(Kp, Vp, pairs)
    assert torch.equal(Kp, wk) and torch.equal(Vp, -wk)


@DTYPES
@pytest.mark.parametrize("layers,H,d,rows,T", [(1, 2, 64, 7, 9), (3, 3, 128, 16, 40), (2, 8, 128, 64, 256)])
def test_compact(layers, H, d, rows, T, dtype):
    B, rng = 5, np.random.default_rng(T)
    lens = rng.integers(0, 3 * rows, B)
    cols = int(max(lens) + T) // rows + 1
    n = B * cols
    table = rng.permutation(n).reshape(B, cols)
    gen = torch.Generator(device="cuda").manual_seed(0)
    Kp = torch.randn(layers, n, H, rows, d, generator=gen, device="cuda").to(dtype)
    Vp = torch.randn(layers, n, H, rows, d, generator=gen, device="cuda").to(dtype)
    A = max(1, T - 3)
    path = np.stack([np.sort(rng.permutation(T)[:A]) for _ in range(B)])
    path[1] = np.arange(A)                      # nothing to move
    accepted = [A, A, 0, 1, A // 2]
    if layers == 1:
        Kp, Vp = Kp[0], Vp[0]

    def moved(pool, rows_ok):
        out = pool.clone()
        for b in range(B):
            if not rows_ok[b]:
                continue
            for i in range(accepted[b]):
                a, z = lens[b] + path[b, i], lens[b] + i
                out[..., int(table[b, z // rows]), :, z % rows, :] = out[..., int(table[b, a // rows]), :, a % rows, :].clone()
        return out

    wk, wv, st = moved(Kp, [1] * B), moved(Vp, [1] * B), status()
    api.cca_pages_compact(Kp, Vp, i32(table), i32(lens), i32(path), i32(accepted), dev_status=st)
    assert torch.equal(Kp, wk) and torch.equal(Vp, wv) and st.item() == 0
    # bad paths, counts, pages: reported, their sequences left as they are
    bad, tab = path.copy(), table.copy()
    bad[0, -1] = bad[0, -2] if A > 1 else -1
    accepted = [A, A + 1, 0, 1, max(1, A // 2)]
    tab[4, lens[4] // rows] = -1
    wk, wv = moved(Kp, [0, 0, 1, 1, 0]), moved(Vp, [0, 0, 1, 1, 0])
    api.cca_pages_compact(Kp, Vp, i32(tab), i32(lens), i32(bad), i32(accepted), dev_status=st)
    assert torch.equal(Kp, wk) and torch.equal(Vp, wv) and st.item() == api.CCA_ERR_INVALID_ARG


@DTYPES
@pytest.mark.parametrize("parents", [True, False])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,rows,rot,layout", [(3, 9, 4, 2, 128, 16, 128, "half"), (2, 1, 1, 1, 64, 5, 24, "interleaved"),
                                                          (2, 70, 6, 3, 64, 64, 0, "half"), (1, 256, 2, 1, 128, 7, 64, "half")])
def test_append(B, T, Hq, Hkv, d, rows, rot, layout, parents, dtype):
    rng = np.random.default_rng(T)
    gen = torch.Generator(device="cuda").manual_seed(0)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    lens = rng.integers(0, 200, B)
    cols = int(max(lens) + T) // rows + 1
    table = rng.permutation(B * cols).reshape(B, cols)
    Kp, Vp = mk(B * cols, Hkv, rows, d), mk(B * cols, Hkv, rows, d)
    Q, K, V = (mk(B, T, h, d).transpose(1, 2) for h in (Hq, Hkv, Hkv))     # as projections leave them
    par = np.array([[int(rng.integers(max(-1, t - 3), t)) for t in range(T)] for _ in range(B)])
    real = np.ones((B, T), bool)
    depth = np.broadcast_to(np.arange(T), (B, T)).copy()
    counts = None
    if parents:
        if T > 3:
            par[0, T // 2:] = -2
        for b in range(B):
            for t in range(T):
                p = par[b, t]
                depth[b, t] = 0 if p < 0 else depth[b, p] + 1
                real[b, t] = p == -1 or (p >= 0 and real[b, p])
    else:
        counts = rng.integers(0, T + 1, B)
        real = np.arange(T)[None] < counts[:, None]
    f = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))
    pos = lens[:, None] + depth
    wq, wk = rotate(Q, pos, f, layout, 1.2), rotate(K, pos, f, layout, 1.2)
    before = Kp.clone(), Vp.clone()
    st = status()
    q = api.cca_rope_append(Q, K, V, Kp, Vp, i32(table), i32(lens), f.cuda() if rot else None, parents=i32(par) if parents else None,
                            counts=None if counts is None else i32(counts), layout=layout, factor=1.2, dev_status=st)
    assert st.item() == 0
    keep = real[:, None, :, None]
    close(q, wq[0] * keep, wq[1] * keep, "Q")
    for b in range(B):
        for t in range(T):
            x = lens[b] + t
            p, r = int(table[b, x // rows]), x % rows
            if real[b, t]:
                close(Kp[p, :, r], wk[0][b, :, t], wk[1][b, :, t], "K")
                assert torch.equal(Vp[p, :, r], V[b, :, t])
                before[0][p, :, r], before[1][p, :, r] = Kp[p, :, r], Vp[p, :, r]
    assert torch.equal(Kp, before[0]) and torch.equal(Vp, before[1])      # nothing else was written


def test_append_out_of_the_table_is_reported():
    gen = torch.Generator(device="cuda").manual_seed(0)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    Kp, Vp, K = mk(4, 1, 4, 64), mk(4, 1, 4, 64), mk(3, 1, 2, 64)
    want = Kp.clone(), Vp.clone()
    want[0][1, :, 3], want[1][1, :, 3] = K[0, :, 0], K[0, :, 0]
    st = status()
    api.cca_rope_append(None, K, K, Kp, Vp, i32([[1], [7], [2]]), i32([3, 0, -1]), dev_status=st)
    assert st.item() == api.CCA_ERR_INVALID_ARG and torch.equal(Kp, want[0]) and torch.equal(Vp, want[1])


@DTYPES
@pytest.mark.parametrize("mode", [0, 1, 2, 3])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,g,rows,crows,lens", [
    (3, 20, 4, 2, 128, 8, 16, 5, [0, 37, 100]), (2, 33, 3, 1, 64, 3, 7, 64, [5, 64]), (1, 1, 2, 2, 128, 1, 16, 16, [9]),
    (2, 64, 8, 1, 128, 64, 24, 4, [63, 200]), (1, 40, 2, 2, 64, 16, 40, 8, [0]),
    (1, 1100, 8, 8, 64, 2, 48, 33, [5])])   # several groups per warp
def test_pool_pages(B, T, Hq, Hkv, d, g, rows, crows, lens, mode, dtype):
    rng = np.random.default_rng(T + mode)
    gen = torch.Generator().manual_seed(T)
    scale = 1.0 if dtype == torch.float32 else d ** -0.25
    mk = lambda *s: (torch.randn(s, generator=gen) * scale).to(dtype)  # noqa: E731
    A = max(1, T - 4)
    first = [n // g * g for n in lens]
    raws = [(mk(Hkv, n + T - f, d), mk(Hkv, n + T - f, d)) for n, f in zip(lens, first)]
    Kp, Vp, table = paged(raws, first, lens, Hkv, d, rows, (max(lens) + T) // rows + 1, dtype, 1)
    ccols = (max(lens) + T) // g // crows + 1
    ctable = rng.permutation(B * ccols).reshape(B, ccols)
    Kc, Vc = mk(B * ccols, Hkv, crows, d).cuda(), mk(B * ccols, Hkv, crows, d).cuda()
    Q = mk(B, Hq, T, d)
    for path in (np.stack([np.sort(rng.permutation(T)[:A]) for _ in range(B)]), None):
        accepted = [A if path is not None else T] + rng.integers(0, A + 1, B - 1).tolist()
        wk, wv = Kc.clone(), Vc.clone()
        st = status()
        api.cca_pool_pages(Q.cuda(), Kp.cuda(), Vp.cuda(), table.cuda(), Kc, Vc, i32(ctable), i32(lens), i32(accepted), g,
                           path=None if path is None else i32(path), pool_mode=mode, dev_status=st)
        assert st.item() == 0
        for b, j, k, v, dk, dv in pool_groups(Q, Kp, Vp, table, lens, accepted, path, g, rows, mode):
            p, r = int(ctable[b, j // crows]), j % crows
            close(Kc[p, :, r], k, dk, f"K group {j}")
            close(Vc[p, :, r], v, dv, f"V group {j}")
            wk[p, :, r], wv[p, :, r] = Kc[p, :, r], Vc[p, :, r]
        assert torch.equal(Kc, wk) and torch.equal(Vc, wv)               # no other row was written


def test_pool_pages_reports_what_is_missing():
    gen = torch.Generator(device="cuda").manual_seed(0)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    Q, Kp, Vp, Kc, Vc = mk(4, 2, 8, 64), mk(8, 1, 8, 64), mk(8, 1, 8, 64), mk(4, 1, 4, 64), mk(4, 1, 4, 64)
    want = Kc.clone()
    st = status()
    table, ctable = [[0, 1], [2, -1], [4, 5], [6, 7]], [[0], [1], [99], [3]]
    api.cca_pool_pages(Q, Kp, Vp, i32(table), Kc, Vc, i32(ctable), i32([4, 4, 4, 4]), i32([8, 8, 8, 9]), 4, dev_status=st)
    # sequence 0 pools groups 1 and 2; 1 only group 1 (its second page is missing); 2 and 3 none
    changed = [(p, r) for p in range(4) for r in range(4) if not torch.equal(Kc[p, :, r], want[p, :, r])]
    assert changed == [(0, 1), (0, 2), (1, 1)] and st.item() == api.CCA_ERR_INVALID_ARG


def test_raw_and_core_pages_in_one_pool():
    gen = torch.Generator(device="cuda").manual_seed(0)
    Kp, Vp = (torch.randn(6, 2, 8, 64, generator=gen, device="cuda") for _ in range(2))
    Q = torch.randn(1, 2, 16, 64, generator=gen, device="cuda")
    apart = Kp.clone(), Vp.clone()
    args = (i32([[3, 1]]),), (i32([[5]]), i32([0]), i32([16]), 4)
    api.cca_pool_pages(Q, *apart, *args[0], Kc := Kp.clone(), Vc := Vp.clone(), *args[1])
    api.cca_pool_pages(Q, Kp, Vp, *args[0], Kp, Vp, *args[1])
    assert torch.equal(Kp, Kc) and torch.equal(Vp, Vc)
    with pytest.raises(api.CcaError):     # a core pool inside the raw pool, with other pages
        api.cca_pool_pages(Q, Kp, Vp, *args[0], Kp[1:].view(-1, 2, 8, 64), Vp[1:], *args[1])


@DTYPES
def test_offsets_pass_32_bits(dtype):
    rows, H, d = 1024, 8, 128
    n = 2 ** 31 // (rows * H * d) + 2
    Kp = torch.zeros(n, H, rows, d, dtype=dtype, device="cuda")
    Vp = torch.zeros(n, H, rows, d, dtype=dtype, device="cuda")
    x = torch.randn(1, H, 3, d, device="cuda").to(dtype)
    last = n - 1
    api.cca_rope_append(None, x, x, Kp, Vp, i32([[last]]), i32([1000]))
    assert torch.equal(Kp[last, :, 1000:1003], x[0]) and torch.equal(Vp[last, :, 1000:1003], x[0])
    api.cca_pages_compact(Kp, Vp, i32([[last]]), i32([1000]), i32([[1, 2]]), i32([2]))
    assert torch.equal(Kp[last, :, 1000:1002], x[0, :, 1:]) and torch.equal(Vp[last, :, 1002], x[0, :, 2])
    api.cca_pages_copy(Kp, Vp, i32([[last, last - 1]]))
    assert torch.equal(Kp[last - 1], Kp[last]) and torch.equal(Vp[last - 1], Vp[last]) and not Kp[:last - 1].any()


def test_a_page_shared_across_columns_is_not_handed_out():
    """A page stands in the same column of every row that holds it.  In a table that breaks the rule a
    page may lose all its holders within one reserve; it is free after the call, and not given out by it:
    the copies behind it read it."""
    n = 12288
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    free = [7, 8, 9000]                          # the free pages lie in different steps of the scan
    refs[free] = 0
    shared = 4100
    refs[shared] = 2
    table = i32([[shared, -1], [-1, shared], [-1, -1]])
    status = i32([0])
    pairs = api.cca_pages_reserve(refs, table, i32([3, 19, 0]), i32([1, 1, 1]), 16, dev_status=status)
    t = table.cpu()
    held = [int(t[0, 0]), int(t[1, 1]), int(t[2, 0])]
    assert held == free
    assert pairs.cpu().tolist() == [[shared, 7], [shared, 8], [-1, -1]]
    assert refs[shared].item() == 0 and refs.sum().item() == n - 1 and status.item() == 0
    K, V = torch.zeros(n, 1, 16, 64, device="cuda"), torch.zeros(n, 1, 16, 64, device="cuda")
    K[shared] = 3.0
    api.cca_pages_copy(K, V, pairs, dev_status=status)
    assert status.item() == 0 and (K[7] == 3.0).all() and (K[8] == 3.0).all()


def test_the_book_keeps_shared_pages_in_their_column():
    """Forks and copies on write leave every page in one column, whatever is dropped between them."""
    rng = np.random.default_rng(5)
    refs, table = i32([0] * 64), i32(np.full((6, 5), -1))
    lens, status, rows = np.zeros(6, dtype=np.int64), i32([0]), 4
    for step in range(60):
        b, o = rng.permutation(6)[:2]
        if rng.random() < 0.4:
            first, last = np.zeros(6), np.zeros(6)
            last[o] = 5
            api.cca_pages_free(refs, table, i32(first), i32(last), dev_status=status)
            api.cca_pages_fork(refs, table, i32([b]), i32([o]), i32(lens), rows, dev_status=status)
            lens[o] = lens[b]
        extra = np.minimum(rng.integers(0, 4, 6), 5 * rows - lens)
        api.cca_pages_reserve(refs, table, i32(lens), i32(extra), rows, dev_status=status)
        lens = np.where(lens + extra >= 5 * rows, lens, lens + extra)
        t = table.cpu().numpy()
        where = {}
        for c in range(5):
            for page in t[:, c][t[:, c] >= 0]:
                assert where.setdefault(int(page), c) == c, step
        count = np.bincount(t[t >= 0], minlength=64)
        assert status.item() == 0 and (refs.cpu().numpy() == count).all(), step


def test_reserve_from_a_large_pool_mostly_held():
    """Free pages few and far apart: several steps of the scan, shared pages among those replaced."""
    n, B, cols, rows = 30000, 40, 6, 16
    rng = np.random.default_rng(8)
    free = np.sort(rng.choice(np.arange(100, n), 500, replace=False))
    book = Book(n, B, cols, rows)
    held = [p for p in range(n) if p not in set(free.tolist())]
    for p in held:
        book.refs[p] = 1                                     # by other tables
    lens = rng.integers(0, 60, B)
    for b in range(0, B, 2):                                 # rows in pairs share their pages
        for c in range(-(-int(max(lens[b], lens[b + 1])) // rows)):
            page = held.pop(int(rng.integers(len(held))))
            book.table[b][c] = book.table[b + 1][c] = page
            book.refs[page] = 2
    extra = rng.integers(0, 36, B)
    refs, table = book.gpu()
    s = status()
    pairs = api.cca_pages_reserve(refs, table, i32(lens), i32(extra), rows, dev_status=s)
    want = book.reserve(lens.tolist(), extra.tolist())
    book.same(refs, table)
    assert s.item() == 0 and pairs.tolist() == want
