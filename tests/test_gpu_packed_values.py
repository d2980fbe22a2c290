"""Packed sequences that hold infinities, NaN and the types' largest values: what each row shows of them, and
what they cost."""
import numpy as np
import pytest
import torch

import packed_ref as ref
from paged_ref import t64
from sparse_long_context_cca_gb300 import api
from test_gpu_packed import BF, F32, IDS, KINDS, Case, device, rand

pytestmark = pytest.mark.gpu


def agree(O, L, want, what):
    """The same infinities and NaN as the formulas, the other values within their bounds."""
    o, l, eo, el = want
    got, lse = t64(O), t64(L)
    for x, y, e in ((got, o, eo), (lse, l, el)):
        fine, signed = np.isfinite(y), np.isinf(y)
        assert np.array_equal(np.isnan(x), np.isnan(y)) and np.array_equal(x[signed], y[signed]), what
        off = np.abs(x[fine] - y[fine])
        assert (off <= e[fine]).all(), (what, (off / e[fine]).max())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64)], ids=["bf16-128", "bf16-64"])
def test_a_value_that_every_later_row_sees_costs_no_time_out(dtype, d):
    # a long document with an infinite value at its front: its rows are infinite there, and no wait runs out meanwhile
    N = 32768
    lib = api.load_library()
    cu = [0, N, N + 300]
    Q, K, V = (rand(h, N + 300, d, dtype=dtype, seed=i) for i, h in enumerate((2, 1, 1)))
    packed = api.cca_pack(device(cu), N + 300, 16)
    clean, _ = api.cca_attn_packed(Q, K, V, None, None, packed)
    for at in (0, N - 3):
        bad = V.clone()
        bad[:, at, 5], bad[:, at, d - 1] = float("inf"), float("nan")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        lib.cca_test_set_wait_limit_ns(20_000_000)
        try:
            O, L = api.cca_attn_packed(Q, K, bad, None, None, packed, dev_status=status)
            torch.cuda.synchronize()
        finally:
            lib.cca_test_set_wait_limit_ns(1_000_000_000)
        assert int(status) == 0
        assert (O[:, at:N, 5] == float("inf")).all() and torch.isnan(O[:, at:N, d - 1]).all()
        rest = [c for c in range(d) if c not in (5, d - 1)]
        assert torch.equal(O[:, :, rest], clean[:, :, rest])
        # rows that do not see it: as they were, up to the weights' rounding (those of its tile are formed again in fp32)
        rows = np.r_[0:at, N:N + 300]
        d_o = (O[:, rows].float() - clean[:, rows].float()).abs()
        assert (d_o <= 2.0 ** -7 * (1 + clean[:, rows].float().abs())).all()


def test_what_a_bad_value_costs():
    # whether one row shows it or all do, a call takes a few times as long at most (row by row it would be hundreds)
    N, d = 32768, 128
    Q, K, V = (rand(h, N, d, dtype=BF, seed=i) for i, h in enumerate((8, 1, 1)))
    packed = api.cca_pack(device([0, N]), N, 16)

    def seconds(v):
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            api.cca_attn_packed(Q, K, v, None, None, packed)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    plain = seconds(V)
    for what, rows in (("front", 0), ("column", slice(None)), ("sparse", slice(0, N, 4000)), ("end", N - 1)):
        for bad in (float("nan"), float("inf")):
            v = V.clone()
            v[:, rows, 7] = bad
            t = seconds(v)
            print(f"{what} {bad}: {t:.2f} ms, plain {plain:.2f}")
            assert t <= 20 * plain, (what, bad, t, plain)


@pytest.mark.parametrize("g,w,mode", [(16, 48, 0), (16, None, 0), (4, 150, 1), (40, 33, 1), (1, 20, 0)])
@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1)])
def test_infinities_and_nan_anywhere(Hq, Hkv, dtype, d, g, w, mode):
    # values of both signs and NaN in single places, of tokens and of cores: each row shows what it sees, column by column
    c = Case([300, 31, 7, 140], Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, g=g, w=w, mode=mode, first=3, tail=5)
    Kc = Vc = None
    if c.packed.cores:
        Kc, Vc = api.cca_pool_packed(c.Q, c.K, c.V, c.packed)
    rng = np.random.default_rng(g)
    for few in (3, 40):
        V = c.V.clone()
        vc = None if Vc is None else Vc.clone()
        for x, rows in ((V, c.T), (vc, c.T // c.g)):
            if x is None:
                continue
            for k in range(few):
                x[int(rng.integers(Hkv)), int(rng.integers(rows)), int(rng.integers(d))] = (float("inf"), -float("inf"), float("nan"))[k % 3]
        V[:, :3], V[:, -5:] = float("nan"), float("inf")                      # rows of no sequence
        O, L = api.cca_attn_packed(c.Q, c.K, V, Kc, vc, c.packed, dev_status=c.status)
        m = c.inside()
        want = [x[:, m] for x in ref.attention(c.Q, c.K, V, Kc, vc, c.cu, c.g, c.w, c.mode)]
        agree(O[:, m], L[:, m], want, few)
    assert int(c.status) == 0


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64)], ids=["bf16-128", "bf16-64"])
def test_finite_values_whose_sums_overflow(dtype, d):
    # weights of up to 2^16 before they are divided, times the type's largest values: sums overflow, the result does not
    N = 400
    Q, K = rand(2, N, d, dtype=dtype, seed=1, size=0.01), rand(1, N, d, dtype=dtype, seed=2, size=0.01)
    V = torch.full((1, N, d), 1e38, dtype=dtype, device="cuda")
    packed = api.cca_pack(device([0, N]), N, 16)
    O, L = api.cca_attn_packed(Q, K, V, None, None, packed)
    agree(O, L, ref.attention(Q, K, V, None, None, [0, N], 16, N), "large")


def test_keys_that_are_not_finite():
    # a key's NaN or infinity reaches the weights of the rows that see it, and no other row
    for dtype, d in KINDS:
        c = Case([200, 90], Hq=4, Hkv=2, d=d, dtype=dtype, g=16, w=None)
        for bad in (float("nan"), float("inf")):
            K = c.K.clone()
            K[:, 77, 3] = bad
            O, L = api.cca_attn_packed(c.Q, K, c.V, None, None, c.packed, dev_status=c.status)
            clean, lse = api.cca_attn_packed(c.Q, c.K, c.V, None, None, c.packed)
            rows = np.r_[0:77, 200:290]
            assert torch.equal(O[:, rows], clean[:, rows]) and torch.equal(L[:, rows], lse[:, rows])
            if bad != bad:
                assert torch.isnan(O[:, 77:200]).all() and torch.isnan(L[:, 77:200]).all()
        assert int(c.status) == 0


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_mean_pooling_takes_no_weights_from_keys(dtype, d):
    # the mean of a group's values does not depend on its keys
    c = Case([64, 33], Hq=4, Hkv=2, d=d, dtype=dtype, g=8, w=16)
    _, want = api.cca_pool_packed(c.Q, c.K, c.V, c.packed, pool_mode=1)
    for bad in (float("nan"), float("inf"), -float("inf")):
        Q, K = c.Q.clone(), c.K.clone()
        K[:, 5], Q[:, 15] = bad, bad
        Kc, Vc = api.cca_pool_packed(Q, K, c.V, c.packed, pool_mode=1)
        assert torch.equal(Vc, want)
        assert not torch.isfinite(Kc[:, 0]).any() and torch.isfinite(Kc[:, 1:]).all()


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
@pytest.mark.parametrize("g,w", [(16, None), (8, 40)])
def test_tokens_whose_keys_and_values_are_not_finite(g, w, dtype, d):
    # a token of which keys and values have overflowed: for the rows whose score of it is minus infinity its weight is zero, and zero
    # times an infinite value is NaN; the other columns, and cores that hold it, are weighed as ever
    N, bad = 300, (5, 131, 290)
    Q, K, V = (rand(h, N, d, dtype=dtype, seed=i) for i, h in enumerate((4, 2, 2)))
    for t in bad:
        K[:, t, 3], V[:, t, 7], V[:, t, 9] = float("inf"), float("inf"), -float("inf")
    V[:, 60, 7] = float("inf")
    w = N if w is None else w
    packed = api.cca_pack(device([0, N]), N, g, w)
    Kc = Vc = None
    if packed.cores:
        Kc, Vc = (rand(2, N // g, d, dtype=dtype, seed=i) for i in (7, 8))
        Kc[:, 2, 5], Vc[:, 2, 11] = -float("inf"), float("inf")
        Kc[:, 9, 5], Vc[:, 9, 11] = float("inf"), float("inf")
    O, L = api.cca_attn_packed(Q, K, V, Kc, Vc, packed)
    q, k, v, got, lse = (t64(x) for x in (Q, K, V, O, L))
    see = ref.visible(N, g, w, 0)
    tol = 2.0 ** -7 if dtype == BF else 2.0 ** -16       # a weight's and the result's rounding, of values of a few units at most
    with np.errstate(all="ignore"):
        for h in range(4):
            kk, vv = ref.keys(k, v, Kc, Vc, h // 2, 0, N, g)
            for i in range(N):
                s = kk[see[i]] @ q[h, i] * d ** -0.5
                p = np.exp(s - s.max())
                o, x = (p[:, None] * vv[see[i]]).sum(0) / p.sum(), got[h, i]
                assert np.array_equal(np.isnan(x), np.isnan(o)) and np.array_equal(x[np.isinf(o)], o[np.isinf(o)]), (h, i)
                fine = np.isfinite(o)
                assert (np.abs(x - o)[fine] <= tol * np.abs(vv[see[i]][:, fine]).max(initial=1.0)).all(), (h, i)
                assert np.isnan(lse[h, i]) == np.isnan(p.sum())
