"""Packed sequences on the GPU: plan, pooling, attention and gradients against plain 64-bit forms, at the
lengths, strides and values where they can go wrong."""
import numpy as np
import pytest
import torch

import packed_ref as ref
from paged_ref import HALF, close, t64
from sparse_long_context_cca_gb300 import api

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def rand(*shape, dtype=F32, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return (size * torch.randn(shape, generator=g)).to(dtype).cuda()


def offsets(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def device(cu):
    return torch.from_numpy(np.asarray(cu, dtype=np.int32)).cuda()


class Case:
    """Token-major tensors of a batch, as projections leave them, read as [H, T, d]."""

    def __init__(self, lens, Hq=4, Hkv=2, d=128, dtype=BF, g=16, w=64, mode=0, first=0, tail=0, seed=0, size=1.0):
        self.cu = offsets(lens, first)
        self.T = int(self.cu[-1]) + tail
        self.g, self.mode = g, mode
        self.w = self.T if w is None else w
        self.Q = rand(self.T, Hq, d, dtype=dtype, seed=seed, size=size).transpose(0, 1)
        self.K = rand(self.T, Hkv, d, dtype=dtype, seed=seed + 1, size=size).transpose(0, 1)
        self.V = rand(self.T, Hkv, d, dtype=dtype, seed=seed + 2).transpose(0, 1)
        self.dO = rand(self.T, Hq, d, dtype=dtype, seed=seed + 3).transpose(0, 1)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.packed = api.cca_pack(device(self.cu), self.T, g, w, window_mode=mode, dev_status=self.status)
        assert int(self.status) == 0

    def inside(self):
        m = np.zeros(self.T, dtype=bool)
        m[self.cu[0]:self.cu[-1]] = True
        return m

    def check(self, pool_mode=0, backward=True, what=""):
        """Pooling, attention and gradients, each against the formulas at the GPU's own inputs of the step."""
        Kc = Vc = None
        if self.packed.cores:
            Kc, Vc = api.cca_pool_packed(self.Q, self.K, self.V, self.packed, pool_mode=pool_mode, dev_status=self.status)
            k, v, ek, ev = ref.pool(self.Q, self.K, self.V, self.cu, self.g, pool_mode)
            close(Kc, k, ek, what + " Kc")
            close(Vc, v, ev, what + " Vc")
        O, L = torch.full_like(self.Q, 7.0), torch.full(self.Q.shape[:2], 7.0, device="cuda")
        api.cca_attn_packed(self.Q, self.K, self.V, Kc, Vc, self.packed, O, L, dev_status=self.status)
        o, l, eo, el = ref.attention(self.Q, self.K, self.V, Kc, Vc, self.cu, self.g, self.w, self.mode)
        m = self.inside()
        close(O[:, m], o[:, m], eo[:, m], what + " O")
        close(L[:, m], l[:, m], el[:, m], what + " LSE")
        assert (O[:, ~m] == 7).all() and (L[:, ~m] == 7).all()      # rows of no sequence: left as they were
        if backward:
            d = [torch.full_like(t, 7.0) for t in (self.Q, self.K, self.V)]
            api.cca_packed_bwd(self.Q, self.K, self.V, Kc, Vc, O, L, self.dO, self.packed, 0.0, pool_mode, *d, dev_status=self.status)
            want, err = ref.backward(self.Q, self.K, self.V, Kc, Vc, O, L, self.dO, self.cu, self.g, self.w, self.mode, pool_mode)
            for name, x, y, e in zip(("dQ", "dK", "dV"), d, want, err):
                close(x[:, m], y[:, m], e[:, m], f"{what} {name}")
                assert (x[:, ~m] == 7).all()
        assert int(self.status) == 0
        return O, L, Kc, Vc


LENS = [[1], [5], [128], [129], [300], [1, 1, 1], [64, 1, 130, 0, 17], [0, 0, 40], [257, 255, 3], [0]]
KINDS = [(BF, 128), (BF, 64), (F32, 128), (F32, 64)]
IDS = ["bf16-128", "bf16-64", "f32-128", "f32-64"]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_lengths(lens, dtype, d):
    if sum(lens) == 0:
        lens, tail = lens, 3
    else:
        tail = 0
    Case(lens, d=d, dtype=dtype, g=16, w=64, tail=tail).check(what="core + window")
    Case(lens, d=d, dtype=dtype, g=16, w=None, tail=tail).check(what="causal")


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
@pytest.mark.parametrize("g,w,mode", [(1, 1, 0), (1, 20, 1), (4, 7, 1), (16, 130, 0), (40, 33, 1), (200, 50, 1), (7, 129, 0)])
def test_groups_and_windows(g, w, mode, dtype, d):
    Case([210, 3, 330, 77], d=d, dtype=dtype, g=g, w=w, mode=mode, first=5, tail=9).check(what=f"g{g} w{w} mode{mode}")


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 2), (5, 5), (16, 2)])
def test_heads(Hq, Hkv, dtype, d):
    Case([70, 150, 31], Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, g=8, w=48).check(what=f"{Hq} over {Hkv}")


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)], ids=["bf16-128", "f32-64"])
def test_mean_pooling(dtype, d):
    Case([210, 3, 130], d=d, dtype=dtype, g=8, w=40).check(pool_mode=1, what="mean")


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 128)], ids=["bf16-128", "f32-128"])
def test_longer(dtype, d):
    # several tiles of 256 rows, of 128 cores and of query rows per core tile
    Case([1500, 700, 2], Hq=2, Hkv=1, d=d, dtype=dtype, g=4, w=200).check(what="long")


def test_peaked_scores():
    # scores of some hundreds: the running maximum moves by more than any lazy rescaling allows
    for dtype, d in KINDS:
        Case([300, 140], Hq=2, Hkv=1, d=d, dtype=dtype, g=16, w=100, size=8.0).check(backward=False, what="peaked")


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_strides(dtype, d):
    # queries, keys and values of one packed projection, output by token for the next projection
    lens, Hq, Hkv, g, w = [150, 33], 4, 2, 16, 48
    T, cu = sum(lens), offsets(lens)
    qkv = rand(T, (Hq + 2 * Hkv) * d + 64, dtype=dtype)
    view = lambda a, h: qkv[:, a * d:(a + h) * d].view(T, h, d).transpose(0, 1)  # noqa: E731
    Q, K, V = view(0, Hq), view(Hq, Hkv), view(Hq + Hkv, Hkv)
    packed = api.cca_pack(device(cu), T, g, w)
    outs = []
    for q, k, v, O in ((Q, K, V, torch.zeros(T, Hq, d, dtype=dtype, device="cuda").transpose(0, 1)),
                       (*(x.contiguous() for x in (Q, K, V)), None)):
        O, L, Kc, Vc = api.cca_prefill_packed(q, k, v, packed, out=(O, None, None, None))
        dO = rand(Hq, T, d, dtype=dtype, seed=4)
        outs.append((O, L, Kc, Vc, *api.cca_packed_bwd(q, k, v, Kc, Vc, O, L, dO, packed)))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_what_is_masked_does_not_matter(dtype, d):
    # infinities, NaN and the type's lowest value in later tokens, other sequences, cores not seen
    lens, g, w = [140, 37, 200], 16, 48
    c = Case(lens, Hq=2, Hkv=1, d=d, dtype=dtype, g=g, w=w, first=3, tail=6)
    Kc, Vc = api.cca_pool_packed(c.Q, c.K, c.V, c.packed)
    O, L = api.cca_attn_packed(c.Q, c.K, c.V, Kc, Vc, c.packed)
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).min):
        K, V, Q = c.K.clone(), c.V.clone(), c.Q.clone()
        kc, vc = Kc.clone(), Vc.clone()
        a, b = int(c.cu[1]), int(c.cu[2])
        m = a + 20                                 # a token of the second sequence, seen from its own row on
        K[:, m], V[:, m, ::2], Q[:, m] = bad, bad, bad
        K[:, :3], V[:, :3], V[:, -6:], K[:, -6:] = bad, bad, bad, bad      # rows of no sequence
        j = int(c.cu[2]) // g + 5                  # core 5 of the third sequence: seen from row 6 * 16 + 47 on
        kc[:, j], vc[:, j] = bad, bad
        used = {int(x) // g + i for x, y in ref.sequences(c.cu) for i in range((int(y) - int(x)) // g)}
        for row in set(range(c.T // g)) - used:    # core rows of no group
            kc[:, row], vc[:, row] = bad, bad
        O2, L2 = api.cca_attn_packed(Q, K, V, kc, vc, c.packed)
        rows = np.r_[3:m, b:b + 6 * g + w - 1]
        tol = 2 * 2.0 ** -8 if dtype == BF else 2.0 ** -18       # rows may take another way through the kernel: see below
        # a row that sees nothing of it: equal up to the roundings of another order of sums
        d_o = (O2[:, rows].float() - O[:, rows].float()).abs()
        assert not torch.isnan(O2[:, rows]).any() and not torch.isnan(L2[:, rows]).any(), bad
        assert (d_o <= tol * (1 + O[:, rows].float().abs())).all() and (L2[:, rows] - L[:, rows]).abs().max() <= 2.0 ** -16
        if not np.isfinite(bad):
            assert torch.isnan(O2[:, m]).all() and torch.isnan(O2[:, b + 6 * g + w - 1]).any()   # who sees it shows it
            far = V.clone()
            # the plain form agrees on every row, in kind and in value
            o, l, eo, el = ref.attention(Q, K, far, kc, vc, c.cu, g, w)
            inside = c.inside()
            got = t64(O2)[:, inside]
            assert np.array_equal(np.isnan(got), np.isnan(o[:, inside]))


def test_an_infinite_value_is_weighed_as_such():
    # a finite score and an infinite value: the row's output is infinite in that column, earlier rows stay
    for dtype, d in KINDS:
        c = Case([200], Hq=2, Hkv=2, d=d, dtype=dtype, g=16, w=None)
        V = c.V.clone()
        V[:, 130, 3] = float("inf")
        O, _ = api.cca_attn_packed(c.Q, c.K, V, None, None, c.packed)
        assert torch.isinf(O[:, 130:, 3]).all() and torch.isfinite(O[:, :130]).all()
        assert torch.isfinite(O[:, 130:, [0, 1, 2, 4]]).all()


def test_gradients_stay_in_their_sequence():
    for dtype, d in KINDS:
        c = Case([100, 150, 90], Hq=2, Hkv=1, d=d, dtype=dtype, g=16, w=48, seed=3)
        outs = []
        for bad in (False, True):
            Q, K, V, dO = (x.clone() for x in (c.Q, c.K, c.V, c.dO))
            if bad:
                for x in (Q, K, V, dO):
                    x[:, 100:250] = float("nan")
            O, L, Kc, Vc = api.cca_prefill_packed(Q, K, V, c.packed)
            outs.append(api.cca_packed_bwd(Q, K, V, Kc, Vc, O, L, dO, c.packed))
        rows = np.r_[0:100, 250:340]
        for a, b in zip(*outs):
            assert torch.equal(a[:, rows], b[:, rows])


def test_plan_positions_and_changed_lengths():
    T, g = 100, 8
    cu = device([2, 2, 41, 90, 90])
    p = api.cca_pack(cu, T, g, 16)
    pos = np.zeros(T)
    for a, b in ((2, 41), (41, 90)):
        pos[a:b] = np.arange(b - a)
    assert np.array_equal(p.positions.cpu().numpy(), pos) and p.sequences == 4
    # a captured batch serves later lengths of the same offsets
    Q, K, V = (rand(h, T, 64, seed=i) for i, h in enumerate((2, 1, 1)))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        api.cca_prefill_packed(Q, K, V, api.cca_pack(cu, T, g, 16))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        p = api.cca_pack(cu, T, g, 16)
        out = api.cca_prefill_packed(Q, K, V, p)
    for lens in ([2, 2, 41, 90, 90], [0, 30, 30, 31, 100], [0, 100, 100, 100, 100]):
        cu.copy_(device(lens))
        graph.replay()
        torch.cuda.synchronize()
        o, l, eo, el = ref.attention(Q, K, V, out[2], out[3], lens, g, 16)
        m = slice(lens[0], lens[-1])
        close(out[0][:, m], o[:, m], eo[:, m], str(lens))


@pytest.mark.parametrize("cu", [[0, 5, 4, 10], [-1, 5, 10, 10], [0, 5, 10, 41], [3, 2, 1, 0]], ids=str)
def test_bad_lengths_are_reported_and_nothing_is_written(cu):
    T, g, d = 40, 4, 128
    for dtype in (BF, F32):
        Q, K, V = (rand(h, T, d, dtype=dtype, seed=i) for i, h in enumerate((2, 1, 1)))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        p = api.cca_pack(device(cu), T, g, 8, dev_status=status)
        assert int(status) == api.CCA_ERR_INVALID_ARG
        out = [torch.full_like(Q, 3.0), torch.full((2, T), 3.0, device="cuda"), torch.full((1, T // g, d), 3.0, dtype=dtype, device="cuda"),
               torch.full((1, T // g, d), 3.0, dtype=dtype, device="cuda")]
        status.zero_()
        O, L, Kc, Vc = api.cca_prefill_packed(Q, K, V, p, out=out, dev_status=status)
        assert int(status) == api.CCA_ERR_INVALID_ARG
        grads = [torch.full_like(x, 3.0) for x in (Q, K, V)]
        api.cca_packed_bwd(Q, K, V, Kc, Vc, O, L, Q, p, 0.0, 0, *grads, dev_status=status)
        assert all((x == 3).all() for x in (*out, *grads))
        api.cca_packed_clear(p, O)
        assert (O == 0).all()


def test_a_plan_of_other_sizes_is_reported():
    T, d = 40, 64
    Q, K, V = (rand(h, T, d, seed=i) for i, h in enumerate((2, 1, 1)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = api.cca_pack(device([0, 10, 40]), T, 4, 8)
    p.w = 9
    O = torch.full_like(Q, 3.0)
    Kc, Vc = torch.zeros(1, 10, d, device="cuda"), torch.zeros(1, 10, d, device="cuda")
    api.cca_attn_packed(Q, K, V, Kc, Vc, p, O, dev_status=status)
    assert int(status) == api.CCA_ERR_INVALID_ARG and (O == 3).all()


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_autograd_of_a_training_step(dtype, d):
    """norms, rotation, pooling and attention of packed documents, with a tail of padding, against the formulas."""
    lens, Hq, Hkv, g, w = [90, 45, 130], 4, 2, 16, 48
    T, cu = sum(lens) + 11, offsets(lens)
    X = [rand(T, h, d, dtype=dtype, seed=i).transpose(0, 1).requires_grad_() for i, h in enumerate((Hq, Hkv, Hkv))]
    qw, kw = (rand(d, dtype=dtype, seed=i, size=0.2).requires_grad_() for i in (5, 6))
    f = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).cuda()
    packed = api.cca_pack(device(cu), T, g, w)
    dO = rand(Hq, T, d, dtype=dtype, seed=9)
    O = api.cca_attention_packed(*X, packed, inv_freq=f, q_weight=qw, k_weight=kw, offset=1.0)
    got = torch.autograd.grad(O, [*X, qw, kw], dO)
    assert (O[:, cu[-1]:] == 0).all() and all((t[:, cu[-1]:] == 0).all() for t in got[:3])
    # the same step by its parts
    q, k = api.norm_rope(X[0][None], X[1][None], qw, kw, f, positions=packed.positions, offset=1.0)
    qd, kd, vd = q[0].detach(), k[0].detach(), X[2].detach()
    O2, L, Kc, Vc = api.cca_prefill_packed(qd, kd, vd, packed)
    m = slice(0, int(cu[-1]))
    assert torch.equal(O[:, m], O2[:, m])
    o, l, eo, el = ref.attention(qd, kd, vd, Kc, Vc, cu, g, w)
    close(O2[:, m], o[:, m], eo[:, m], "O")
    want, err = ref.backward(qd, kd, vd, Kc, Vc, O2, L, dO, cu, g, w)
    grads = api.cca_packed_bwd(qd, kd, vd, Kc, Vc, O2, L, dO, packed)
    for x, y, e in zip(grads, want, err):
        close(x[:, m], y[:, m], e[:, m], "grads")
    api.cca_packed_clear(packed, *grads)
    back = torch.autograd.grad([q, k], [X[0], X[1], qw, kw], [grads[0][None], grads[1][None]])
    assert torch.equal(got[2], grads[2]) and all(torch.equal(a, b) for a, b in zip((got[0], got[1], got[3], got[4]), back))


def test_gradient_against_differences():
    """fp32 gradients of the whole step (pooling and attention) against central differences of the 64-bit form."""
    lens, Hq, Hkv, d, g, w = [40, 9, 60], 2, 1, 64, 8, 16
    T, cu = sum(lens), offsets(lens)
    X = [rand(h, T, d, seed=i).requires_grad_() for i, h in enumerate((Hq, Hkv, Hkv))]
    dO = rand(Hq, T, d, seed=9)
    packed = api.cca_pack(device(cu), T, g, w)
    got = torch.autograd.grad(api.cca_attention_packed(*X, packed), X, dO)

    def value(q, k, v):
        kc, vc, _, _ = ref.pool(q, k, v, cu, g)
        return float((ref.attention(q, k, v, torch.from_numpy(kc), torch.from_numpy(vc), cu, g, w)[0] * t64(dO)).sum())

    class Wide:     # 64-bit values under an fp32 name: the bounds that come along are not used
        dtype = F32

        def __init__(self, x):
            self.x, self.shape = x, x.shape

        def detach(self):
            return self.x
    rng, h = np.random.default_rng(0), 1e-5
    for _ in range(3):
        u = [torch.from_numpy(rng.standard_normal(t.shape)) for t in X]
        x = [t.detach().cpu().double() for t in X]
        slope = (value(*(Wide(a + h * b) for a, b in zip(x, u))) - value(*(Wide(a - h * b) for a, b in zip(x, u)))) / (2 * h)
        mine = sum(float((a.cpu().double() * b).sum()) for a, b in zip(got, u))
        size = sum(float((a.cpu().double().abs() * b.abs()).sum()) for a, b in zip(got, u))
        # differences are good to h^2 relative, fp32 gradients of some hundred terms to 2^-15 of their magnitudes
        assert abs(mine - slope) <= 2.0 ** -15 * size


def test_results_repeat_and_do_not_depend_on_neighbours():
    # the same to the bit twice, and for a sequence alone and among others
    for dtype, d in KINDS:
        c = Case([300, 170, 60], Hq=4, Hkv=2, d=d, dtype=dtype, g=8, w=64, seed=2)
        a = api.cca_prefill_packed(c.Q, c.K, c.V, c.packed)
        g1 = api.cca_packed_bwd(c.Q, c.K, c.V, a[2], a[3], a[0], a[1], c.dO, c.packed)
        g2 = api.cca_packed_bwd(c.Q, c.K, c.V, a[2], a[3], a[0], a[1], c.dO, c.packed)
        assert all(torch.equal(x, y) for x, y in zip(g1, g2))
        rows = slice(300, 470)
        q, k, v = (x[:, rows].contiguous() for x in (c.Q, c.K, c.V))
        one = api.cca_prefill_packed(q, k, v, api.cca_pack(device([0, 170]), 170, 8, 64))
        assert torch.equal(one[0], a[0][:, rows]) and torch.equal(one[1], a[1][:, rows])


def test_two_streams_and_other_workspaces():
    c = Case([500, 200], Hq=4, Hkv=2, d=128, dtype=BF, g=16, w=100)
    want = api.cca_prefill_packed(c.Q, c.K, c.V, c.packed)
    grads = api.cca_packed_bwd(c.Q, c.K, c.V, want[2], want[3], want[0], want[1], c.dO, c.packed)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        o = api.cca_prefill_packed(c.Q, c.K, c.V, c.packed, stream=s)
        outs.append((o, api.cca_packed_bwd(c.Q, c.K, c.V, o[2], o[3], o[0], o[1], c.dO, c.packed, stream=s)))
    torch.cuda.synchronize()
    for o, g in outs:
        assert all(torch.equal(x, y) for x, y in zip((*o, *g), (*want, *grads)))


def test_many_short_sequences():
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 6, 700).tolist()
    for dtype, d in ((BF, 128), (F32, 64)):
        Case(lens, Hq=2, Hkv=1, d=d, dtype=dtype, g=2, w=3).check(what="short")


def test_refusals():
    T, d = 40, 128
    Q, K, V = (rand(h, T, d, dtype=BF, seed=i) for i, h in enumerate((4, 2, 2)))
    cu = device([0, 40])
    p = api.cca_pack(cu, T, 16, 8)
    with pytest.raises(ValueError):
        api.cca_pack(cu.long(), T)
    with pytest.raises(ValueError):
        api.cca_pack(cu[:1], T)
    with pytest.raises(ValueError):
        api.cca_pack(cu, 0)
    with pytest.raises(ValueError):
        api.cca_pack(cu.cpu(), T)
    with pytest.raises(api.CcaError):
        api.cca_pack(cu, T, 16, 0)
    with pytest.raises(api.CcaError):
        api.cca_pack(cu, T, 16, 8, window_mode=2)
    with pytest.raises(ValueError):
        api.cca_pool_packed(Q[:, :39], K[:, :39], V[:, :39], p)          # another number of tokens
    with pytest.raises(ValueError):
        api.cca_pool_packed(Q, K.float(), V, p)
    with pytest.raises(ValueError):
        api.cca_pool_packed(Q, K, V[:1], p)
    with pytest.raises(api.CcaError) as e:
        api.cca_pool_packed(Q, K, V, p, pool_mode=2)
    assert e.value.status == api.CCA_ERR_UNSUPPORTED
    with pytest.raises(api.CcaError):
        api.cca_attn_packed(Q, K, V, None, None, p)                      # cores are seen, none are given
    with pytest.raises(api.CcaError):
        api.cca_attn_packed(Q[:3], K, V, None, None, api.cca_pack(cu, T))    # heads that do not divide
    with pytest.raises(api.CcaError):
        api.cca_attn_packed(Q, K, V, None, None, api.cca_pack(cu, T), O=Q)   # over its own input
    with pytest.raises(ValueError):
        api.cca_attn_packed(Q.transpose(1, 2), K.transpose(1, 2), V.transpose(1, 2), None, None, api.cca_pack(cu, d))
    with pytest.raises(ValueError):
        api.cca_attn_packed(Q, K, V, None, None, api.cca_pack(cu, T), O=torch.empty_like(Q).requires_grad_())
    with pytest.raises(ValueError):
        api.cca_attention_packed(Q, K, V, p, positions=p.positions)      # rotary arguments without frequencies
    O, L, Kc, Vc = api.cca_prefill_packed(Q, K, V, p)
    with pytest.raises(ValueError):
        api.cca_packed_bwd(Q, K, V, Kc, Vc, O, L, Q, p, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(api.CcaError):
        api.cca_packed_bwd(Q, K, V, Kc, Vc, O, L, Q, p, dK=torch.empty(2, 1, d, dtype=BF, device="cuda").expand(2, T, d))
    with pytest.raises(ValueError):
        api.cca_attn_packed(Q.half(), K.half(), V.half(), None, None, p)


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_gradients_take_nothing_from_the_workspace(dtype, d):
    # a workspace full of NaN, many times: warps of a tile that are ahead of others must not hand it on early
    c = Case([1500, 700, 2], Hq=2, Hkv=1, d=d, dtype=dtype, g=4, w=200)
    O, L, Kc, Vc = api.cca_prefill_packed(c.Q, c.K, c.V, c.packed)
    first = None
    for _ in range(60):
        ws = torch.full((32 << 20,), 255, dtype=torch.uint8, device="cuda")
        g = api.cca_packed_bwd(c.Q, c.K, c.V, Kc, Vc, O, L, c.dO, c.packed, workspace=ws)
        first = g if first is None else first
        assert all(torch.equal(a, b) and not torch.isnan(a).any() for a, b in zip(g, first))


def test_a_plan_of_another_number_of_sequences_is_reported():
    # where the lists lie depends on the number: a plan is read only by calls of the same
    T, d = 64, 64
    cu = device([0, 10, 20, 30, 64])
    Q, K, V = (rand(h, T, d, seed=i) for i, h in enumerate((2, 1, 1)))
    p = api.cca_pack(cu, T, 4, T)
    other = api.load_library().cca_pack_size(3, T, 4)
    q = api.Packed(p.plan[:other], p.positions, 3, T, 4, T, 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    O, L = torch.full_like(Q, 3.0), torch.full((2, T), 3.0, device="cuda")
    api.cca_attn_packed(Q, K, V, None, None, q, O, L, dev_status=status)
    assert int(status) == api.CCA_ERR_INVALID_ARG and (O == 3).all() and (L == 3).all()


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_broadcast_tensors(dtype, d):
    # heads or tokens that share memory: refused by the calls, copied by the function with gradients
    T = 50
    packed = api.cca_pack(device([0, 20, 50]), T, 4, 8)
    Q = rand(4, T, d, dtype=dtype, seed=1)
    one = rand(1, T, d, dtype=dtype, seed=2)
    wide = one.expand(2, T, d)
    with pytest.raises(api.CcaError):
        api.cca_pool_packed(Q, wide, wide, packed)
    with pytest.raises(api.CcaError):
        api.cca_attn_packed(Q, rand(2, 1, d, dtype=dtype).expand(2, T, d), wide.contiguous(), None, None, api.cca_pack(device([0, T]), T))
    x = [Q.clone().requires_grad_(), one.clone().requires_grad_(), one.clone().requires_grad_()]
    y = [t.detach().clone().requires_grad_() for t in (Q, wide, wide)]
    dO = rand(1, T, d, dtype=dtype, seed=5).expand(4, T, d)
    a = torch.autograd.grad(api.cca_attention_packed(x[0], x[1].expand(2, T, d), x[2].expand(2, T, d), packed), x, dO)
    b = torch.autograd.grad(api.cca_attention_packed(*y, packed), y, dO.contiguous())
    assert torch.equal(a[0], b[0])
    for i in (1, 2):
        close(a[i], t64(b[i]).sum(0, keepdims=True), 2 * HALF[dtype] * np.abs(t64(b[i])).sum(0, keepdims=True), "sum over heads")
    z = y[0].detach().requires_grad_()
    api.cca_attention_packed(z, *(t.detach() for t in y[1:]), packed).sum().backward()      # a gradient of one element
    assert torch.isfinite(z.grad).all()


def test_a_plan_made_anew_before_the_backward_pass_is_refused():
    T, d = 60, 64
    X = [rand(h, T, d, seed=i).requires_grad_() for i, h in enumerate((2, 1, 1))]
    f = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).cuda()
    for freq in (None, f):
        p = api.cca_pack(device([0, 20, 60]), T, 4, 8)
        O = api.cca_attention_packed(*X, p, inv_freq=freq)
        api.cca_pack(device([0, 30, 60]), T, 4, 8, plan=p.plan)
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            torch.autograd.grad(O.sum(), X)


@pytest.mark.parametrize("r", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("d", [128, 64])
def test_short_sequences_that_share_a_tile(r, d):
    # the query heads of a short sequence stand below one another in a tile: lengths around 32, 64, 128, 256
    lens = [31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1, 2]
    for g, w in ((16, None), (4, 24)):
        Case(lens, Hq=2 * r, Hkv=2, d=d, g=g, w=w, first=3, tail=2, seed=r).check(what=f"r={r} w={w}")


def test_offsets_beyond_32_bits():
    # tokens of one wide buffer each: the last rows lie more than 2^31 elements behind the first
    T, W, d = 66000, 34000, 128
    lens = [300, 65400, 290]
    assert (T - 1) * W > 2 ** 31
    cu = offsets(lens, 5)
    buffers = [torch.zeros(T, W, dtype=BF, device="cuda") for _ in range(3)]
    packed = api.cca_pack(device(cu), T, 16, 200)
    near = [rand(T, h, d, dtype=BF, seed=i).transpose(0, 1) for i, h in enumerate((2, 1, 1, 2))]

    def far(k, h, src=None):
        x = buffers[k // 2][:, W - (k % 2 + 1) * 1024:][:, :h * d].unflatten(1, (h, d)).transpose(0, 1)
        if src is not None:
            x.copy_(src)
        return x
    Q, K, V, dO = (far(i, near[i].shape[0], near[i]) for i in range(4))
    a = api.cca_prefill_packed(*near[:3], packed)
    O = far(4, 2)
    b = api.cca_prefill_packed(Q, K, V, packed, out=(O, None, None, None))
    m = slice(int(cu[0]), int(cu[-1]))
    assert all(torch.equal(x[:, m], y[:, m]) for x, y in zip(a[:2], b[:2])) and torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
    ga = api.cca_packed_bwd(*near[:3], a[2], a[3], a[0], a[1], near[3], packed)
    gb = api.cca_packed_bwd(Q, K, V, b[2], b[3], O, b[1], dO, packed, dQ=far(5, 2))
    assert all(torch.equal(x[:, m], y[:, m]) for x, y in zip(ga, gb))
    api.cca_packed_clear(packed, O)
    assert (O[:, :5] == 0).all() and (O[:, int(cu[-1]):] == 0).all() and torch.equal(O[:, m], a[0][:, m])
    # the last sequence and the first are small enough for the formulas
    for s in (0, 2):
        rows = slice(int(cu[s]), int(cu[s + 1]))
        c = slice(int(cu[s]) // 16, int(cu[s]) // 16 + lens[s] // 16)
        o, l, eo, el = ref.attention(*(x[:, rows] for x in near[:3]), a[2][:, c], a[3][:, c], [0, lens[s]], 16, 200)
        close(O[:, rows], o, eo, "O")
        close(b[1][:, rows], l, el, "LSE")


def test_a_captured_training_step():
    # forward and backward in one graph, replayed for other inputs and lengths
    T, Hq, Hkv, d, g, w = 300, 4, 2, 128, 16, 48
    X = [rand(T, h, d, dtype=BF, seed=i).transpose(0, 1) for i, h in enumerate((Hq, Hkv, Hkv))]
    cu, dO = device([0, 100, 300]), rand(Hq, T, d, dtype=BF, seed=8)
    leaves = [x.detach().requires_grad_() for x in X]

    def step():
        O = api.cca_attention_packed(*leaves, api.cca_pack(cu, T, g, w))
        return (O, *torch.autograd.grad(O, leaves, dO))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    leaves = [x.detach().requires_grad_() for x in leaves]      # no eager graph holds these
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    for k, lens in enumerate(([0, 100, 300], [3, 290, 296], [0, 0, 17])):
        cu.copy_(device(lens))
        with torch.no_grad():
            for i, x in enumerate(leaves):
                x.copy_(rand(T, x.shape[0], d, dtype=BF, seed=20 * k + i).transpose(0, 1))
        graph.replay()
        torch.cuda.synchronize()
        eager = [x.detach().clone().requires_grad_() for x in leaves]
        O = api.cca_attention_packed(*eager, api.cca_pack(device(lens), T, g, w))
        assert all(torch.equal(a, b) for a, b in zip(out, (O, *torch.autograd.grad(O, eager, dO))))


def test_a_backward_pass_is_not_captured_while_an_eager_graph_holds_its_leaves():
    T, d = 60, 64
    X = [rand(h, T, d, seed=i).requires_grad_() for i, h in enumerate((2, 1, 1))]
    dO = rand(2, T, d, seed=7)

    def step():
        O = api.cca_attention_packed(*X, api.cca_pack(cu, T, 4, 8))
        return O, torch.autograd.grad(O, X, dO)
    cu = device([0, 25, T])
    held, want = step()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="being captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            step()
    del held
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()[1]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d", [128, 64])
def test_waits_that_run_out_are_reported(d):
    # with no queries copied the first wait of every kernel ends; the next calls are right
    lib = api.load_library()
    c = Case([500, 300, 40], Hq=4, Hkv=2, d=d, g=16, w=100)
    O, L, Kc, Vc = api.cca_prefill_packed(c.Q, c.K, c.V, c.packed)
    for call in (lambda: api.cca_attn_packed(c.Q, c.K, c.V, Kc, Vc, c.packed, dev_status=c.status),
                 lambda: api.cca_packed_bwd(c.Q, c.K, c.V, Kc, Vc, O, L, c.dO, c.packed, dev_status=c.status)):
        torch.cuda.synchronize()
        lib.cca_test_set_wait_limit_ns(20_000_000)
        lib.cca_test_skip_q_load(1)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            lib.cca_test_skip_q_load(0)
            lib.cca_test_set_wait_limit_ns(1_000_000_000)
        assert int(c.status) == api.CCA_ERR_TIMEOUT
        c.status.zero_()
        c.check(what="after a time-out")


def test_thousands_of_sequences():
    # the plan of many sequences, against one built on the host
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 9000)
    lens[4000] = 70001
    cu, g, w = offsets(lens, 7), 8, 16
    T = int(cu[-1]) + 9
    p = api.cca_pack(device(cu), T, g, w)
    h = p.plan.view(torch.int32).cpu().numpy()
    assert h[1] == T and h[5] == 9000 and h[6] == 7 and h[7] == cu[-1]
    seen = np.maximum(lens - w, 0) // g
    at = 16
    for list_, size in enumerate((-(-lens // 256), -(-lens // 128), -(-seen // 128))):
        order = sorted(((int(k), -int(n), s) for s, (n, t) in enumerate(zip(lens, size)) for k in range(t)), key=lambda x: (-x[0], x[1], x[2]))
        want = np.array([[cu[s], -n, k, cu[s] // g] for k, n, s in order])
        assert h[8 + list_] == len(want)
        assert np.array_equal(h[at:at + 4 * len(want)].reshape(-1, 4), want)
        at += 4 * ((T // 256, T // 128, T // g // 128)[list_] + 9000)
    pos = np.zeros(T)
    for a, n in zip(cu, lens):
        pos[a:a + n] = np.arange(n)
    assert np.array_equal(p.positions.cpu().numpy(), pos)


def test_slices_of_one_projection():
    # inputs from one tensor, gradients into another: the same as apart; slices that do share columns are refused
    lens, Hq, Hkv, d, g, w = [90, 33, 200], 4, 2, 128, 16, 48
    T, H = sum(lens), Hq + 2 * Hkv
    for dtype in (BF, F32):
        x = rand(T, H, d, dtype=dtype)
        Q, K, V = (x[:, a:b].transpose(0, 1) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, H)))
        packed = api.cca_pack(device(offsets(lens)), T, g, w)
        O, L, Kc, Vc = api.cca_prefill_packed(Q, K, V, packed)
        dO = rand(Hq, T, d, dtype=dtype, seed=3)
        want = api.cca_packed_bwd(Q, K, V, Kc, Vc, O, L, dO, packed)
        dx = torch.zeros(T, H, d, dtype=dtype, device="cuda")
        grads = [dx[:, a:b].transpose(0, 1) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, H))]
        got = api.cca_packed_bwd(Q, K, V, Kc, Vc, O, L, dO, packed, dQ=grads[0], dK=grads[1], dV=grads[2])
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(torch.cat(want).transpose(0, 1), dx)
        for a in (Hq - 1, Hq + 1):
            with pytest.raises(api.CcaError):
                api.cca_packed_bwd(Q, K, V, Kc, Vc, O, L, dO, packed, dQ=grads[0] if a < Hq else None, dK=dx[:, a:a + Hkv].transpose(0, 1), dV=grads[2])
        with pytest.raises(api.CcaError):
            api.cca_attn_packed(Q, K, V, Kc, Vc, packed, O=x[:, 1:1 + Hq].transpose(0, 1))


@pytest.mark.parametrize("g,w,mode", [(2 ** 31 - 1, 2 ** 31 - 1, 0), (2 ** 31 - 1, 5, 1), (16, 2 ** 31 - 1, 1), (300, 7, 0), (90, 1, 1)])
def test_groups_and_windows_of_any_size(g, w, mode):
    # groups that no sequence fills, windows past every length
    for dtype, d in ((BF, 128), (F32, 64)):
        c = Case([130, 7, 95], Hq=4, Hkv=2, d=d, dtype=dtype, g=g, w=w, mode=mode)
        if c.packed.cores and g > c.T:
            raise AssertionError("no group fits")
        c.check(what=f"g={g} w={w}")
        Kc, Vc = api.cca_pool_packed(c.Q, c.K, c.V, c.packed)
        assert Kc.shape == Vc.shape == (2, c.T // g, d)


def test_inputs_of_which_some_need_gradients():
    T, d = 90, 128
    packed = api.cca_pack(device([0, 40, T]), T, 8, 16)
    X = [rand(T, h, d, dtype=BF, seed=i).transpose(0, 1) for i, h in enumerate((4, 2, 2))]
    dO = rand(4, T, d, dtype=BF, seed=5)
    whole = [x.detach().clone().requires_grad_() for x in X]
    want = torch.autograd.grad(api.cca_attention_packed(*whole, packed), whole, dO)
    for k in range(3):
        some = [x.detach().clone().requires_grad_(i == k) for i, x in enumerate(X)]
        got, = torch.autograd.grad(api.cca_attention_packed(*some, packed), some[k], dO)
        assert torch.equal(got, want[k])
    with torch.no_grad():
        assert not api.cca_attention_packed(*whole, packed).requires_grad
    again = torch.autograd.grad(api.cca_attention_packed(*whole, packed), whole[0], dO, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        torch.autograd.grad(again.float().square().sum(), whole[0])


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("w,g", [(None, 16), (900, 4)])
def test_keys_whose_rows_are_shared_by_two_items(w, g, d):
    # eight query heads over one: long tiles of keys are dealt out in halves, whoever ends second adds them up
    c = Case([1300, 40, 900], Hq=8, Hkv=1, d=d, g=g, w=w, first=2, tail=3)
    O, L, Kc, Vc = c.check(what="halves")
    want = api.cca_packed_bwd(c.Q, c.K, c.V, Kc, Vc, O, L, c.dO, c.packed, dQ=torch.zeros_like(c.Q), dK=torch.zeros_like(c.K), dV=torch.zeros_like(c.V))
    for _ in range(30):
        ws = torch.full((48 << 20,), 255, dtype=torch.uint8, device="cuda")
        got = api.cca_packed_bwd(c.Q, c.K, c.V, Kc, Vc, O, L, c.dO, c.packed, workspace=ws, dQ=torch.zeros_like(c.Q), dK=torch.zeros_like(c.K),
                                 dV=torch.zeros_like(c.V))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
