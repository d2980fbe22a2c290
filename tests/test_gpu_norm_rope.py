"""Norms of queries and keys with their rotation on the GPU: against the formulas in 64 bits, gradients against
the formulas and against differences, strides, the storing form, graphs, streams and refusals."""
import numpy as np
import pytest
import torch

from packed_ref import HALF, norm_rope, norm_rope_backward
from paged_ref import close, t64
from sparse_long_context_cca_gb300 import api

pytestmark = pytest.mark.gpu


def freqs(rot, base=10000.0):
    return (base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)).cuda()


def rand(*shape, dtype=torch.float32, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return (size * torch.randn(shape, generator=g)).to(dtype).cuda()


def weights(H, d, per_head, dtype, seed=5):
    return rand(*((H, d) if per_head else (d,)), dtype=dtype, seed=seed, size=0.3)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (64, 32), (128, 24), (64, 10), (128, 2), (64, 0)])
def test_matches_definition(d, rot, dtype, layout):
    B, Hq, Hkv, N = 2, 5, 2, 37
    Q, K = rand(B, Hq, N, d, dtype=dtype, size=3.0), rand(B, Hkv, N, d, dtype=dtype, seed=1)
    f = freqs(rot) if rot else None
    fr = [] if f is None else f.cpu()
    pos = np.broadcast_to(100 + np.arange(N), (B, N))
    for per_head, wt, offset in ((False, dtype, 1.0), (True, torch.float32, 0.0)):
        qw, kw = weights(Hq, d, per_head, wt), weights(Hkv, d, per_head, wt, 9)
        q, k = api.cca_norm_rope(Q, K, qw, kw, f, start=100, layout=layout, factor=1.25, offset=offset, eps=1e-5)
        for name, x, w, y in (("Q", Q, qw, q), ("K", K, kw, k)):
            close(y, *norm_rope(x, w, pos, fr, layout, 1.25, 1e-5, offset), f"{name} d{d} rot{rot} {layout} {per_head}")


@pytest.mark.parametrize("N", [1, 2, 7, 300, 4099])
def test_lengths_one_tensor_and_no_weights(N):
    Q = rand(1, 2, N, 128, dtype=torch.bfloat16)
    f = freqs(128)
    q, k = api.cca_norm_rope(Q, None, None, None, f)
    assert k is None
    close(q, *norm_rope(Q, None, np.arange(N)[None], f.cpu()), f"N{N}")


def test_one_tensor_of_each_kind_of_weight():
    # shared weights beside weights for each head, and none beside some
    B, N, d = 1, 9, 128
    Q, K = rand(B, 6, N, d), rand(B, 3, N, d, seed=1)
    pos = np.arange(N)[None]
    f = freqs(d)
    for qw, kw in ((weights(6, d, True, torch.float32), weights(3, d, False, torch.float32)),
                   (None, weights(3, d, True, torch.float32)), (weights(6, d, False, torch.float32), None)):
        q, k = api.cca_norm_rope(Q, K, qw, kw, f)
        close(q, *norm_rope(Q, qw, pos, f.cpu()), "Q")
        close(k, *norm_rope(K, kw, pos, f.cpu()), "K")


def test_rows_of_zeros_and_extremes():
    d = 64
    Q = rand(1, 1, 4, d)
    Q[0, 0, 0] = 0
    Q[0, 0, 1] = 1e-15      # below eps: the row is divided by sqrt(eps)
    Q[0, 0, 2] *= 1e15
    q, _ = api.cca_norm_rope(Q, None, None, None, freqs(d), eps=1e-6)
    close(q, *norm_rope(Q, None, np.arange(4)[None], freqs(d).cpu()), "rows")
    assert (q[0, 0, 0] == 0).all()
    Q[0, 0, 3, 5] = float("nan")
    q2, _ = api.cca_norm_rope(Q, None, None, None, freqs(d), eps=1e-6)
    assert torch.isnan(q2[0, 0, 3]).all() and torch.equal(q2[0, 0, :3], q[0, 0, :3])   # a row's own affair


def test_far_and_negative_positions():
    B, H, N, d = 2, 2, 64, 64
    Q = rand(B, H, N, d)
    pos = np.random.default_rng(3).integers(-2 ** 31, 2 ** 31 - 1, (B, N)).astype(np.int32)
    f = freqs(d)
    q, _ = api.cca_norm_rope(Q, None, None, None, f, positions=torch.from_numpy(pos).cuda())
    close(q, *norm_rope(Q, None, pos, f.cpu()), "per sequence")
    q, _ = api.cca_norm_rope(Q, None, None, None, f, positions=torch.from_numpy(pos[0]).cuda())
    close(q, *norm_rope(Q, None, np.broadcast_to(pos[0], (B, N)), f.cpu()), "shared")


def test_projection_layout_and_packed_in_place():
    B, N, Hq, Hkv, d = 2, 19, 4, 2, 64
    packed = rand(B, N, (Hq + 2 * Hkv) * d, dtype=torch.bfloat16).contiguous()
    view = lambda a, h: packed[..., a * d:(a + h) * d].view(B, N, h, d).transpose(1, 2)  # noqa: E731
    Q, K = view(0, Hq), view(Hq, Hkv)
    f, qw, kw = freqs(d), weights(Hq, d, False, torch.bfloat16), weights(Hkv, d, False, torch.bfloat16, 7)
    pos = np.broadcast_to(np.arange(N), (B, N))
    want = [norm_rope(Q, qw, pos, f.cpu()), norm_rope(K, kw, pos, f.cpu())]
    rest = packed[..., (Hq + Hkv) * d:].clone()
    q, k = api.cca_norm_rope(Q, K, qw, kw, f)
    assert q.is_contiguous() and k.is_contiguous()
    close(q, *want[0], "Q")
    close(k, *want[1], "K")
    api.cca_norm_rope(Q, K, qw, kw, f, out=(Q, K))
    assert torch.equal(Q, q) and torch.equal(K, k) and torch.equal(packed[..., (Hq + Hkv) * d:], rest)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,rot,per_head,wide", [(128, 128, False, False), (64, 24, True, True), (128, 20, False, True),
                                                 (64, 64, True, False), (64, 0, False, False)])
def test_gradients(d, rot, per_head, wide, dtype, layout):
    B, Hq, Hkv, N = 2, 5, 2, 33
    wt = torch.float32 if wide else dtype
    Q, K = rand(B, Hq, N, d, dtype=dtype, size=2.0), rand(B, Hkv, N, d, dtype=dtype, seed=1)
    qw, kw = weights(Hq, d, per_head, wt), weights(Hkv, d, per_head, wt, 9)
    f = freqs(rot) if rot else None
    fr = [] if f is None else f.cpu()
    pos = torch.tensor(np.random.default_rng(1).integers(0, 500, (B, N)), dtype=torch.int32).cuda()
    leaves = [t.requires_grad_() for t in (Q, K, qw, kw)]
    q, k = api.norm_rope(*leaves, f, positions=pos, layout=layout, factor=1.1, offset=1.0, eps=1e-5)
    dq, dk = rand(B, Hq, N, d, dtype=dtype, seed=2), rand(B, Hkv, N, d, dtype=dtype, seed=3)
    got = torch.autograd.grad([q, k], leaves, [dq, dk])
    for i, (x, w, dy) in enumerate(((Q, qw, dq), (K, kw, dk))):
        close((q, k)[i].detach(), *norm_rope(x, w, pos.cpu(), fr, layout, 1.1, 1e-5, 1.0), "forward")
        (dx, dw), (ex, ew) = norm_rope_backward(x, dy, w, pos.cpu(), fr, layout, 1.1, 1e-5, 1.0)
        if not per_head:
            dw, ew = dw.sum(0), ew.sum(0) + x.shape[1] * 2.0 ** -24 * np.abs(dw).sum(0)
        close(got[i], dx, ex, "dx")
        close(got[2 + i], dw, ew + HALF[wt] * (np.abs(dw) + ew), "dw")


def test_many_rows_and_heads_and_repeats():
    # more rows than blocks, head groups, and sums that repeat to the bit
    B, Hq, Hkv, N, d = 1, 24, 8, 2500, 64
    Q, K = rand(B, Hq, N, d).requires_grad_(), rand(B, Hkv, N, d, seed=1).requires_grad_()
    for per_head in (False, True):
        qw, kw = weights(Hq, d, per_head, torch.float32).requires_grad_(), weights(Hkv, d, per_head, torch.float32, 3).requires_grad_()
        f, dq, dk = freqs(d), rand(B, Hq, N, d, seed=2), rand(B, Hkv, N, d, seed=3)
        runs = []
        for _ in range(2):
            q, k = api.norm_rope(Q, K, qw, kw, f)
            runs.append(torch.autograd.grad([q, k], [Q, K, qw, kw], [dq, dk]))
        assert all(torch.equal(a, b) for a, b in zip(*runs))
        for i, (x, w, dy) in enumerate(((Q, qw, dq), (K, kw, dk))):
            (dx, dw), (ex, ew) = norm_rope_backward(x, dy, w, np.arange(N)[None], f.cpu())
            if not per_head:
                dw, ew = dw.sum(0), ew.sum(0) + x.shape[1] * 2.0 ** -24 * np.abs(dw).sum(0)
            close(runs[0][i], dx, ex, "dx")
            close(runs[0][2 + i], dw, ew + HALF[torch.float32] * (np.abs(dw) + ew), "dw")


def test_gradient_against_differences():
    B, H, N, d = 1, 2, 5, 64
    Q, qw = rand(B, H, N, d), weights(H, d, False, torch.float32)
    f, dq = freqs(d), rand(B, H, N, d, seed=2)
    Q.requires_grad_(), qw.requires_grad_()
    q, _ = api.norm_rope(Q, None, qw, None, f, factor=1.1, offset=1.0)
    gx, gw = torch.autograd.grad(q, [Q, qw], dq)
    rng = np.random.default_rng(0)
    pos = np.arange(N)[None]
    value = lambda x, w: float((norm_rope(x, w, pos, f.cpu(), "half", 1.1, 1e-6, 1.0)[0] * t64(dq)).sum())  # noqa: E731
    for _ in range(4):
        ux, uw = torch.from_numpy(rng.standard_normal(Q.shape)), torch.from_numpy(rng.standard_normal(qw.shape))
        x, w, h = Q.detach().cpu().double(), qw.detach().cpu().double(), 1e-5
        slope = (value_of(value, x + h * ux, w + h * uw) - value_of(value, x - h * ux, w - h * uw)) / (2 * h)
        mine = float((gx.cpu().double() * ux).sum() + (gw.cpu().double() * uw).sum())
        # central differences of a smooth function in 64 bits are good to h^2 = 1e-10 relative, fp32 gradients to 2^-17
        assert abs(mine - slope) <= 2.0 ** -17 * float((gx.cpu().double().abs() * ux.abs()).sum() + (gw.cpu().double().abs() * uw.abs()).sum())


def value_of(value, x, w):
    class Wide:     # a 64-bit tensor under an fp32 name: the bound that comes along is not used
        dtype, shape = torch.float32, x.shape

        def detach(self):
            return x
    return value(Wide(), w)


def test_gradients_of_some_and_of_broadcast():
    B, Hq, Hkv, N, d = 1, 2, 1, 6, 64
    f, qw, kw = freqs(d), weights(Hq, d, False, torch.float32), weights(Hkv, d, False, torch.float32, 2)
    K0, Q0 = rand(B, Hkv, N, d), rand(B, Hq, N, d, seed=4)
    full = [t.clone().requires_grad_() for t in (Q0, K0, qw, kw)]
    want = torch.autograd.grad([x.sum() for x in api.norm_rope(*full, f)], full)
    for pick in ((0,), (1,), (2,), (3,), (1, 2), (0, 3)):
        leaves = [t.clone().requires_grad_(i in pick) for i, t in enumerate((Q0, K0, qw, kw))]
        out = api.norm_rope(*leaves, f)
        got = torch.autograd.grad([x.sum() for x in out if x.requires_grad], [leaves[i] for i in pick])
        assert all(torch.equal(a, want[i]) for a, i in zip(got, pick)), pick
    # only the keys are used: the queries' gradient is zero
    q, k = api.norm_rope(*full, f)
    got = torch.autograd.grad(k.sum(), full)
    assert (got[0] == 0).all() and (got[2] == 0).all() and torch.equal(got[1], want[1])
    # one key head seen by all query heads
    one = K0.clone().requires_grad_()
    _, k = api.norm_rope(Q0, one.expand(B, 3, N, d), None, None, f)
    g, = torch.autograd.grad(k.sum(), one)
    single = K0.clone().requires_grad_()
    _, k1 = api.norm_rope(Q0, single, None, None, f)
    g1, = torch.autograd.grad(k1.sum(), single)
    assert torch.allclose(g, 3 * g1, rtol=2.0 ** -20, atol=0)


def test_no_second_derivative():
    Q = rand(1, 1, 3, 64).requires_grad_()
    q, _ = api.norm_rope(Q, None, None, None, freqs(64))
    with pytest.raises(RuntimeError):
        torch.autograd.grad(q.sum(), Q, create_graph=True)


def append_case(B, T, Hq, Hkv, d, dtype, rows, lens, seed=0):
    cols = (max(lens) + T + rows - 1) // rows
    Kp, Vp = rand(B * cols, Hkv, rows, d, dtype=dtype, seed=seed), rand(B * cols, Hkv, rows, d, dtype=dtype, seed=seed + 1)
    order = torch.randperm(B * cols, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    return Kp, Vp, order.view(B, cols).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,d,rot,T,per_head", [(torch.bfloat16, 128, 128, 1, False), (torch.bfloat16, 64, 24, 7, True),
                                                    (torch.float32, 128, 64, 5, False), (torch.float32, 64, 0, 33, True)])
def test_append(dtype, d, rot, T, per_head, layout):
    B, Hq, Hkv, rows = 3, 6, 2, 16
    lens = [0, 13, 40]
    Kp, Vp, table, ln = append_case(B, T, Hq, Hkv, d, dtype, rows, lens)
    Q, K, V = rand(B, T, Hq, d, dtype=dtype).transpose(1, 2), rand(B, T, Hkv, d, dtype=dtype, seed=1).transpose(1, 2), rand(B, T, Hkv, d, dtype=dtype, seed=2).transpose(1, 2)
    qw, kw = weights(Hq, d, per_head, dtype), weights(Hkv, d, per_head, dtype, 4)
    f = freqs(rot) if rot else None
    fr = [] if f is None else f.cpu()
    counts = torch.tensor([T, max(T - 2, 0), T], dtype=torch.int32).cuda()
    wantK, wantV = t64(Kp), t64(Vp)
    bound = np.zeros_like(wantK)
    pos = np.array(lens)[:, None] + np.arange(T)
    k64, ek = norm_rope(K, kw, pos, fr, layout, 1.1, 1e-6, 1.0)
    for b in range(B):
        for t in range(int(counts[b])):
            p, r = int(table[b, (lens[b] + t) // rows]), (lens[b] + t) % rows
            wantK[p, :, r], bound[p, :, r], wantV[p, :, r] = k64[b, :, t], ek[b, :, t], t64(V)[b, :, t]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = api.cca_norm_rope_append(Q, K, V, Kp, Vp, table, ln, qw, kw, f, counts=counts, layout=layout, factor=1.1, offset=1.0, dev_status=status)
    assert int(status) == 0
    close(Kp, wantK, bound, "K pages")
    assert np.array_equal(t64(Vp), wantV)
    y, e = norm_rope(Q, qw, pos, fr, layout, 1.1, 1e-6, 1.0)
    for b in range(B):
        y[b, :, int(counts[b]):], e[b, :, int(counts[b]):] = 0, 0
    close(q, y, e, "Q")


def test_append_of_a_tree_equals_norm_then_rope_append():
    # a drafted tree: the same as norming first and storing by cca_rope_append (which is tested by itself)
    B, T, Hq, Hkv, d, rows = 2, 6, 4, 2, 64, 16
    dtype = torch.float32
    parents = torch.tensor([[-1, 0, 0, 1, -2, 4], [-1, -1, 1, 2, 3, 9]], dtype=torch.int32).cuda()
    Q, K, V = rand(B, Hq, T, d), rand(B, Hkv, T, d, seed=1), rand(B, Hkv, T, d, seed=2)
    qw, kw = weights(Hq, d, False, dtype), weights(Hkv, d, False, dtype, 4)
    f = freqs(d)
    got, want = append_case(B, T, Hq, Hkv, d, dtype, rows, [3, 20]), append_case(B, T, Hq, Hkv, d, dtype, rows, [3, 20])
    q = api.cca_norm_rope_append(Q, K, V, got[0], got[1], got[2], got[3], qw, kw, f, parents=parents)
    nq, nk = api.cca_norm_rope(Q, K, qw, kw)
    q2 = api.cca_rope_append(nq, nk, V, want[0], want[1], want[2], want[3], f, parents=parents)
    for a, b in ((q, q2), (got[0], want[0]), (got[1], want[1])):
        assert (a - b).abs().max() <= 8 * 2.0 ** -24 * 8      # a few roundings of values below 8
    assert (q[0, :, 4:] == 0).all()
    # without queries the same keys are stored
    again = append_case(B, T, Hq, Hkv, d, dtype, rows, [3, 20])
    assert api.cca_norm_rope_append(None, K, V, again[0], again[1], again[2], again[3], None, kw, f, parents=parents) is None
    assert torch.equal(again[0], got[0])


def test_append_reports_what_is_not_there():
    B, T, H, d, rows = 2, 4, 1, 64, 16
    Kp, Vp, table, ln = append_case(B, T, H, H, d, torch.float32, rows, [14, 30])
    table[0, 1] = -1                     # the last two tokens of sequence 0
    table[1, 1] = Kp.shape[0]            # two tokens of sequence 1, and the next page
    before = Kp.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = rand(B, H, T, d)
    api.cca_norm_rope_append(None, x, x, Kp, Vp, table, ln, None, None, freqs(d), dev_status=status)
    assert int(status) == api.CCA_ERR_INVALID_ARG
    changed = (Kp != before).any(-1).any(1)           # [pages, rows]
    assert int(changed.sum()) == 2 + 2                # rows 14, 15 of sequence 0; rows 32, 33 of sequence 1
    status.zero_()
    ln[0] = -5
    api.cca_norm_rope_append(None, x, x, Kp, Vp, table, ln, None, None, freqs(d), dev_status=status)
    assert int(status) == api.CCA_ERR_INVALID_ARG


def test_other_stream_and_graph():
    B, H, N, d = 1, 3, 50, 128
    Q = rand(B, H, N, d, dtype=torch.bfloat16)
    f, w = freqs(d), weights(H, d, False, torch.bfloat16)
    want, _ = api.cca_norm_rope(Q, None, w, None, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = api.cca_norm_rope(Q, None, w, None, f, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    x = torch.zeros_like(Q).requires_grad_()
    dy = rand(B, H, N, d, dtype=torch.bfloat16, seed=3)
    wg = w.clone().requires_grad_()
    with torch.cuda.stream(s):
        for _ in range(2):
            y, _ = api.norm_rope(x, None, wg, None, f)
            torch.autograd.grad(y, [x, wg], dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y, _ = api.norm_rope(x, None, wg, None, f)
        gx, gw = torch.autograd.grad(y, [x, wg], dy)
    x.data.copy_(Q)
    graph.replay()
    torch.cuda.synchronize()
    q = Q.clone().requires_grad_()
    y2, _ = api.norm_rope(q, None, wg, None, f)
    want = torch.autograd.grad(y2, [q, wg], dy)
    assert torch.equal(y, y2) and torch.equal(gx, want[0]) and torch.equal(gw, want[1])


def test_attention_takes_the_norms():
    B, Hq, Hkv, N, d, g, w = 1, 4, 2, 192, 128, 16, 32
    Q, K, V = (rand(B, h, N, d, dtype=torch.bfloat16, seed=i).requires_grad_() for i, h in enumerate((Hq, Hkv, Hkv)))
    qw, kw = weights(Hq, d, False, torch.bfloat16).requires_grad_(), weights(Hkv, d, False, torch.bfloat16, 4).requires_grad_()
    f = freqs(d)
    dO = rand(B, Hq, N, d, dtype=torch.bfloat16, seed=8)
    O = api.cca_attention(Q, K, V, g, w, inv_freq=f, q_weight=qw, k_weight=kw, offset=1.0)
    got = torch.autograd.grad(O, [Q, K, V, qw, kw], dO)
    q, k = api.norm_rope(Q, K, qw, kw, f, offset=1.0)
    O2 = api.cca_attention(q, k, V, g, w)
    want = torch.autograd.grad(O2, [Q, K, V, qw, kw], dO)
    assert torch.equal(O, O2) and all(torch.equal(a, b) for a, b in zip(got, want))
    bare = api.cca_attention(Q, K, V, g, w, norm=True)
    q, k = api.norm_rope(Q, K)
    assert torch.equal(bare, api.cca_attention(q, k, V, g, w))


def test_refusals():
    x, f = rand(1, 2, 8, 64), freqs(64)
    w = weights(2, 64, False, torch.float32)
    with pytest.raises(ValueError):
        api.cca_norm_rope(x, None, weights(3, 64, True, torch.float32), None, f)      # heads
    with pytest.raises(ValueError):
        api.cca_norm_rope(x, None, weights(2, 32, False, torch.float32), None, f)     # columns
    with pytest.raises(ValueError):
        api.cca_norm_rope(x, None, w.bfloat16(), None, f)
    with pytest.raises(ValueError):
        api.cca_norm_rope(x, None, w.double(), None, f)
    with pytest.raises(ValueError):
        api.cca_norm_rope(x, None, None, w, f)                                        # a weight of no tensor
    with pytest.raises(ValueError):
        api.cca_norm_rope(x, None, torch.stack([w, w], 1)[:, 0], None, f)             # not contiguous
    with pytest.raises(ValueError):
        api.cca_norm_rope(x, x, w, rand(64, dtype=torch.bfloat16), f)                 # two types
    with pytest.raises(ValueError):
        api.cca_norm_rope(x, None, w.cpu(), None, f)
    with pytest.raises(api.CcaError):
        api.cca_norm_rope(x, x, w, w, f, out=(x, x))
    with pytest.raises(api.CcaError):
        api.cca_norm_rope(x, None, w, None, f, eps=-1.0)
    with pytest.raises(ValueError):
        api.cca_norm_rope(x.requires_grad_(), None, w, None, f, out=(x, None))


def test_offsets_beyond_32_bits():
    # rows of one wide buffer each: the last ones lie more than 2^31 elements behind the first
    N, W, H, d = 66000, 34000, 2, 128
    assert (N - 1) * W > 2 ** 31
    x, dy = rand(1, N, H, d, dtype=torch.bfloat16).transpose(1, 2), rand(1, N, H, d, dtype=torch.bfloat16, seed=2).transpose(1, 2)
    f, w = freqs(d), weights(H, d, False, torch.float32)
    want, _ = api.cca_norm_rope(x, None, w, None, f, start=100)

    def far(src):
        y = torch.zeros(N, W, dtype=torch.bfloat16, device="cuda")[:, W - 1024:][:, :H * d].unflatten(1, (H, d)).transpose(0, 1)[None]
        y.copy_(src)
        return y
    a = far(x)
    got, _ = api.cca_norm_rope(a, None, w, None, f, start=100)
    assert torch.equal(got, want)
    leaves, back = [x.detach().requires_grad_(), w.clone().requires_grad_()], []
    for t, g in ((leaves[0], dy), (a.requires_grad_(), far(dy))):
        y, _ = api.norm_rope(t, None, leaves[1], None, f, start=100)
        back.append(torch.autograd.grad(y, [t, leaves[1]], g))
    assert all(torch.equal(p, q) for p, q in zip(*back))
    with torch.no_grad():
        api.cca_norm_rope(a, None, w, None, f, start=100, out=(a, None))      # in place
    assert torch.equal(a, want)


def test_a_backward_pass_is_not_captured_while_an_eager_graph_holds_its_leaves():
    x, w, f = rand(1, 2, 40, 64).requires_grad_(), weights(2, 64, True, torch.float32).requires_grad_(), freqs(64)
    dy = rand(1, 2, 40, 64, seed=4)

    def step():
        y, _ = api.norm_rope(x, None, w, None, f)
        return y, torch.autograd.grad(y, [x, w], dy)
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


def test_two_graphs_replayed_together():
    # each captured pass has a workspace of its own
    f, w = freqs(128), weights(1, 128, False, torch.float32).requires_grad_()
    graphs, streams, outs, wants = [], [], [], []
    for k in range(2):
        x, dy = rand(1, 8, 3000, 128, dtype=torch.bfloat16, seed=k).requires_grad_(), rand(1, 8, 3000, 128, dtype=torch.bfloat16, seed=9 + k)
        y, _ = api.norm_rope(x, None, w, None, f)
        wants.append(torch.autograd.grad(y, [x, w], dy))
        del y
        torch.cuda.synchronize()
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        leaf, lw = x.detach().requires_grad_(), w.detach().requires_grad_()
        with torch.cuda.graph(graph, stream=s):
            y, _ = api.norm_rope(leaf, None, lw, None, f)
            outs.append(torch.autograd.grad(y, [leaf, lw], dy))
        graphs.append((graph, leaf, lw, dy, y)), streams.append(s)
    for _ in range(20):
        for (graph, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
