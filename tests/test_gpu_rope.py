"""Rotary positions on the GPU against a 64-bit rotation: layouts, partial heads, strides, far
positions, gradients, and the attention that takes them."""
import numpy as np
import pytest
import torch

from paged_ref import close, rotate
from sparse_long_context_cca_gb300 import api

pytestmark = pytest.mark.gpu


def freqs(rot, base=10000.0):
    return (base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)).cuda()


def rand(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (64, 32), (128, 24), (64, 10), (128, 2), (64, 6)])
def test_matches_definition(d, rot, dtype, layout):
    B, Hq, Hkv, N = 2, 3, 2, 37
    Q, K = rand(B, Hq, N, d, dtype=dtype), rand(B, Hkv, N, d, dtype=dtype, seed=1)
    f = freqs(rot)
    q, k = api.cca_rope(Q, K, f, start=100, layout=layout, factor=1.25)
    pos = np.broadcast_to(100 + np.arange(N), (B, N))
    for name, x, y in (("Q", Q, q), ("K", K, k)):
        close(y, *rotate(x, pos, f.cpu(), layout, 1.25), f"{name} d{d} rot{rot} {layout}")


@pytest.mark.parametrize("N", [1, 2, 4099])
def test_lengths_and_one_tensor(N):
    Q = rand(1, 2, N, 128, dtype=torch.bfloat16)
    f = freqs(128)
    q, k = api.cca_rope(Q, None, f)
    assert k is None
    close(q, *rotate(Q, np.arange(N)[None], f.cpu(), "half"), f"N{N}")


def test_far_and_negative_positions():
    # positions up to the largest 32-bit one, and negative ones; shared and per sequence
    B, H, N, d = 2, 2, 64, 64
    Q = rand(B, H, N, d)
    rng = np.random.default_rng(3)
    pos = rng.integers(-2 ** 31, 2 ** 31 - 1, (B, N)).astype(np.int32)
    pos[0, :4] = [2 ** 31 - 1, -2 ** 31, 0, -1]
    f = freqs(d)
    q, _ = api.cca_rope(Q, None, f, positions=torch.from_numpy(pos).cuda())
    close(q, *rotate(Q, pos, f.cpu(), "half"), "per sequence")
    q, _ = api.cca_rope(Q, None, f, positions=torch.from_numpy(pos[0]).cuda())
    close(q, *rotate(Q, np.broadcast_to(pos[0], (B, N)), f.cpu(), "half"), "shared")
    q, _ = api.cca_rope(Q, None, f, start=2 ** 40)
    close(q, *rotate(Q, np.broadcast_to(2 ** 40 + np.arange(N, dtype=np.float64), (B, N)), f.cpu(), "half"), "start")


def test_projection_layout_and_packed_in_place():
    # queries and keys as views of one packed projection [B, N, (Hq + 2 Hkv) * d]
    B, N, Hq, Hkv, d = 2, 19, 4, 2, 64
    packed = rand(B, N, (Hq + 2 * Hkv) * d, dtype=torch.bfloat16).contiguous()
    view = lambda a, h: packed[..., a * d:(a + h) * d].view(B, N, h, d).transpose(1, 2)  # noqa: E731
    Q, K = view(0, Hq), view(Hq, Hkv)
    f = freqs(d)
    want = [rotate(x, np.broadcast_to(np.arange(N), (B, N)), f.cpu(), "half") for x in (Q, K)]
    rest = packed[..., (Hq + Hkv) * d:].clone()
    q, k = api.cca_rope(Q, K, f)
    assert q.is_contiguous() and k.is_contiguous()
    close(q, *want[0], "Q")
    close(k, *want[1], "K")
    api.cca_rope(Q, K, f, out=(Q, K))
    assert torch.equal(Q, q) and torch.equal(K, k) and torch.equal(packed[..., (Hq + Hkv) * d:], rest)


def test_one_packed_token_in_place():
    B, Hq, Hkv, d = 3, 4, 2, 64
    packed = rand(B, 1, (Hq + Hkv) * d)
    Q = packed[..., :Hq * d].view(B, 1, Hq, d).transpose(1, 2)
    K = packed[..., Hq * d:].view(B, 1, Hkv, d).transpose(1, 2)
    f = freqs(d)
    q, k = api.cca_rope(Q, K, f, start=7)
    api.cca_rope(Q, K, f, start=7, out=(Q, K))
    assert torch.equal(Q, q) and torch.equal(K, k)


def test_refuses_overlap_and_bad_rows():
    x = rand(1, 2, 8, 64)
    f = freqs(64)
    for out in ((x, x), (x[:, :, :, :], None)):
        if out[1] is not None:
            with pytest.raises(api.CcaError):
                api.cca_rope(x, x, f, out=out)            # the same tensor twice, in place
    big = rand(1, 2, 9, 64)
    with pytest.raises(api.CcaError):
        api.cca_rope(big[:, :, :8], None, f, out=(big[:, :, 1:], None))
    with pytest.raises(api.CcaError):
        api.cca_rope(x, None, f, out=(x[:, :1].expand(1, 2, 8, 64), None))   # rows that share memory
    with pytest.raises(ValueError):
        api.cca_rope(x.transpose(2, 3), None, f)
    with pytest.raises(ValueError):
        api.cca_rope(x, None, freqs(128))
    with pytest.raises(ValueError):
        api.cca_rope(x, None, f.float())
    with pytest.raises(ValueError):
        api.cca_rope(x, None, f, positions=torch.zeros(7, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradients(layout):
    B, Hq, Hkv, N, d, rot = 2, 2, 1, 9, 64, 40
    f = freqs(rot)
    pos = torch.tensor(np.random.default_rng(1).integers(0, 500, (B, N)), dtype=torch.int32).cuda()
    Q, K = rand(B, Hq, N, d).requires_grad_(), rand(B, Hkv, N, d, seed=1).requires_grad_()
    q, k = api.rope(Q, K, f, positions=pos, layout=layout, factor=1.1)
    dq, dk = rand(B, Hq, N, d, seed=2), rand(B, Hkv, N, d, seed=3)
    gq, gk = torch.autograd.grad([q, k], [Q, K], [dq, dk])
    close(gq, *rotate(dq, pos.cpu(), f.cpu(), layout, 1.1, -1.0), "dQ")
    close(gk, *rotate(dk, pos.cpu(), f.cpu(), layout, 1.1, -1.0), "dK")
    # against differences: the map is linear, so <dq, R e> over a direction e is exact but for rounding
    e = rand(B, Hq, N, d, seed=4)
    plus, _ = api.cca_rope(Q.detach() + e, K.detach(), f, positions=pos, layout=layout, factor=1.1)
    minus, _ = api.cca_rope(Q.detach() - e, K.detach(), f, positions=pos, layout=layout, factor=1.1)
    diff = ((plus.double() - minus.double()) / 2 * dq.double()).sum()
    along = (gq.double() * e.double()).sum()
    size = (dq.double().abs().sum(-1, keepdim=True) * e.double().abs().sum(-1, keepdim=True)).sum()
    assert abs(float(diff - along)) <= 2.0 ** -19 * float(size)


def test_gradient_of_a_sum_and_of_one_output():
    # .sum() hands back an expanded gradient (strides 0); an unused output hands back none
    Q, K = rand(1, 2, 5, 64).requires_grad_(), rand(1, 1, 5, 64, seed=1).requires_grad_()
    f = freqs(64)
    q, _ = api.rope(Q, K, f, start=3)
    alone, none = api.rope(Q, None, f, start=3)
    assert none is None and torch.equal(alone, q)
    assert torch.equal(torch.autograd.grad(alone.sum(), Q)[0], torch.autograd.grad(q.sum(), Q, retain_graph=True)[0])
    gq, gk = torch.autograd.grad(q.sum(), [Q, K])
    close(gq, *rotate(torch.ones(1, 2, 5, 64), 3 + np.arange(5)[None], f.cpu(), "half", 1.0, -1.0), "dQ")
    assert not gk.any()


def test_attention_with_positions():
    # cca_attention(inv_freq=...) is the rotation, then the attention, with gradients through both
    B, Hq, Hkv, N, d, g, w = 1, 2, 1, 96, 64, 8, 24
    f = freqs(d)
    Q, K, V = (rand(B, h, N, d, seed=s).requires_grad_() for s, h in ((0, Hq), (1, Hkv), (2, Hkv)))
    dO = rand(B, Hq, N, d, seed=5)
    O = api.cca_attention(Q, K, V, g, w, inv_freq=f, start=11, layout="interleaved")
    got = torch.autograd.grad(O, [Q, K, V], dO)
    q, k = api.cca_rope(Q.detach(), K.detach(), f, start=11, layout="interleaved")
    q, k, v = q.requires_grad_(), k.requires_grad_(), V.detach().requires_grad_()
    O2 = api.cca_attention(q, k, v, g, w)
    want = torch.autograd.grad(O2, [q, k, v], dO)
    assert torch.equal(O, O2) and torch.equal(got[2], want[2])
    back = api.cca_rope(want[0], want[1], f, start=11, layout="interleaved", inverse=True)
    assert torch.equal(got[0], back[0]) and torch.equal(got[1], back[1])
    with pytest.raises(ValueError):
        api.cca_attention(Q, K, V, g, w, start=11)


def test_relative_positions():
    # scores depend on distances alone: shifting every position leaves q.k as it was, within the
    # bounds of the two rotations
    d = 128
    Q, K = rand(1, 1, 16, d), rand(1, 1, 16, d, seed=1)
    f = freqs(d)
    s = []
    for start in (0, 1_000_000):
        q, k = api.cca_rope(Q, K, f, start=start)
        s.append(q.double()[0, 0] @ k.double()[0, 0].T)
    size = (Q.double().abs()[0, 0].sum(-1)[:, None] * K.double().abs()[0, 0].amax(-1)[None] * 2)
    assert ((s[0] - s[1]).abs() <= 4 * 2.0 ** -22 * size * 2).all()


def test_graph_capture_and_other_stream():
    Q, K = rand(1, 2, 33, 128, dtype=torch.bfloat16), rand(1, 1, 33, 128, dtype=torch.bfloat16, seed=1)
    pos = torch.zeros(33, dtype=torch.int32, device="cuda")
    f = freqs(128)
    out = (torch.empty_like(Q), torch.empty_like(K))
    api.cca_rope(Q, K, f, positions=pos, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cca_rope(Q, K, f, positions=pos, out=out)
    pos.copy_(torch.arange(33, dtype=torch.int32) * 9)
    Q.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    close(out[0], *rotate(Q, np.arange(33)[None] * 9, f.cpu(), "half"), "replayed")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        q, _ = api.cca_rope(Q, K, f, positions=pos, stream=stream)
        side.synchronize()
        assert torch.equal(q, out[0])


@pytest.mark.parametrize("rot,scaling", [(64, None), (64, "linear"), (64, "ntk"), (128, "bands"), (128, "yarn")])
def test_frequencies(rot, scaling):
    f, factor = api.rope_frequencies(rot, 10000.0, scaling, 8.0 if scaling else 1.0, 8192, *((1.0, 32.0) if scaling == "yarn" else ()))
    plain = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    f = f.cpu().numpy()
    assert f.dtype == np.float64 and f.shape == plain.shape
    if scaling is None:
        np.testing.assert_allclose(f, plain, rtol=1e-15)
    elif scaling == "linear":
        np.testing.assert_allclose(f, plain / 8, rtol=1e-15)
    else:
        np.testing.assert_allclose([f[0], f[-1]], [plain[0], plain[-1] / 8], rtol=1e-12)
        assert (f <= plain * (1 + 1e-12)).all() and (f >= plain / 8 * (1 - 1e-12)).all() and (np.diff(f) < 0).all()
    assert factor == pytest.approx(0.1 * np.log(8) + 1 if scaling == "yarn" else 1.0, rel=1e-15)


def test_gradient_of_the_gradient():
    """The rotation is linear: differentiating its gradient rotates forth again."""
    Q, K = rand(1, 2, 7, 64).requires_grad_(), rand(1, 1, 7, 64, seed=1).requires_grad_()
    f = freqs(64)
    q, k = api.rope(Q, K, f, start=9, factor=1.5)
    dq, dk = rand(1, 2, 7, 64, seed=2).requires_grad_(), rand(1, 1, 7, 64, seed=3).requires_grad_()
    gq, gk = torch.autograd.grad([q, k], [Q, K], [dq, dk], create_graph=True)
    e, z = rand(1, 2, 7, 64, seed=4), rand(1, 1, 7, 64, seed=5)
    hq, hk = torch.autograd.grad([gq, gk], [dq, dk], [e, z])
    pos = 9 + np.arange(7)[None]
    close(hq, *rotate(e, pos, f.cpu(), "half", 1.5), "ddQ")
    close(hk, *rotate(z, pos, f.cpu(), "half", 1.5), "ddK")


def test_forward_and_backward_in_one_graph():
    f = freqs(128)
    mk = lambda s, h: rand(1, h, 21, 128, dtype=torch.bfloat16, seed=s)  # noqa: E731
    Q, K, dq, dk = mk(0, 3).requires_grad_(), mk(1, 1).requires_grad_(), mk(2, 3), mk(3, 1)

    def step():
        q, k = api.rope(Q, K, f, layout="interleaved")
        return (q, k, *torch.autograd.grad([q, k], [Q, K], [dq, dk]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        Q.copy_(mk(4, 3))
        dk.copy_(mk(5, 1))
    graph.replay()
    torch.cuda.synchronize()
    pos = np.arange(21)[None]
    close(out[0], *rotate(Q, pos, f.cpu(), "interleaved"), "Q")
    close(out[3], *rotate(dk, pos, f.cpu(), "interleaved", 1.0, -1.0), "dK")


@pytest.mark.parametrize("attention", [False, True], ids=["rope", "attention"])
def test_backward_in_a_graph(attention):
    """A captured step gives the eager step's gradients; while an eager graph still holds the leaves on the
    default stream it is refused (autograd would end the process), and the next capture works."""
    leaves = [rand(1, h, 96, 128, dtype=torch.bfloat16, seed=h).requires_grad_() for h in (4, 2, 2)][:3 if attention else 2]
    f = freqs(128)

    def step():
        if attention:
            loss = api.cca_attention(*leaves, 16, 32, inv_freq=f).float().square().sum()
        else:
            q, k = api.rope(*leaves, f)
            loss = q[0, 0, 3].float().square().sum() + k.float().sin().sum()
        return loss, torch.autograd.grad(loss, leaves)

    eager, want = step()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="being captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            step()
    del eager
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, got = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refuses_a_flag_without_a_truth_value():
    x = rand(1, 2, 8, 64)
    with pytest.raises(ValueError, match="inverse"):
        api.cca_rope(x, None, freqs(64), inverse=torch.zeros(2))
    api.cca_rope(x, None, freqs(64), inverse=torch.ones((), dtype=torch.bool))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", [(1, 1, 1, 0, 64, 64), (1, 1, 3, 1, 128, 128), (3, 5, 7, 2, 64, 32), (2, 33, 9, 8, 128, 64),
                                              (1, 700, 5, 5, 128, 128), (1, 1500, 32, 8, 128, 128), (1, 3000, 32, 8, 64, 64)])
def test_few_and_many_heads_per_thread(B, N, Hq, Hkv, d, rot, dtype, layout):
    """Angles made by a block together or by each thread, heads that do not fill the last block."""
    Q, K = rand(B, Hq, N, d, dtype=dtype), rand(B, Hkv, N, d, dtype=dtype, seed=1) if Hkv else None
    f = freqs(rot)
    q, k = api.cca_rope(Q, K, f, start=70000, layout=layout, factor=1.25)
    pos = 70000 + np.arange(N)[None].repeat(B, 0)
    close(q, *rotate(Q, pos, f.cpu(), layout, 1.25), "Q")
    if Hkv:
        close(k, *rotate(K, pos, f.cpu(), layout, 1.25), "K")
    back = api.cca_rope(q, k, f, start=70000, layout=layout, factor=1.25, inverse=True)
    for i, (y, x) in enumerate(zip(back, (q, k))):
        if x is not None:
            close(y, *rotate(x, pos, f.cpu(), layout, 1.25, -1.0), f"back {i}")


def test_backward_in_a_graph_past_held_leaves():
    """A captured pass that does not come to a held leaf, or to one held on another stream, is not refused."""
    Q, K = (rand(1, 2, 40, 64, seed=s).requires_grad_() for s in (1, 2))
    f = freqs(64)

    def step(leaves):
        q, k = api.rope(Q, K, f)
        loss = (q * k).square().sum()
        return loss, torch.autograd.grad(loss, leaves)

    want = step([Q, K])[1]
    held = K.exp()                          # keeps K on the default stream
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step([Q])[1]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
    del held
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        held = step([Q, K])[0]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step([Q, K])[1]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and held.isfinite()


def test_one_gradient_of_two():
    Q, K = rand(2, 4, 21, 64).requires_grad_(), rand(2, 2, 21, 64, seed=1).requires_grad_()
    f = freqs(48)
    dq, dk = rand(2, 4, 21, 64, seed=2), rand(2, 2, 21, 64, seed=3)
    run = lambda leaves, q, k, **kw: torch.autograd.grad(api.rope(q, k, f, start=9), leaves, [dq, dk], **kw)  # noqa: E731
    want = run([Q, K], Q, K)
    for i, leaf in enumerate((Q, K)):
        assert torch.equal(run([leaf], Q, K)[0], want[i])
        assert torch.equal(run([leaf], *[x if x is leaf else x.detach() for x in (Q, K)])[0], want[i])
        # differentiated again: the rotation of the second gradient
        d = rand(*leaf.shape, seed=7)
        dy = [g.clone().requires_grad_() for g in (dq, dk)]
        g, = torch.autograd.grad(api.rope(Q, K, f, start=9), [leaf], dy, create_graph=True)
        again, = torch.autograd.grad(g, [dy[i]], d)
        assert torch.equal(again, api.cca_rope(d, None, f, start=9)[0])


def test_in_place_rotation_counts_as_a_write():
    """What autograd saved of a tensor that is rotated in place is out of date, and its backward pass says so."""
    f = freqs(64)
    for append in (False, True):
        x = rand(1, 2, 8, 64).requires_grad_()
        q = (x * 2.0).detach()
        y = (x * q).sum()                        # saves q
        with torch.no_grad():
            if append:
                k = rand(1, 1, 8, 64, seed=1)
                Kp, Vp = (torch.zeros(1, 1, 16, 64, device="cuda") for _ in range(2))
                zero = torch.zeros(1, dtype=torch.int32, device="cuda")
                api.cca_rope_append(q, k, k, Kp, Vp, zero[:, None].contiguous(), zero, f, out=q)
            else:
                api.cca_rope(q, None, f, out=(q, None))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()


def written_by_calls():
    """(name, tensors that the call writes, the call) for every call that writes what it is given."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    f = freqs(64)
    q, k = rand(1, 2, 4, 64), rand(1, 1, 4, 64, seed=1)
    Kp, Vp, Kc, Vc = (torch.zeros(4, 1, 16, 64, device="cuda") for _ in range(4))
    table, ctable, lens, one, zero = i32(0, 1).view(1, 2), i32(0).view(1, 1), i32(8), i32(1), i32(0)
    O, L, out, out_k = torch.empty_like(q), torch.empty(1, 2, 4, device="cuda"), torch.empty_like(q), torch.empty_like(k)
    refs, book, pairs = i32(0, 0, 0, 0), i32(-1, -1, -1, -1).view(2, 2), i32(-1, -1, -1, -1).view(2, 2)
    return [
        ("rope", (out, out_k), lambda: api.cca_rope(q, k, f, out=(out, out_k))),
        ("append", (out, Kp, Vp), lambda: api.cca_rope_append(q, k, k, Kp, Vp, table, lens, f, out=out)),
        ("tree", (O, L), lambda: api.cca_tree_fwd(q, Kp, Vp, table, Kc, Vc, ctable, lens, 8, 16, O=O, LSE=L)),
        ("pool", (Kc, Vc), lambda: api.cca_pool_pages(q, Kp, Vp, table, Kc, Vc, ctable, i32(4), i32(4), 8)),
        ("compact", (Kp, Vp), lambda: api.cca_pages_compact(Kp, Vp, table, lens, i32(1).view(1, 1), one)),
        ("copy", (Kp, Vp), lambda: api.cca_pages_copy(Kp, Vp, i32(0, 3).view(1, 2))),
        ("reserve", (refs, book, pairs), lambda: api.cca_pages_reserve(refs, book, i32(0, 0), i32(4, 0), 16, pairs=pairs)),
        ("fork", (refs, book), lambda: api.cca_pages_fork(refs, book, zero, one, i32(4, 0), 16)),
        ("free", (refs, book), lambda: api.cca_pages_free(refs, book, i32(0, 0), i32(2, 2))),
    ]


def test_every_call_counts_what_it_writes():
    for name, written, run in written_by_calls():
        before = [t._version for t in written]
        run()
        assert all(t._version > n for t, n in zip(written, before)), name
        with torch.inference_mode():
            run()
    torch.cuda.synchronize()


def test_refuses_to_write_what_requires_a_gradient():
    """As for any out= of torch: the write would be missing from the tensor's history."""
    f = freqs(64)
    for leaf in (True, False):
        q = rand(1, 2, 8, 64).requires_grad_()
        q = q if leaf else q * 1.0
        with pytest.raises(ValueError, match="requires a gradient"):
            api.cca_rope(q, None, f, out=(q, None))
        with torch.no_grad():
            api.cca_rope(q, None, f, out=(q, None))
    api.cca_rope(rand(1, 2, 8, 64).requires_grad_(), None, f)        # only read
    for name, written, run in written_by_calls():
        for t in written:
            if t.is_floating_point():
                t.requires_grad_()
                with pytest.raises(ValueError, match="requires a gradient"):
                    run()
                t.requires_grad_(False)


def test_a_refused_rotation_raises_the_librarys_error():
    """rope() raises what cca_rope() raises, with the status and its text."""
    x = rand(1, 2, 8, 96)
    f = freqs(64)
    seen = []
    for call in (lambda: api.cca_rope(x, None, f), lambda: api.rope(x, None, f), lambda: api.rope(x, x[:, :1].contiguous(), f),
                 lambda: api.rope(x.requires_grad_(), None, f)):
        with pytest.raises(api.CcaError) as e:
            call()
        seen.append((e.value.status, str(e.value)))
    assert len(set(seen)) == 1 and seen[0][0] == api.CCA_ERR_UNSUPPORTED
    with pytest.raises(api.CcaError):
        api.rope(rand(1, 2, 8, 64), None, f, factor=float("nan"))
