"""Packed calls with scales and pooling modes other than the default: each kernel takes them by itself (scores, the
weights that the gradients form again, the pooling and its gradient, the last factor of dQ and dK)."""
import numpy as np
import pytest
import torch

import packed_ref as ref
from paged_ref import close, t64
from sparse_long_context_cca_gb300 import api
from test_gpu_packed import BF, F32, IDS, KINDS, Case, device, offsets, rand

pytestmark = pytest.mark.gpu


def check(c, scale, pool_mode, what):
    """Every call against the formulas at the GPU's own inputs of the step, directly and through autograd."""
    Kc = Vc = None
    if c.packed.cores:
        Kc, Vc = api.cca_pool_packed(c.Q, c.K, c.V, c.packed, scale=scale, pool_mode=pool_mode, dev_status=c.status)
        k, v, ek, ev = ref.pool(c.Q, c.K, c.V, c.cu, c.g, pool_mode, scale)
        close(Kc, k, ek, what + " Kc")
        close(Vc, v, ev, what + " Vc")
    O, L = api.cca_attn_packed(c.Q, c.K, c.V, Kc, Vc, c.packed, scale=scale, dev_status=c.status)
    o, l, eo, el = ref.attention(c.Q, c.K, c.V, Kc, Vc, c.cu, c.g, c.w, c.mode, scale)
    m = c.inside()
    close(O[:, m], o[:, m], eo[:, m], what + " O")
    close(L[:, m], l[:, m], el[:, m], what + " LSE")
    grads = api.cca_packed_bwd(c.Q, c.K, c.V, Kc, Vc, O, L, c.dO, c.packed, scale, pool_mode, dev_status=c.status)
    want, err = ref.backward(c.Q, c.K, c.V, Kc, Vc, O, L, c.dO, c.cu, c.g, c.w, c.mode, pool_mode, scale)
    for name, x, y, e in zip(("dQ", "dK", "dV"), grads, want, err):
        close(x[:, m], y[:, m], e[:, m], f"{what} {name}")
    leaves = [x.detach().clone().requires_grad_() for x in (c.Q, c.K, c.V)]
    P = api.cca_attention_packed(*leaves, c.packed, scale, pool_mode, dev_status=c.status)
    assert torch.equal(P[:, m], O[:, m])
    assert all(torch.equal(a[:, m], b[:, m]) for a, b in zip(torch.autograd.grad(P, leaves, c.dO), grads))
    o2 = api.cca_prefill_packed(c.Q, c.K, c.V, c.packed, scale, pool_mode)
    assert torch.equal(o2[0][:, m], O[:, m]) and torch.equal(o2[1][:, m], L[:, m])
    assert int(c.status) == 0


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
@pytest.mark.parametrize("scale", [0.05, 0.3])
@pytest.mark.parametrize("pool_mode", [0, 1])
@pytest.mark.parametrize("g,w,mode", [(8, 48, 0), (8, 48, 1), (40, 33, 1), (16, None, 0)])
def test_scales_and_modes(g, w, mode, pool_mode, scale, dtype, d):
    c = Case([210, 3, 130], d=d, dtype=dtype, g=g, w=w, mode=mode, first=3, tail=4)
    check(c, scale, pool_mode, f"scale {scale} mode {pool_mode}")


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_a_scale_where_rows_of_core_tiles_are_split(dtype, d):
    # several tiles of 128 cores, whose query rows go to several items, and tiles of keys shared by two
    check(Case([1500, 700, 2], Hq=2, Hkv=1, d=d, dtype=dtype, g=4, w=200), 0.07, 0, "split")
    if dtype == BF:
        check(Case([1300, 40], Hq=8, Hkv=1, d=d, dtype=dtype, g=16, w=None), 0.07, 0, "halves")


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_a_scale_for_rows_that_are_formed_again(dtype, d):
    # values behind a row are not finite: its own are weighed with the call's scale
    c = Case([200, 60], Hq=4, Hkv=2, d=d, dtype=dtype, g=16, w=48)
    Kc, Vc = api.cca_pool_packed(c.Q, c.K, c.V, c.packed, scale=0.3)
    V = c.V.clone()
    V[:, 150] = float("nan")
    O, L = api.cca_attn_packed(c.Q, c.K, V, Kc, Vc, c.packed, scale=0.3)
    o, l, eo, el = ref.attention(c.Q, c.K, V, Kc, Vc, c.cu, 16, 48, 0, 0.3)
    rows = np.r_[0:150, 198:260]
    close(O[:, rows], o[:, rows], eo[:, rows], "O")
    close(L, l, el, "LSE")
    assert torch.isnan(O[:, 150:198]).all()


def small(dtype=F32):
    X = [rand(h, 50, 64, dtype=dtype, seed=i).requires_grad_() for i, h in enumerate((4, 2, 2))]
    return X, api.cca_pack(device([0, 20, 50]), 50, 4, 8), rand(4, 50, 64, dtype=dtype, seed=7)


def test_hooks():
    # of tensors and of the function's node: they see the gradients and may change them
    X, packed, dO = small()
    O = api.cca_attention_packed(*X, packed)
    want = torch.autograd.grad(O, X, dO, retain_graph=True)
    seen = []
    handles = [O.register_hook(lambda g: g * 2), X[0].register_hook(lambda g: seen.append(g.clone())),
               O.grad_fn.register_hook(lambda i, o: seen.append(len(o)))]
    O.backward(dO, retain_graph=True)
    for h in handles:
        h.remove()
    for x, g in zip(X, want):
        close(x.grad, 2 * t64(g), 2.0 ** -14 * (1 + np.abs(t64(g))), "doubled")
    assert len(seen) == 2 and any(torch.is_tensor(s) and torch.equal(s, X[0].grad) for s in seen)
    again = torch.autograd.grad(O, X, dO)
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_what_the_functions_do_not_offer_is_an_error():
    # batching, forward mode and functional gradients: errors, neither results nor a broken process
    X, packed, dO = small()
    plain = [x.detach() for x in X]
    f = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    for call in (lambda q, k, v: api.cca_attention_packed(q, k, v, packed), lambda q, k, v: api.norm_rope(q[None], k[None], inv_freq=f)[0]):
        want = call(*plain)
        with pytest.raises(Exception):
            torch.func.vmap(call)(*(x[None].expand(3, *x.shape) for x in plain))
        with pytest.raises(Exception):
            torch.func.jvp(call, tuple(plain), tuple(plain))
        with pytest.raises(Exception):
            torch.func.grad(lambda q: call(q, *plain[1:]).sum())(plain[0])
        with torch.autograd.forward_ad.dual_level(), pytest.raises(Exception):
            call(torch.autograd.forward_ad.make_dual(plain[0], plain[0]), *plain[1:])
        assert torch.equal(call(*plain), want)
