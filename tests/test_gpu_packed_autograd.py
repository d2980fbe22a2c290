"""Autograd of packed attention: what is differentiated twice, errors that the device finds, gradients that lie
anywhere in memory, parameters that each call takes by itself."""
import numpy as np
import pytest
import torch

import packed_ref as ref
from paged_ref import HALF, close, t64
from sparse_long_context_cca_gb300 import api
from test_gpu_packed import BF, F32, IDS, KINDS, Case, device, offsets, rand

pytestmark = pytest.mark.gpu


def step(lens, Hq=4, Hkv=2, d=128, dtype=BF, g=16, w=48, tail=0, seed=0):
    T = sum(lens) + tail
    X = [rand(T, h, d, dtype=dtype, seed=seed + i).transpose(0, 1).requires_grad_() for i, h in enumerate((Hq, Hkv, Hkv))]
    return X, rand(Hq, T, d, dtype=dtype, seed=seed + 9), device(offsets(lens)), T


@pytest.mark.parametrize("wide", [False, True], ids=["plain", "broadcast"])
@pytest.mark.parametrize("needs", [(0, 1, 2), (0,), (2,)], ids=str)
def test_a_penalty_on_gradients_is_refused_and_not_left_out(needs, wide):
    # loss + penalty(gradients): the second order term cannot be had, so the sum's gradient is an error, not the loss's alone
    T, d = 90, 64
    packed = api.cca_pack(device([0, 40, T]), T, 8, 16)
    leaves = [rand(1 if wide else h, T, d, seed=i).requires_grad_(i in needs) for i, h in enumerate((4, 2, 2))]
    X = [x.expand(h, T, d) for x, h in zip(leaves, (4, 2, 2))]
    asked = [leaves[i] for i in needs]
    dO = rand(4, T, d, seed=5)
    for grad in (dO, dO.clone().requires_grad_()):
        O = api.cca_attention_packed(*X, packed)
        got = torch.autograd.grad(O, asked, grad, create_graph=True)
        want = torch.autograd.grad(api.cca_attention_packed(*X, packed), asked, dO)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(a.requires_grad for a in got)
        loss = sum(x.square().sum() for x in asked) + sum(a.square().sum() for a in got)
        with pytest.raises(RuntimeError, match="differentiated again"):
            torch.autograd.grad(loss, asked)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_lengths_that_the_device_refuses_reach_the_caller(dtype):
    X, dO, _, T = step([40], dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    packed = api.cca_pack(device([0, 30, 20]), T, 16, 8)
    O = api.cca_attention_packed(*X, packed, dev_status=status)
    assert int(status) == api.CCA_ERR_INVALID_ARG and (O == 0).all()
    status.zero_()                                  # the backward pass reports by itself, into a word that was reset
    assert all((x == 0).all() for x in torch.autograd.grad(O, X, dO))
    assert int(status) == api.CCA_ERR_INVALID_ARG
    status.zero_()
    f = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
    good = api.cca_pack(device([0, T]), T, 16, 8)
    O = api.cca_attention_packed(*X, good, inv_freq=f, norm=True, dev_status=status)
    torch.autograd.grad(O, X, dO)
    assert int(status) == 0
    for bad in (torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="dev_status"):
            api.cca_attention_packed(*X, good, dev_status=bad)


@pytest.mark.parametrize("d", [128, 64])
def test_waits_that_run_out_reach_the_caller(d):
    # the kernels' test hook copies no queries: the first wait of each ends, forward and backward
    lib = api.load_library()
    X, dO, cu, T = step([500, 300, 40], d=d, w=100)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    packed = api.cca_pack(cu, T, 16, 100)

    def run(on, call):
        torch.cuda.synchronize()
        lib.cca_test_set_wait_limit_ns(20_000_000 if on else 1_000_000_000)
        lib.cca_test_skip_q_load(on)
        try:
            out = call()
            torch.cuda.synchronize()
        finally:
            lib.cca_test_skip_q_load(0)
            lib.cca_test_set_wait_limit_ns(1_000_000_000)
        code = int(status)
        status.zero_()
        return out, code
    want, code = run(0, lambda: api.cca_attention_packed(*X, packed, dev_status=status))
    assert code == 0
    assert run(1, lambda: api.cca_attention_packed(*X, packed, dev_status=status))[1] == api.CCA_ERR_TIMEOUT
    grads, code = run(0, lambda: torch.autograd.grad(want, X, dO, retain_graph=True))
    assert code == 0
    assert run(1, lambda: torch.autograd.grad(want, X, dO, retain_graph=True))[1] == api.CCA_ERR_TIMEOUT
    again, code = run(0, lambda: torch.autograd.grad(want, X, dO))
    assert code == 0 and all(torch.equal(a, b) for a, b in zip(again, grads))


def shifted(x):
    """The same values, contiguous, one element behind a 16-byte boundary."""
    y = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)[1:].view(x.shape)
    y.copy_(x.detach())
    assert y.is_contiguous() and y.data_ptr() % 16 != 0
    return y


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_tensors_off_the_copies_boundary(dtype, d):
    # inputs and gradients that lie between 16-byte boundaries are copied, as broadcast ones are
    X, dO, cu, T = step([40, 33], d=d, dtype=dtype, g=8, w=16)
    packed = api.cca_pack(cu, T, 8, 16)
    want = torch.autograd.grad(api.cca_attention_packed(*X, packed), X, dO)
    Y = [shifted(x).requires_grad_() for x in X]
    got = torch.autograd.grad(api.cca_attention_packed(*Y, packed), Y, shifted(dO))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # such a gradient as autograd makes it: of the output behind an odd number of other values
    odd = torch.zeros(3, dtype=dtype, device="cuda", requires_grad=True)
    O = api.cca_attention_packed(*X, packed)
    row = torch.cat([odd, O.reshape(-1)])
    got = torch.autograd.grad(row, X, torch.cat([odd.detach(), dO.reshape(-1)]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,d", KINDS, ids=IDS)
def test_norms_and_rotations_off_the_copies_boundary(dtype, d):
    f = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).cuda()
    X = [rand(2, h, 21, d, dtype=dtype, seed=h).requires_grad_() for h in (4, 2)]
    dY = [rand(2, h, 21, d, dtype=dtype, seed=10 + h) for h in (4, 2)]
    w = rand(d, dtype=dtype, seed=3).requires_grad_()
    for call, more in ((lambda q, k: api.norm_rope(q, k, w, w, f), [w]), (lambda q, k: api.rope(q, k, f), [])):
        want = [x.detach() for x in call(*X)], torch.autograd.grad(call(*X), X + more, dY)
        Y = [shifted(x).requires_grad_() for x in X]
        got = [x.detach() for x in call(*Y)], torch.autograd.grad(call(*Y), Y + more, [shifted(g) for g in dY])
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


def test_a_batch_of_impossible_sizes_is_refused():
    # an empty plan for g = 0: no number of groups can be formed from it
    X, _, _, T = step([40])
    for p in (api.Packed(torch.empty(0, dtype=torch.uint8, device="cuda"), None, 1, T, 0, 8, 0),
              api.Packed(torch.empty(0, dtype=torch.uint8, device="cuda"), None, 0, T, 4, 8, 0)):
        for call in (lambda: api.cca_pool_packed(*X, p), lambda: api.cca_attn_packed(*X, None, None, p), lambda: api.cca_attention_packed(*X, p),
                     lambda: api.cca_packed_clear(p, X[0].detach())):
            with pytest.raises(ValueError, match="sequences"):
                call()
