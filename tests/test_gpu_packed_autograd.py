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
