"""Gradients of cca_attention that someone differentiates again (an error, and not a term that is left out), and
tensors that begin between 16-byte boundaries."""
import pytest
import torch

from sparse_long_context_cca_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True], ids=["plain", "broadcast"])
def test_a_penalty_on_gradients_is_refused(wide):
    g = torch.Generator().manual_seed(4)
    leaves = [torch.randn(1, 1 if wide else h, 64, 64, generator=g).cuda().requires_grad_() for h in (4, 2, 2)]
    X = [x.expand(1, h, 64, 64) for x, h in zip(leaves, (4, 2, 2))]
    dO = torch.randn(1, 4, 64, 64, generator=g).cuda()
    for grad in (dO, dO.clone().requires_grad_()):
        got = torch.autograd.grad(api.cca_attention(*X, 8, 16), leaves, grad, create_graph=True)
        want = torch.autograd.grad(api.cca_attention(*X, 8, 16), leaves, dO)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        with pytest.raises(RuntimeError, match="differentiated again"):
            torch.autograd.grad(leaves[0].square().sum() + sum(x.square().sum() for x in got), leaves)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_tensors_off_the_copies_boundary(dtype):
    g = torch.Generator().manual_seed(5)
    X = [torch.randn(1, h, 64, 128, generator=g).to(dtype).cuda() for h in (4, 2, 2, 4)]

    def shifted(x):
        y = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)[1:].view(x.shape)
        y.copy_(x)
        return y
    outs = []
    for place in (lambda x: x.clone(), shifted):
        leaves = [place(x).requires_grad_() for x in X[:3]]
        O = api.cca_attention(*leaves, 8, 16)
        outs.append((O.detach(), *torch.autograd.grad(O, leaves, place(X[3]))))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
