"""Gradients of add_rms_norm taken with create_graph: right, and not to be differentiated again."""
import pytest
import torch

import ffn_gated_activation_b200 as pkg

pytestmark = pytest.mark.gpu

EPS = 1e-5


def inputs(device):
    g = torch.Generator().manual_seed(1)
    return [t.to(device) for t in (torch.randn(5, 64, generator=g), torch.randn(5, 64, generator=g),
                                   1 + 0.1 * torch.randn(64, generator=g))]


@pytest.mark.parametrize("which", ["x", "residual", "weight", "all"])
def test_a_constant_gradient_does_not_hide_it(which, cuda_device):
    """A penalty on the gradient of y for constant grad_outputs: an error, not a term left out."""
    tensors = dict(zip(("x", "residual", "weight"), inputs(cuda_device)))
    wanted = [t.requires_grad_(True) for n, t in tensors.items() if which in (n, "all")]
    for out in ("y", "yh"):
        y, h = pkg.add_rms_norm(tensors["x"], tensors["weight"], EPS, residual=tensors["residual"])
        outs, ones = ([y], [torch.ones_like(y)]) if out == "y" else ([y, y + h], [torch.ones_like(y)] * 2)
        grads = torch.autograd.grad(outs, wanted, ones, create_graph=True)
        plain = torch.autograd.grad(outs, wanted, ones)
        assert all(torch.equal(a, b) for a, b in zip(grads, plain)) and all(g.requires_grad for g in grads)
        loss = y.square().sum() + sum(g.square().sum() for g in grads)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            loss.backward()


def test_without_a_residual(cuda_device):
    x, _, w = inputs(cuda_device)
    for t in (x, w):
        t.requires_grad_(True)
        y = pkg.add_rms_norm(x, w, EPS)
        (g,) = torch.autograd.grad(y.sum(), (t,), create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.sum().backward()
        y.detach()
        t.requires_grad_(False)


def test_graphs_that_are_not_differentiated_again_run(cuda_device):
    x, r, w = (t.requires_grad_(True) for t in inputs(cuda_device))
    y, h = pkg.add_rms_norm(x, w, EPS, residual=r)
    (y.square().sum() + h.sum()).backward(create_graph=True)
    assert all(t.grad is not None for t in (x, r, w))
    want = torch.autograd.grad([*pkg.add_rms_norm(x, w, EPS, residual=r)], (x, r, w),
                               [2 * y.detach(), torch.ones_like(h)])
    assert all(torch.equal(a.grad.detach(), b) for a, b in zip((x, r, w), want))
    for t in (x, r, w):
        t.grad = None


def test_under_checkpointing(cuda_device):
    """Saved tensors that are recomputed, and may be unpacked once, with and without a graph of the backward."""
    from torch.utils.checkpoint import checkpoint

    tensors = [t.requires_grad_(True) for t in inputs(cuda_device)]
    step = lambda x, r, w: sum(t.square().sum() for t in pkg.add_rms_norm(x, w, EPS, residual=r))
    plain = torch.autograd.grad(step(*tensors), tensors)
    for create in (False, True):
        got = torch.autograd.grad(checkpoint(step, *tensors, use_reentrant=False), tensors, create_graph=create)
        assert all(torch.equal(a, b) for a, b in zip(got, plain))
