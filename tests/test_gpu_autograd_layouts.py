"""Gradients in the layouts that the autograd engine makes of ordinary programs:
slices of a wider gradient, whose rows do not start on 16 bytes."""
import pytest
import torch

import ffn_gated_activation_b200 as pkg

pytestmark = pytest.mark.gpu

EPS = 1e-6


def normal(*shape, seed, dtype=torch.bfloat16, device=None):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(device)


def leaves(shape, dtype, device):
    return [t.requires_grad_(True) for t in (normal(*shape, seed=1, dtype=dtype, device=device),
                                             normal(*shape, seed=2, dtype=dtype, device=device),
                                             torch.linspace(0.5, 1.5, shape[-1], device=device))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(7, 256), (1, 256), (2, 5, 64), (40, 2056)])
@pytest.mark.parametrize("before,after", [(0, 4), (4, 0), (3, 1), (8, 0)])
def test_norm_outputs_concatenated_with_a_few_columns(shape, dtype, before, after, cuda_device):
    """The gradients equal those of the aligned call with the same numbers, bit for bit."""
    x, r, w = leaves(shape, dtype, cuda_device)
    pad = [torch.zeros(*shape[:-1], n, dtype=dtype, device=cuda_device) for n in (before, after)]
    wide = shape[:-1] + (shape[-1] + before + after,)
    gy, gh = (normal(*wide, seed=s, dtype=dtype, device=cuda_device) for s in (3, 4))
    y, h = pkg.add_rms_norm(x, w, EPS, residual=r)
    got = torch.autograd.grad((torch.cat((pad[0], y, pad[1]), -1), torch.cat((pad[0], h, pad[1]), -1)), (x, r, w), (gy, gh))
    cut = [g[..., before:before + shape[-1]].clone(memory_format=torch.contiguous_format) for g in (gy, gh)]
    dx, dw = pkg.situ_glu_rms_norm_bwd(cut[0], h.detach(), w.detach(), EPS, grad_h=cut[1])
    assert torch.equal(got[0], dx) and torch.equal(got[1], dx) and torch.equal(got[2], dw)


def test_norm_gradients_at_odd_offsets(cuda_device):
    """A contiguous gradient that starts between two 16-byte boundaries, and none for h."""
    x, _, w = leaves((9, 128), torch.bfloat16, cuda_device)
    flat = normal(9 * 128 + 3, seed=5, device=cuda_device)
    y = pkg.add_rms_norm(x, w, EPS)
    for offset in (1, 2, 3):
        g = flat[offset:offset + 9 * 128].view(9, 128)
        dx, dw = torch.autograd.grad(y, (x, w), g, retain_graph=True)
        want = pkg.situ_glu_rms_norm_bwd(g.clone(), x.detach(), w.detach(), EPS)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("weights", ["row", "col", None])
def test_activation_concatenated_with_a_few_columns(weights, dtype, cuda_device):
    x = normal(9, 2 * 136, seed=6, dtype=dtype, device=cuda_device).requires_grad_(True)
    w = {"row": torch.rand(9, 1), "col": torch.rand(136), None: None}[weights]
    w = w.to(cuda_device).requires_grad_(True) if w is not None else None
    for before, after in ((0, 4), (3, 1)):
        g = normal(9, 136 + before + after, seed=7, dtype=dtype, device=cuda_device)
        pad = [torch.zeros(9, n, dtype=dtype, device=cuda_device) for n in (before, after)]
        y = pkg.weighted_situ(x, w)
        got = torch.autograd.grad(torch.cat((pad[0], y, pad[1]), -1), [t for t in (x, w) if t is not None], g)
        cut = g[:, before:before + 136].clone(memory_format=torch.contiguous_format)
        dx, dw = pkg.situ_glu_bwd(x.detach(), w.detach() if w is not None else None, cut)
        assert torch.equal(got[0], dx) and (w is None or torch.equal(got[1], dw))
