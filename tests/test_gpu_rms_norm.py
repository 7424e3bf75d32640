"""Residual addition + RMS norm against the formula in 64 bits.

Tolerances, counted from the arithmetic.  u = 2^-24 is an fp32 half step and
half(t) the storage type's (bf16 2^-8, fp32 2^-24), both relative.
  * h: one fp32 addition and one rounding.
  * y = h q w from the stored h: a thread adds at most 32 squares per lane of a
    pair, the row then takes 11 more additions, so the sum of squares is within
    45 u; q = rsqrt (2 ulp = 4 u) of it is within 27 u with the mean and epsilon;
    two products: 30 u in all.
  * d_x: the same sums bound each of its terms relative to the terms' sizes, so
    64 u of |grad_h| + |q g| + |h| q^3 mean |g h| covers them.
  * d_weight: terms that are each within 32 u.  The rows of one of the C chunks
    (C = T up to 2368, 592 or 148 by the row's width) are added in order, ceil(T / C)
    additions; then the chunks in 1024 / 8 groups, ceil(C / 128) + 32 + 4 additions, or
    in 1024 / 32 groups, ceil(C / 32) + 32.  ceil(T / C) + ceil(C / 32) + 36 covers both.
"""
import numpy as np
import pytest
import torch

import ffn_gated_activation_b200 as pkg
from ffn_gated_activation_b200 import abi

import parity

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
EPS = 1e-5
# one warp a row with 1 to 4 vectors a lane; a CTA a row with 2, 4 and 8; ragged last vectors
SHAPES = [(torch.bfloat16, h) for h in (8, 256, 264, 520, 1024, 1032, 4104, 7168, 8192, 8200, 32768)] + \
         [(torch.float32, h) for h in (4, 128, 516, 2052, 8196, 16384)]


def make(dtype, tokens, hidden, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(tokens, hidden, generator=g) * std).to(dtype)


def close(got, ref, bound, what):
    got, ref = got.cpu().double(), ref.double()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}: " \
        f"{got[bad][0].item()} vs {ref[bad][0].item()}"


def dw_bound(tokens, hidden):
    """d_weight's additions and its terms' error, in u of the sum of magnitudes."""
    chunks = min(tokens, 2368 if hidden <= 1024 else 592 if hidden <= 4096 else 148)
    return (-(-tokens // chunks) + -(-chunks // 32) + 36 + 32) * U


def ref_y(h, w):
    h = h.double()
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * w.double()


def ref_grads(h, w, gy, gh):
    h, g = h.double(), gy.double() * w.double()
    q = 1 / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)
    along = (g * h).mean(-1, keepdim=True)
    gh = gh.double() if gh is not None else torch.zeros_like(h)
    dx = gh + q * g - h * q ** 3 * along
    scale = gh.abs() + (q * g).abs() + h.abs() * q ** 3 * (g * h).abs().mean(-1, keepdim=True)
    terms = gy.double() * h * q
    return dx, scale, terms.sum(0), terms.abs().sum(0)


@pytest.mark.parametrize("tokens", [1, 37])
@pytest.mark.parametrize("dtype,hidden", SHAPES)
def test_forward_and_backward(dtype, hidden, tokens, cuda_device):
    wdtype = torch.float32 if hidden % 3 else dtype
    x, r = make(dtype, tokens, hidden, 1), make(dtype, tokens, hidden, 2, 3.0)
    gy, gh = make(dtype, tokens, hidden, 3), make(dtype, tokens, hidden, 4)
    w = (1 + 0.2 * torch.randn(hidden, generator=torch.Generator().manual_seed(5))).to(wdtype)
    dev = [t.to(cuda_device) for t in (x, w, r, gy, gh)]
    half, tiny = HALF[dtype], 1e-37
    y, h = pkg.situ_glu_rms_norm_fwd(dev[0], dev[1], EPS, residual=dev[2])
    total = x.double() + r.double()
    close(h, total, (half + 2 * U) * total.abs() + tiny, "h")
    hs = h.cpu()
    ref = ref_y(hs, w)
    close(y, ref, (half + 31 * U) * ref.abs() + tiny, "y")
    y0, none = pkg.situ_glu_rms_norm_fwd(h, dev[1], EPS)
    assert none is None and torch.equal(y0, y)
    for g in (dev[4], None):
        dx, dw = pkg.situ_glu_rms_norm_bwd(dev[3], h, dev[1], EPS, grad_h=g)
        rdx, scale, rdw, mag = ref_grads(hs, w, gy, gh if g is not None else None)
        close(dx, rdx, half * rdx.abs() + 64 * U * scale + tiny, "d_x")
        close(dw, rdw, HALF[wdtype] * rdw.abs() + dw_bound(tokens, hidden) * mag + tiny, "d_weight")
    dx2, none = pkg.situ_glu_rms_norm_bwd(dev[3], h, dev[1], EPS, want_dw=False)
    assert none is None and torch.equal(dx2, dx)


@pytest.mark.parametrize("rule", ["ocp", "ceil"])
@pytest.mark.parametrize("dtype,hidden", [(torch.bfloat16, 32), (torch.bfloat16, 736), (torch.bfloat16, 992),
                                          (torch.bfloat16, 4128), (torch.bfloat16, 8192), (torch.float32, 64), (torch.float32, 2080)])
def test_mxfp8(dtype, hidden, rule, cuda_device):
    tokens = 19
    x, r = make(dtype, tokens, hidden, 11), make(dtype, tokens, hidden, 12, 3.0)
    x[3] = 0
    r[3] = 0
    w = 1 + 0.2 * torch.randn(hidden, generator=torch.Generator().manual_seed(13))
    codes, scale, h = pkg.situ_glu_rms_norm_fwd_mxfp8(x.to(cuda_device), w.to(cuda_device), EPS,
                                                      residual=r.to(cuda_device), rule=rule)
    ref = ref_y(h.cpu(), w).numpy()
    parity.check_mx("rms_norm mxfp8", codes.cpu().view(torch.uint8).numpy(), scale.cpu().numpy(), ref,
                    31 * U * np.abs(ref), abi.SITU_MX_RULE_OCP if rule == "ocp" else abi.SITU_MX_RULE_CEIL)
    y, h2 = pkg.situ_glu_rms_norm_fwd(x.to(cuda_device), w.to(cuda_device), EPS, residual=r.to(cuda_device))
    assert torch.equal(h, h2)


@pytest.mark.parametrize("tokens,hidden", [(1500, 520), (5001, 256), (1300, 1544), (700, 7176)])
def test_many_rows_and_the_launch_size(tokens, hidden, cuda_device):
    """More rows than chunks and CTAs; every result is the same under any launch cap."""
    args = [make(torch.bfloat16, tokens, hidden, s).to(cuda_device) for s in (21, 22, 23, 24)]
    w = torch.linspace(0.5, 1.5, hidden, device=cuda_device)
    h, gy, gh = args[0], args[1], args[2]

    def everything():
        y, hh = pkg.situ_glu_rms_norm_fwd(args[0], w, EPS, residual=args[3])
        return [y, hh, *pkg.situ_glu_rms_norm_bwd(gy, h, w, EPS, grad_h=gh)]

    first = everything()
    rdx, scale, rdw, mag = ref_grads(h.cpu(), w.cpu(), gy.cpu(), gh.cpu())
    close(first[2], rdx, HALF[torch.bfloat16] * rdx.abs() + 64 * U * scale, "d_x")
    close(first[3], rdw, U * rdw.abs() + dw_bound(tokens, hidden) * mag, "d_weight")
    for cap in (1, 7):
        prev = abi.situ_glu_set_max_ctas(cap)
        try:
            for a, b in zip(first, everything()):
                assert torch.equal(a, b)
        finally:
            abi.situ_glu_set_max_ctas(prev)


def test_strides_empty_and_leading_axes(cuda_device):
    wide = make(torch.bfloat16, 12, 640, 31).to(cuda_device)
    x, r = wide[:, 64:320], wide[:, 320:576]
    w = torch.ones(256, device=cuda_device)
    y, h = pkg.situ_glu_rms_norm_fwd(x, w, EPS, residual=r)
    yc, hc = pkg.situ_glu_rms_norm_fwd(x.contiguous(), w, EPS, residual=r.contiguous())
    assert torch.equal(y, yc) and torch.equal(h, hc)
    y3, h3 = pkg.situ_glu_rms_norm_fwd(x.reshape(3, 4, 256), w, EPS, residual=r.reshape(3, 4, 256))
    assert y3.shape == (3, 4, 256) and torch.equal(y3.reshape(12, 256), y)
    out = torch.full((12, 512), 7.0, dtype=torch.bfloat16, device=cuda_device)
    pkg.situ_glu_rms_norm_fwd(x, w, EPS, residual=r, out=out[:, 128:384])
    assert torch.equal(out[:, 128:384], y) and bool((out[:, :128] == 7).all()) and bool((out[:, 384:] == 7).all())
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=cuda_device)
    assert pkg.situ_glu_rms_norm_fwd(e, w, EPS, residual=e)[0].shape == (0, 256)
    assert pkg.situ_glu_rms_norm_fwd_mxfp8(e, w, EPS)[0].shape == (0, 256)
    dx, dw = pkg.situ_glu_rms_norm_bwd(e, e, w, EPS)
    assert dx.shape == (0, 256) and bool((dw == 0).all())


def test_special_rows_stay_their_own(cuda_device):
    x = make(torch.float32, 6, 512, 41)
    x[1, 5], x[2, 7], x[4] = float("nan"), float("inf"), 0
    w = torch.ones(512, device=cuda_device)
    y, _ = pkg.situ_glu_rms_norm_fwd(x.to(cuda_device), w, EPS)
    y = y.cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 7]) and bool((y[4] == 0).all())
    for row in (0, 3, 5):
        ref = ref_y(x[row], w.cpu())
        close(y[row], ref, 32 * U * ref.abs(), f"row {row}")
    codes, scale, _ = pkg.situ_glu_rms_norm_fwd_mxfp8(x.to(cuda_device), w, EPS)
    assert bool((scale[1].cpu() == 255).all()) and bool((scale[0].cpu() < 255).all())


def test_autograd_against_differences(cuda_device):
    """Gradients against central differences of the forward, in fp32 with large
    steps.  With s = 2^-6 the differences' truncation is s^2 / 6 of the third
    derivative (O(1) here: below 2^-13 of the gradient's scale) and their
    rounding 2^-23 |loss| / s, |loss| <= 2^7."""
    tokens, hidden = 3, 64
    x, r = make(torch.float32, tokens, hidden, 51).to(cuda_device), make(torch.float32, tokens, hidden, 52).to(cuda_device)
    w = (1 + 0.1 * make(torch.float32, 1, hidden, 53)[0]).to(cuda_device)
    gy, gh = make(torch.float32, tokens, hidden, 54).to(cuda_device), make(torch.float32, tokens, hidden, 55).to(cuda_device)
    leaves = [t.clone().requires_grad_(True) for t in (x, r, w)]
    y, h = pkg.add_rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1])
    torch.autograd.backward((y, h), (gy, gh))
    assert torch.equal(leaves[0].grad, leaves[1].grad) and leaves[0].grad.data_ptr() != leaves[1].grad.data_ptr()

    def loss(x, r, w):
        y, h = pkg.situ_glu_rms_norm_fwd(x, w, EPS, residual=r)
        return float((y.double() * gy.double()).sum() + (h.double() * gh.double()).sum())

    s = 2.0 ** -6
    for which, grad in ((0, leaves[0].grad), (1, leaves[1].grad), (2, leaves[2].grad)):
        for i in (0, 17, 63):
            args = [x.clone(), r.clone(), w.clone()]
            flat = args[which].view(-1)
            at = float(flat[i])
            flat[i] = at + s
            up = loss(*args)
            flat[i] = at - s
            down = loss(*args)
            assert abs((up - down) / (2 * s) - float(grad.view(-1)[i])) <= 2.0 ** -9, (which, i)


def test_autograd_forms(cuda_device):
    """No residual, only one output used, a broadcast gradient, frozen weight, leading axes."""
    x = make(torch.bfloat16, 12, 256, 61).to(cuda_device).reshape(3, 4, 256)
    w = torch.ones(256, device=cuda_device)
    a = x.clone().requires_grad_(True)
    y = pkg.add_rms_norm(a, w, EPS)
    y.sum().backward()  # an expanded (stride 0) gradient
    dx, _ = pkg.situ_glu_rms_norm_bwd(torch.ones_like(x), x, w, EPS)
    assert torch.equal(a.grad, dx)
    a, r, wl = (t.clone().requires_grad_(True) for t in (x, x, w))
    y, h = pkg.add_rms_norm(a, wl, EPS, residual=r)
    h.sum().backward()  # nothing reaches y
    assert bool((a.grad == 1).all()) and bool((r.grad == 1).all()) and bool((wl.grad == 0).all())
    a, r, wl = (t.clone().requires_grad_(True) for t in (x, x, w))
    y, h = pkg.add_rms_norm(a, wl, EPS, residual=r)
    y.backward(torch.ones_like(y))
    dx, dw = pkg.situ_glu_rms_norm_bwd(torch.ones_like(x), h.detach(), w, EPS)
    assert torch.equal(a.grad, dx) and torch.equal(wl.grad, dw)


def test_a_second_derivative_is_an_error(cuda_device):
    x = make(torch.float32, 3, 64, 91).to(cuda_device).requires_grad_(True)
    w = torch.ones(64, device=cuda_device, requires_grad=True)
    (dx,) = torch.autograd.grad(pkg.add_rms_norm(x, w, EPS).square().sum(), (x,), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()
