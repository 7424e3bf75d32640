"""RMS norm of rows of any magnitude that the storage types hold, against the formula in 64 bits.

Tolerances as in test_gpu_rms_norm.py, u = 2^-24: y within 31 u and the output's
rounding; 2^-133 covers outputs below bf16's smallest normal number, 2^-149 fp32's.
A row that is summed a second time has the same sums of its elements times a power of
two, which is exact; 1 / rms of rows above 2^126 is a subnormal number, off by 2^-23
at the most (rms <= 2^127), i.e. two u more: 33 u.
"""
import numpy as np
import pytest
import torch

import ffn_gated_activation_b200 as pkg
from ffn_gated_activation_b200 import abi

import parity
from test_gpu_rms_norm import HALF, U, close, make

pytestmark = pytest.mark.gpu

SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}
# powers of two of a row's rms, with the epsilon: where epsilon is 0 the rows' own squares count
LARGE, SMALL = (40, 61, 66, 100, 124), (-30, -49, -51, -64, -100, -120)
# one warp a row, a CTA a row of two, four and eight vectors a thread
WIDTHS = [(torch.bfloat16, h) for h in (64, 1000, 4104, 8200, 32768)] + [(torch.float32, h) for h in (128, 2052, 8196)]


def rows_of(dtype, hidden, powers, seed):
    """A row of each power, an ordinary one between them."""
    x = make(torch.float32, 2 * len(powers), hidden, seed).double()
    for i, p in enumerate(powers):
        x[2 * i] = (x[2 * i] * 2.0 ** p).clamp(-2.0 ** 127, 2.0 ** 127)
    return x.to(dtype)


def weight_of(hidden, seed):
    return 1 + 0.2 * torch.randn(hidden, generator=torch.Generator().manual_seed(seed))


def ref_unit(h, eps):
    h = h.double()
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)


@pytest.mark.parametrize("powers,eps", [(LARGE, 1e-6), (LARGE, 0.0), (SMALL, 0.0), (SMALL, 1e-6), (SMALL, 2.0 ** -110), (LARGE, 1e38)])
@pytest.mark.parametrize("dtype,hidden", WIDTHS)
def test_forward(dtype, hidden, powers, eps, cuda_device):
    x, w = rows_of(dtype, hidden, powers, 1), weight_of(hidden, 2)
    y, _ = pkg.situ_glu_rms_norm_fwd(x.to(cuda_device), w.to(cuda_device), eps)
    ref = ref_unit(x, eps) * w.double()
    close(y, ref, (HALF[dtype] + 33 * U) * ref.abs() + SMALLEST[dtype], "y")
    r = torch.zeros_like(x)
    y2, h = pkg.situ_glu_rms_norm_fwd(x.to(cuda_device), w.to(cuda_device), eps, residual=r.to(cuda_device))
    assert torch.equal(h.cpu(), x) and torch.equal(y2, y)


@pytest.mark.parametrize("powers,eps", [(LARGE, 1e-6), (SMALL, 0.0)])
@pytest.mark.parametrize("dtype,hidden", [(torch.bfloat16, 992), (torch.bfloat16, 8192), (torch.float32, 2080)])
def test_mxfp8(dtype, hidden, powers, eps, cuda_device):
    x, w = rows_of(dtype, hidden, powers, 3), weight_of(hidden, 4)
    codes, scale, _ = pkg.situ_glu_rms_norm_fwd_mxfp8(x.to(cuda_device), w.to(cuda_device), eps)
    ref = (ref_unit(x, eps) * w.double()).numpy()
    parity.check_mx("rms_norm mxfp8", codes.cpu().view(torch.uint8).numpy(), scale.cpu().numpy(), ref, 33 * U * np.abs(ref),
                    abi.SITU_MX_RULE_OCP)


@pytest.mark.parametrize("dtype,power", [(torch.bfloat16, -131), (torch.float32, -131), (torch.float32, -141)])
def test_rows_of_subnormal_numbers(dtype, power, cuda_device):
    """1 / rms is above fp32's largest number; the normalised row is not."""
    for hidden in (128, 2056, 16384):
        x = rows_of(dtype, hidden, (power, power), 5)
        y, _ = pkg.situ_glu_rms_norm_fwd(x.to(cuda_device), torch.ones(hidden, device=cuda_device), 0.0)
        ref = ref_unit(x, 0.0)
        close(y, ref, (HALF[dtype] + 33 * U) * ref.abs(), "y")


# the direct kernels (a warp; eight vectors a thread), the staged one with one, two and four vectors a thread
@pytest.mark.parametrize("powers,eps", [(LARGE, 1e-6), (LARGE, 0.0), (SMALL, 0.0), (SMALL, 2.0 ** -110)])
@pytest.mark.parametrize("dtype,hidden", WIDTHS + [(torch.bfloat16, 1544), (torch.bfloat16, 512), (torch.bfloat16, 768),
                                                   (torch.float32, 516), (torch.float32, 4100), (torch.float32, 256)])
def test_backward(dtype, hidden, powers, eps, cuda_device):
    """d_x within 64 u of its terms' sizes and one rounding, d_weight within its terms' 33 u
    and its additions' (two dozen rows: a chunk each, one join of 36 additions)."""
    h, w = rows_of(dtype, hidden, powers, 6), weight_of(hidden, 7)
    gy, gh = make(dtype, h.shape[0], hidden, 8), make(dtype, h.shape[0], hidden, 9)
    unit, g = ref_unit(h, eps), gy.double() * w.double()
    q = 1 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + eps)
    along = unit * (g * unit).mean(-1, keepdim=True)
    size = q * (g.abs() + unit.abs() * (g * unit).abs().mean(-1, keepdim=True))
    terms = gy.double() * unit
    for grad_h in (None, gh):
        dx, dw = pkg.situ_glu_rms_norm_bwd(gy.to(cuda_device), h.to(cuda_device), w.to(cuda_device), eps,
                                           grad_h=grad_h.to(cuda_device) if grad_h is not None else None)
        more = grad_h.double() if grad_h is not None else torch.zeros_like(unit)
        ref = more + q * (g - along)
        close(dx, ref, HALF[dtype] * ref.abs() + 64 * U * (size + more.abs()) + SMALLEST[dtype], "d_x")
        close(dw, terms.sum(0), U * terms.sum(0).abs() + (33 + 40) * U * terms.abs().sum(0), "d_weight")
