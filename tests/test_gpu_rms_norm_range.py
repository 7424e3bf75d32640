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
