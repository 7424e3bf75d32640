"""d_weight's sums: fp32 within a chunk of rows, 64 bits over the chunks."""
import pytest
import torch

import ffn_gated_activation_b200 as pkg

from test_gpu_rms_norm import U, make, ref_grads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden", [(592, 2048), (592, 2052), (2368, 512), (148, 4100), (148, 8196), (40, 256)])
def test_one_row_a_chunk(tokens, hidden, cuda_device):
    """Rows that cancel pair by pair: the chunks' fp32 numbers add up to zero exactly, whatever their order
    (24 bits each, within 2^20 of one another: 53 bits hold every sum on the way)."""
    eps = 1e-5
    h, gy = make(torch.float32, tokens, hidden, 71), make(torch.float32, tokens, hidden, 72)
    half = tokens // 2
    h[half:2 * half], gy[half:2 * half] = h[:half].clone(), -gy[:half]
    w = torch.ones(hidden)
    _, dw = pkg.situ_glu_rms_norm_bwd(gy.to(cuda_device), h.to(cuda_device), w.to(cuda_device), eps)
    assert tokens % 2 == 0 and bool((dw.cpu() == 0).all())


@pytest.mark.parametrize("tokens,hidden", [(2051, 2048), (5000, 512), (700, 8192)])
def test_relative_error_of_the_whole(tokens, hidden, cuda_device):
    """In the 2-norm, roundings counted with their rms of u / sqrt 3: a term's three (q, two products) and
    rsqrt's, 1.2 u; at most nine additions of a chunk to sums that grow to the chunk's, 0.6 u of the whole;
    the last rounding, 0.6 u.  sqrt(1.2^2 + 0.6^2 + 0.6^2) = 1.5 < 2."""
    h, gy, w = make(torch.float32, tokens, hidden, 73, 3.0), make(torch.float32, tokens, hidden, 74), torch.ones(hidden)
    _, dw = pkg.situ_glu_rms_norm_bwd(gy.to(cuda_device), h.to(cuda_device), w.to(cuda_device), 1e-5)
    _, _, ref, _ = ref_grads(h, w, gy, None)
    err = float((dw.cpu().double() - ref).norm() / ref.norm())
    assert err <= 2 * U
