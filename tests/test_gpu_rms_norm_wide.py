"""The widest rows of the norm's backward with more rows than chunks and CTAs: staged
rows of four vectors a thread (their ring wraps, sums run over several rows), rows of
eight vectors with their sums in shared memory.  Bounds as in test_gpu_rms_norm.py."""
import pytest
import torch

import ffn_gated_activation_b200 as pkg
from ffn_gated_activation_b200 import abi

from test_gpu_rms_norm import EPS, HALF, U, close, dw_bound, make, ref_grads, ref_y

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,tokens,hidden", [(BF, 700, 8200), (BF, 500, 16384), (F, 700, 4100), (F, 500, 8192),
                                                 (BF, 400, 32768), (F, 400, 16384), (F, 1300, 2052), (BF, 460, 16392)])
def test_many_wide_rows(dtype, tokens, hidden, cuda_device):
    h, gy, gh = (make(dtype, tokens, hidden, s) for s in (81, 82, 83))
    w = torch.linspace(0.5, 1.5, hidden)
    dev = [t.to(cuda_device) for t in (gy, h, w, gh)]
    for with_gh in (True, False):
        run = lambda: pkg.situ_glu_rms_norm_bwd(*dev[:3], EPS, grad_h=dev[3] if with_gh else None)
        dx, dw = run()
        rdx, scale, rdw, mag = ref_grads(h, w, gy, gh if with_gh else None)
        close(dx, rdx, HALF[dtype] * rdx.abs() + 64 * U * scale, "d_x")
        close(dw, rdw, U * rdw.abs() + dw_bound(tokens, hidden) * mag, "d_weight")
        for cap in (1, 7):
            prev = abi.situ_glu_set_max_ctas(cap)
            try:
                for a, b in zip((dx, dw), run()):
                    assert torch.equal(a, b)
            finally:
                abi.situ_glu_set_max_ctas(prev)
    assert abi.situ_glu_device_status(0) == 0


@pytest.mark.parametrize("dtype,hidden", [(BF, 8200), (BF, 32768), (F, 4100), (F, 16384)])
def test_many_wide_rows_forward(dtype, hidden, cuda_device):
    x, r, w = make(dtype, 600, hidden, 84), make(dtype, 600, hidden, 85), torch.linspace(0.5, 1.5, hidden)
    dev = [t.to(cuda_device) for t in (x, r, w)]
    y, h = pkg.situ_glu_rms_norm_fwd(dev[0], dev[2], EPS, residual=dev[1])
    ref = ref_y(h.cpu(), w)
    close(y, ref, (HALF[dtype] + 31 * U) * ref.abs(), "y")


# ---- offsets past 32 bits ------------------------------------------------------------

def spread(rows, dtype, pitch, device):
    """The rows, `pitch` elements apart, in a buffer of their own."""
    n, hidden = rows.shape
    flat = torch.empty((n - 1) * pitch + hidden, dtype=dtype, device=device)
    view = flat.as_strided((n, hidden), (pitch, 1))
    if rows.dtype == dtype:
        view.copy_(rows)
    return view


@pytest.mark.parametrize("hidden", [256, 2048, 16384, 32768])
def test_backward_offsets_past_32_bits(hidden, cuda_device):
    """Rows 2^31 bytes and more apart: the same as next to each other."""
    n, pitch = 4, 2 ** 30 + 8 * hidden  # elements: 2 GiB and a little a row, 6 GiB a matrix
    h, gy, gh = (make(BF, n, hidden, s).to(cuda_device) for s in (86, 87, 88))
    w = torch.linspace(0.5, 1.5, hidden, device=cuda_device)
    dx, dw = pkg.situ_glu_rms_norm_bwd(gy, h, w, EPS, grad_h=gh)
    out = spread(torch.empty(n, hidden, device="meta"), BF, pitch, cuda_device)
    far = pkg.situ_glu_rms_norm_bwd(spread(gy, BF, pitch, cuda_device), spread(h, BF, pitch, cuda_device), w, EPS,
                                    grad_h=spread(gh, BF, pitch, cuda_device), d_x=out)
    assert torch.equal(far[0], dx) and torch.equal(far[1], dw)


@pytest.mark.parametrize("hidden", [256, 4096])
def test_mxfp8_offsets_past_32_bits(hidden, cuda_device):
    n, pitch = 4, 2 ** 30 + 8 * hidden
    x, r = (make(BF, n, hidden, s).to(cuda_device) for s in (89, 90))
    w = torch.linspace(0.5, 1.5, hidden, device=cuda_device)
    codes, scale, h = pkg.situ_glu_rms_norm_fwd_mxfp8(x, w, EPS, residual=r)
    y, _ = pkg.situ_glu_rms_norm_fwd(x, w, EPS, residual=r)
    far_x, far_r = spread(x, BF, pitch, cuda_device), spread(r, BF, pitch, cuda_device)
    meta = torch.empty(n, hidden, device="meta")
    outs = [spread(meta, t, 2 * pitch, cuda_device) for t in (torch.uint8,)]
    far_scale = spread(torch.empty(n, hidden // 32, device="meta"), torch.uint8, 2 * pitch, cuda_device)
    far_h = spread(meta, BF, pitch, cuda_device)
    got = pkg.situ_glu_rms_norm_fwd_mxfp8(far_x, w, EPS, residual=far_r, data=outs[0], scale=far_scale, h_out=far_h)
    assert torch.equal(got[0], codes.view(torch.uint8)) and torch.equal(got[1], scale) and torch.equal(got[2], h)
    far_y = spread(meta, BF, pitch, cuda_device)
    got = pkg.situ_glu_rms_norm_fwd(far_x, w, EPS, residual=far_r, out=far_y, h_out=far_h)
    assert torch.equal(got[0], y) and torch.equal(got[1], h)
