"""Quantisation of small matrices, which one cluster of CTAs does in one launch:
its CTAs exchange their maxima, those without a block of their own among them."""
import pytest
import torch

import ffn_gated_activation_b200 as pkg

from test_gpu_nvfp4_product import check_codes, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 32), (3, 16), (1, 16 * 1024), (2, 16 * 1024), (9, 16 * 1000)])
def test_maxima_of_a_cluster(rows, cols, dtype, cuda_device):
    """The maximum in the last, the first and a middle block, one to all eight CTAs having blocks."""
    for seed, at in enumerate((0, rows * cols // 2, rows * cols - 1)):
        x = make(dtype, rows, cols, seed=seed)
        x.view(-1)[at] = -9.0 - seed
        data, scale, amax = pkg.situ_glu_nvfp4_quantize(x.to(cuda_device))
        assert float(amax) == 9.0 + seed
        check_codes(x, data, scale, amax)


def test_many_clusters_in_flight(cuda_device):
    """Many calls side by side, so that a cluster's CTAs start while others end: each its own maximum."""
    streams = [torch.cuda.Stream() for _ in range(4)]
    xs = [make(torch.bfloat16, 1, 16, seed=i).to(cuda_device) for i in range(64)]
    alone = [float(x.abs().max()) for x in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(25):
        got += [(i, pkg.situ_glu_nvfp4_quantize(x, stream=streams[i % 4])) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    assert all(float(q[2]) == alone[i] for i, q in got)
    for i in range(64):
        check_codes(xs[i].cpu(), *got[-64 + i][1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("a", [1.0, 2.0 ** -20, 2.0 ** -59, 2.0 ** -80, 3.40625, 1.2345678, 2.0 ** 60])
def test_elements_far_above_a_given_maximum(a, dtype, cuda_device):
    """Codes saturate with their own sign, up to the type's largest numbers; ordinary
    elements of the same blocks keep their correctly rounded codes."""
    x = make(dtype, 12, 64, seed=6, std=a)
    x[0], x[1], x[2, ::2], x[2, 1::2] = 2e38, -2e38, 3e38, -3e38
    x[3, 5], x[4, 20], x[5, 40], x[6, 63] = 2e38, -2e38, -a * 2.0 ** 60, a * 2.0 ** 66
    x[7, :16], x[8, :16], x[9, 3] = 20 * a, -20 * a, -7 * a
    x[10, ::3] = -1e38
    given = torch.tensor([a], device=cuda_device)
    data, scale, _ = pkg.situ_glu_nvfp4_quantize(x.to(cuda_device), amax=given)
    check_codes(x, data, scale, given.cpu(), f"amax {a}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_offsets_past_32_bits(dtype, cuda_device):
    """Outputs whose rows, in all, pass 2^32 bytes and elements, and operands with rows far apart."""
    from test_gpu_nvfp4_product import product_case

    tokens, k, n = 300, 256, 264
    a, w = product_case(tokens, k, n, [0, 130, tokens], seed=60, device=cuda_device)
    off = torch.tensor([0, 130, tokens], device=cuda_device)
    want = pkg.situ_glu_nvfp4_gemm(a, w, off, out_dtype=dtype)
    pitch = 2 ** 32 // (tokens - 20) // 16 * 16  # elements: the last rows start behind the 2^32nd
    flat = torch.empty((tokens - 1) * pitch + n, dtype=dtype, device=cuda_device)
    out = flat.as_strided((tokens, n), (pitch, 1))
    far = []
    for t, cols in ((a[0], k // 2), (a[1].view(torch.uint8), k // 16)):  # the rows of codes and of scales, too
        wide = torch.empty((tokens - 1) * pitch + cols, dtype=torch.uint8, device=cuda_device).as_strided((tokens, cols), (pitch, 1))
        far.append(wide.copy_(t))
    got = pkg.situ_glu_nvfp4_gemm((far[0], far[1], a[2]), w, off, out_dtype=dtype, out=out)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,n", [(40, 72), (2500, 1544)])  # narrow and wide tiles
@pytest.mark.parametrize("aa,aw,codes", [(1e-17, 1e-17, None), (1e-20, 1e-16, None), (1e-12, 1e-30, 0x7E), (1e23, 1e23, 0x01),
                                         (3e38, 1e2, 0x20), (1e-38, 1e38, None), (3e38, 3e38, None), (0.0, 1.0, None)])
def test_products_of_extreme_tensor_scales(aa, aw, codes, tokens, n, dtype, cuda_device):
    """The tensor scales' product may leave fp32 where the result does not.  Bound as in
    test_gpu_nvfp4_product.py, and half of the smallest number of the type."""
    from test_gpu_nvfp4_product import HALF, U, product_case, values

    k = 128
    a, w = product_case(tokens, k, n, [0, tokens], seed=61, device=cuda_device)
    if codes is not None:  # every block scale the same: the smallest, the largest, an ordinary one
        a[1].view(torch.uint8).fill_(codes)
        w[1].view(torch.uint8).fill_(codes)
    a[0][3] = 0
    a, w = (a[0], a[1], torch.full_like(a[2], aa)), (w[0], w[1], torch.full_like(w[2], aw))
    got = pkg.situ_glu_nvfp4_gemm(a, w, torch.tensor([0, tokens], device=cuda_device), out_dtype=dtype).cpu().double()
    av, wv = values(*a), values(w[0][0], w[1][0], w[2])
    ref, mag = av @ wv.T, av.abs() @ wv.abs().T
    most = float(torch.finfo(dtype).max)
    smallest = 2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -150
    bound = (HALF[dtype] + 2 * U) * ref.abs() + 2.0 ** -18 * mag + smallest
    assert bool((got[3] == 0).all())
    fine = ref.abs() + bound < most
    assert bool(((got - ref).abs() <= bound)[fine].all())
    over = ref.abs() - bound > most  # beyond the type's largest number, whatever the sum's rounding
    assert bool(((got.abs() >= most) & (torch.sign(got) == torch.sign(ref)))[over].all())


def test_products_of_tensor_scales_that_are_not_finite(cuda_device):
    """Zero times an infinite or NaN factor is NaN, as the values say."""
    from test_gpu_nvfp4_product import product_case

    a, w = product_case(40, 128, 72, [0, 40], seed=62, device=cuda_device)
    a[0][3] = 0
    for bad in (float("inf"), float("nan")):
        for dtype in (torch.bfloat16, torch.float32):
            for x, y in ((bad, 1.0), (1.0, bad)):
                got = pkg.situ_glu_nvfp4_gemm((a[0], a[1], torch.full_like(a[2], x)), (w[0], w[1], torch.full_like(w[2], y)),
                                              out_dtype=dtype)
                assert bool(torch.isnan(got[3]).all()) and not bool(torch.isfinite(got).any())
