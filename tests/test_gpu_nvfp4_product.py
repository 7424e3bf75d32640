"""NVFP4 storage and the grouped NVFP4 product against 64-bit arithmetic.

Quantisation is exact: scales and codes equal the nearest (ties to even) of the
exact quotients, which float64 represents for every input here.  Dequantisation
is within one rounding of the type and 2 u (u = 2^-24: the block's unit and the
product).  The product: fp32 sums on the tensor cores within 2^-18 of the sums
of magnitudes (as the fused FC1's), plus the output's rounding (bf16 2^-8, fp32
u) and the tensor scale's (2 u).
"""
import pytest
import torch

import ffn_gated_activation_b200 as pkg
from ffn_gated_activation_b200 import abi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def nearest(v, grid):
    """Index of the grid's nearest entry, a tie to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.bucketize(v, mid)
    tie = v == mid[i.clamp(max=mid.numel() - 1)]
    return torch.where(tie & (i % 2 == 1) & (i < mid.numel()), i + 1, i)


def reference_codes(x, amax):
    """(magnitude codes, signs, scale codes) of finite x in float64; amax is A."""
    x, a = x.double(), float(amax)
    if a == 0 or a != a or a in (float("inf"), float("-inf")):
        a = 2688.0
    m = x.abs().unflatten(-1, (-1, 16)).amax(-1)
    sc = nearest(m * 448.0 / a, E4M3)
    unit = (E4M3[sc] * a).repeat_interleave(16, -1)
    q = torch.where(unit > 0, x.abs() * 2688.0 / torch.where(unit > 0, unit, 1.0), 0.0)
    return nearest(q, E2M1), torch.signbit(x), sc


def unpack(data):
    d = data.cpu().long()
    return torch.stack((d & 15, d >> 4), -1).flatten(-2)


def values(data, scale, amax):
    code = unpack(data)
    v = torch.where(code < 8, E2M1[code & 7], -E2M1[code & 7])
    return v * scale.cpu().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * (amax.cpu().double() / 2688.0)


def check_codes(x, data, scale, amax, what=""):
    mag, sign, sc = reference_codes(x.cpu(), amax)
    got = unpack(data)
    assert torch.equal(scale.cpu().view(torch.uint8).long(), sc), what
    assert torch.equal(got & 7, mag), what
    assert torch.equal((got >= 8) & (mag > 0), sign & (mag > 0)), what


def make(dtype, *shape, seed, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 48), (5, 1040), (37, 512), (700, 336)])
def test_round_trip(rows, cols, dtype, cuda_device):
    x = make(dtype, rows, cols, seed=rows + cols, std=0.3)
    x[0, :16] = 0  # a block of zeros
    if cols > 16:
        x[-1, 16:32] *= 1e-5  # a block whose scale rounds to zero or a subnormal
    data, scale, amax = pkg.situ_glu_nvfp4_quantize(x.to(cuda_device))
    assert float(amax) == float(x.float().abs().max())
    check_codes(x, data, scale, amax)
    for out in (torch.bfloat16, torch.float32):
        back = pkg.situ_glu_nvfp4_dequantize(data, scale, amax, dtype=out)
        ref = values(data, scale, amax)
        assert bool(((back.cpu().double() - ref).abs() <= (HALF[out] + 2 * U) * ref.abs()).all())
    _, _, alone = pkg.situ_glu_nvfp4_quantize(x.to(cuda_device), amax_only=True)
    assert torch.equal(alone, amax)
    again = pkg.situ_glu_nvfp4_quantize(x.to(cuda_device), amax=amax)
    assert torch.equal(again[0], data) and torch.equal(again[1].view(torch.uint8), scale.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_borders_between_codes(dtype, cuda_device):
    """Values on and next to every midpoint of the scales and the codes, for
    several tensor maxima."""
    for amax in (1.0, 6.0, 448.0, 2688.0, 3.40625, 1e-3, 2.0 ** -100, 1e30):
        a = float(torch.tensor(amax).to(dtype))
        rows = []
        for s in (1, 2, 9, 64, 100, 126):
            unit = float(E4M3[s]) * a / 2688.0
            mids = torch.cat(((E2M1[1:] + E2M1[:-1]) / 2, E2M1)) * unit
            near = mids.float().to(dtype)  # 15 values
            top = torch.tensor([E4M3[s] * a / 448.0]).to(dtype)
            for step in (-1, 0, 1):
                v = near.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
                rows.append(torch.cat((torch.where(near > 0, v + step, v).view(dtype), top)))
        for s in range(1, 126):  # block maxima at the midpoints between scales
            top = torch.tensor([float(E4M3[s] + E4M3[s + 1]) / 2 * a / 448.0]).to(dtype)
            rows.append(torch.cat((torch.full((15,), float(top) / 3).to(dtype), top)))
        x = torch.stack(rows)
        given = torch.tensor([a], device=cuda_device)
        data, scale, _ = pkg.situ_glu_nvfp4_quantize(x.to(cuda_device), amax=given)
        check_codes(x, data, scale, given.cpu(), f"amax {amax}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_given_maxima_that_do_not_fit(dtype, cuda_device):
    """Others than the matrix' own: none, too small, with 24 bits, tiny, not finite."""
    x = make(dtype, 8, 64, seed=3)
    x[1] *= 1e-38 if dtype == torch.float32 else 1e-30
    for a in (0.0, 0.25, 3.4000001, 7.7777, 1e-40, 1e-37, 1e37, float("inf"), float("nan")):
        given = torch.tensor([a], device=cuda_device)
        data, scale, _ = pkg.situ_glu_nvfp4_quantize(x.to(cuda_device), amax=given)
        check_codes(x, data, scale, given.cpu(), f"amax {a}")


def test_special_blocks(cuda_device):
    x = make(torch.bfloat16, 4, 64, seed=4)
    x[1, 3], x[2, 40] = float("nan"), float("-inf")
    data, scale, amax = pkg.situ_glu_nvfp4_quantize(x.to(cuda_device))
    finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    assert float(amax) == float(finite.float().abs().max())
    sc = scale.cpu().view(torch.uint8)
    assert sc[1, 0] == 0x7F and sc[2, 2] == 0x7F and int((sc == 0x7F).sum()) == 2
    assert bool((data.cpu()[1, :8] == 0).all())
    back = pkg.situ_glu_nvfp4_dequantize(data, scale, amax).cpu()
    assert torch.isnan(back[1, :16]).all() and int(torch.isnan(back).sum()) == 32
    zero = pkg.situ_glu_nvfp4_quantize(torch.zeros(2, 32, device=cuda_device))
    assert float(zero[2]) == 0 and bool((zero[0] == 0).all()) and bool((zero[1].view(torch.uint8) == 0).all())
    assert bool((pkg.situ_glu_nvfp4_dequantize(*zero) == 0).all())
    none = pkg.situ_glu_nvfp4_quantize(torch.zeros(0, 32, device=cuda_device))
    assert none[0].shape == (0, 16) and float(none[2]) == 0


def test_storage_strides(cuda_device):
    wide = make(torch.bfloat16, 9, 200, seed=5).to(cuda_device)
    x = wide[:, 8:168]  # rows of 16-byte, not 32-byte alignment
    ref = pkg.situ_glu_nvfp4_quantize(x.contiguous())
    data = torch.full((9, 96), 0xEE, dtype=torch.uint8, device=cuda_device)
    scale = torch.full((9, 13), 0xEE, dtype=torch.uint8, device=cuda_device)
    pkg.situ_glu_nvfp4_quantize(x, data=data[:, 8:88], scale=scale[:, 2:12])
    assert torch.equal(data[:, 8:88], ref[0]) and torch.equal(scale[:, 2:12], ref[1].view(torch.uint8))
    assert bool((data[:, :8] == 0xEE).all()) and bool((data[:, 88:] == 0xEE).all()) and bool((scale[:, 12:] == 0xEE).all())
    out = torch.full((9, 200), 5.0, dtype=torch.bfloat16, device=cuda_device)
    back = pkg.situ_glu_nvfp4_dequantize(data[:, 8:88], scale[:, 2:12], ref[2], out=out[:, 8:168])
    assert torch.equal(back, pkg.situ_glu_nvfp4_dequantize(*ref)) and bool((out[:, 168:] == 5).all())


# ---- product -----------------------------------------------------------------------

def stored(x, device):
    return pkg.situ_glu_nvfp4_quantize(x.to(device))


def check_product(got, a, w, offsets, dtype):
    """Rows of every expert against float64; the others must be as they were (3)."""
    av = values(*a)
    e_n = w[0].shape[0]
    wa = w[2].cpu().expand(e_n) if w[2].numel() == 1 else w[2].cpu()
    got = got.cpu().double()
    seen = torch.zeros(got.shape[0], dtype=torch.bool)
    for e in range(e_n):
        lo, hi = offsets[e], offsets[e + 1]
        if hi <= lo:
            continue
        seen[lo:hi] = True
        wv = values(w[0][e], w[1][e], wa[e])
        ref, mag = av[lo:hi] @ wv.T, av[lo:hi].abs() @ wv.abs().T
        bad = ~((got[lo:hi] - ref).abs() <= (HALF[dtype] + 2 * U) * ref.abs() + 2.0 ** -18 * mag)
        assert not bad.any(), f"expert {e}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"
    assert bool((got[~seen] == 3).all())


def padded(scale):
    """The scales with their rows 16 bytes apart or a multiple of it (k need not be one of 256)."""
    pitch = -(-scale.shape[-1] // 16) * 16
    wide = torch.full(scale.shape[:-1] + (pitch,), 0x7F, dtype=torch.uint8, device=scale.device)  # NaNs in the gaps
    wide[..., :scale.shape[-1]] = scale.view(torch.uint8)
    return wide[..., :scale.shape[-1]]


def product_case(tokens, k, n, offsets, seed, device):
    experts = len(offsets) - 1
    a = stored(make(torch.bfloat16, tokens, k, seed=seed), device)
    parts = [stored(make(torch.bfloat16, n, k, seed=seed + 1 + e, std=0.5 + e), device) for e in range(experts)]
    w = (torch.stack([p[0] for p in parts]), torch.stack([p[1].view(torch.uint8) for p in parts]),
         torch.cat([p[2] for p in parts]))
    return a, w


# one and several stages of k with whole and part last ones, part tiles of rows and columns, one
# and many tiles a cluster, narrow (few tiles) and wide tiles
@pytest.mark.parametrize("tokens,k,n", [(1, 64, 8), (1, 256, 64), (3, 128, 72), (128, 256, 64), (129, 320, 192),
                                        (200, 1024, 200), (64, 4160, 136), (1000, 576, 3000), (2500, 512, 1544),
                                        (2600, 768, 1544), (5000, 2304, 1000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(tokens, k, n, dtype, cuda_device):
    a, w = product_case(tokens, k, n, [0, tokens], seed=tokens + k, device=cuda_device)
    out = torch.full((tokens, n), 3.0, dtype=dtype, device=cuda_device)
    got = pkg.situ_glu_nvfp4_gemm(a, w, torch.tensor([0, tokens], device=cuda_device), out_dtype=dtype, out=out)
    check_product(got, a, w, [0, tokens], dtype)
    one = pkg.situ_glu_nvfp4_gemm(a, (w[0][0], w[1][0], w[2]), out_dtype=dtype)  # no offsets: one expert, every row
    assert torch.equal(one, got)
    assert abi.situ_glu_device_status(0) == 0


@pytest.mark.parametrize("offsets", [[0, 10, 10, 300], [5, 130, 131, 290], [0, 0, 0, 0], [0, 300, 300, 300]])
def test_groups(offsets, cuda_device):
    """Empty experts, rows before the first and behind the last left as they were."""
    a, w = product_case(300, 384, 264, offsets, seed=7, device=cuda_device)
    out = torch.full((300, 264), 3.0, dtype=torch.float32, device=cuda_device)
    got = pkg.situ_glu_nvfp4_gemm(a, w, torch.tensor(offsets, device=cuda_device), out_dtype=torch.float32, out=out)
    check_product(got, a, w, offsets, torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k", [64, 320, 1344])
def test_groups_of_wide_tiles(k, dtype, cuda_device):
    offsets = [3, 700, 700, 2990]
    a, w = product_case(3000, k, 1608, offsets, seed=17, device=cuda_device)
    a, w = (a[0], padded(a[1]), a[2]), (w[0], padded(w[1]), w[2])
    out = torch.full((3000, 1608), 3.0, dtype=dtype, device=cuda_device)
    got = pkg.situ_glu_nvfp4_gemm(a, w, torch.tensor(offsets, device=cuda_device), out_dtype=dtype, out=out)
    check_product(got, a, w, offsets, dtype)
    prev = abi.situ_glu_set_max_ctas(6)  # three clusters, many tiles each
    try:
        again = torch.full((3000, 1608), 3.0, dtype=dtype, device=cuda_device)
        pkg.situ_glu_nvfp4_gemm(a, w, torch.tensor(offsets, device=cuda_device), out_dtype=dtype, out=again)
        assert torch.equal(again, got)
    finally:
        abi.situ_glu_set_max_ctas(prev)
    assert abi.situ_glu_device_status(0) == 0


@pytest.mark.parametrize("tokens,n,offsets", [(37, 136, [0, 9, 9, 37]), (2900, 1608, [2, 1400, 1403, 2899])])
def test_alignment_of_the_scales(tokens, n, offsets, cuda_device):
    """Scales brought by copies of 4 and 8 bytes and by TMA: the same product, whatever lies
    between and behind the rows."""
    k = 1344  # rows of 84 bytes of scales
    a, w = product_case(tokens, k, n, offsets, seed=23, device=cuda_device)
    off = torch.tensor(offsets, device=cuda_device)

    def pitched(t, pitch, shift):
        rows = t.numel() // (k // 16)
        wide = torch.full((rows * pitch + 16,), 0x7F, dtype=torch.uint8, device=cuda_device)  # NaN scales around
        view = wide[shift:shift + rows * pitch].view(rows, pitch)[:, :k // 16]
        view.copy_(t.reshape(rows, k // 16).view(torch.uint8))
        return view.view(*t.shape[:-1], k // 16) if t.dim() == 2 else view.unflatten(0, tuple(t.shape[:-1]))

    results = []
    for pitch, shift in ((84, 0), (84, 4), (88, 0), (88, 8), (96, 4), (96, 8), (96, 0), (112, 0)):
        out = torch.full((tokens, n), 3.0, dtype=torch.float32, device=cuda_device)
        results.append(pkg.situ_glu_nvfp4_gemm((a[0], pitched(a[1], pitch, shift), a[2]),
                                               (w[0], pitched(w[1], pitch, shift), w[2]), off,
                                               out_dtype=torch.float32, out=out))
    check_product(results[0], a, w, offsets, torch.float32)
    for r in results[1:]:
        assert torch.equal(r, results[0])


def test_offsets_outside_the_rows_are_clamped(cuda_device):
    a, w = product_case(100, 128, 64, [0, 0, 0], seed=8, device=cuda_device)
    out = torch.full((100, 64), 3.0, dtype=torch.float32, device=cuda_device)
    pkg.situ_glu_nvfp4_gemm(a, w, torch.tensor([-5, 40, 1 << 40], device=cuda_device), out_dtype=torch.float32, out=out)
    check_product(out, a, w, [0, 40, 100], torch.float32)


@pytest.mark.parametrize("experts,k,n", [(70, 192, 40), (1024, 64, 8)])  # 1024: the most there may be
def test_many_experts(experts, k, n, cuda_device):
    cuts = torch.sort(torch.randint(0, 401, (experts - 1,), generator=torch.Generator().manual_seed(2)))[0]
    offsets = [0, *cuts.tolist(), 400]
    a, w = product_case(400, k, n, offsets, seed=9, device=cuda_device)
    out = torch.full((400, n), 3.0, dtype=torch.bfloat16, device=cuda_device)
    pkg.situ_glu_nvfp4_gemm(a, w, torch.tensor(offsets, device=cuda_device), out=out)
    check_product(out, a, w, offsets, torch.bfloat16)


def test_product_strides_and_launch_size(cuda_device):
    """Scales that do not load as 16-byte vectors, padded pitches, one tensor
    scale for all experts, and the same bits under any launch cap."""
    offsets = [0, 150, 300]
    off = torch.tensor(offsets, device=cuda_device)
    a, w = product_case(300, 448, 200, offsets, seed=10, device=cuda_device)
    w = (w[0], w[1], w[2][:1].contiguous())
    first = pkg.situ_glu_nvfp4_gemm(a, w, off, out_dtype=torch.float32)
    check_product(first, a, w, offsets, torch.float32)
    ad = torch.zeros(300, 272, dtype=torch.uint8, device=cuda_device)[:, 16:240]
    asc = torch.zeros(300, 36, dtype=torch.uint8, device=cuda_device)[:, 4:32]
    ws = torch.zeros(2, 200, 48, dtype=torch.uint8, device=cuda_device)[:, :, 16:44]
    ad.copy_(a[0])
    asc.copy_(a[1].view(torch.uint8))
    ws.copy_(w[1])
    out = torch.full((300, 232), 3.0, device=cuda_device)
    got = pkg.situ_glu_nvfp4_gemm((ad, asc, a[2]), (w[0], ws, w[2]), off, out_dtype=torch.float32, out=out[:, 16:216])
    assert torch.equal(got, first) and bool((out[:, :16] == 3).all()) and bool((out[:, 216:] == 3).all())
    for cap in (1, 3):
        prev = abi.situ_glu_set_max_ctas(cap)
        try:
            assert torch.equal(pkg.situ_glu_nvfp4_gemm(a, w, off, out_dtype=torch.float32), first)
        finally:
            abi.situ_glu_set_max_ctas(prev)
    assert pkg.situ_glu_nvfp4_gemm((a[0][:0], a[1][:0], a[2]), w, torch.zeros(3, dtype=torch.int64, device=cuda_device)).shape == (0, 200)


def test_nan_scales_reach_their_rows_and_columns(cuda_device):
    a, w = product_case(140, 128, 64, [0, 140], seed=11, device=cuda_device)
    clean = pkg.situ_glu_nvfp4_gemm(a, w, out_dtype=torch.float32) if w[0].shape[0] == 1 else None
    a[1].view(torch.uint8)[133, 2] = 0x7F
    w[1][0, 9, 5] = 0x7F
    got = pkg.situ_glu_nvfp4_gemm(a, w, out_dtype=torch.float32)
    assert torch.isnan(got[133]).all() and torch.isnan(got[:, 9]).all()
    rows = [i for i in range(140) if i != 133]
    cols = [i for i in range(64) if i != 9]
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
