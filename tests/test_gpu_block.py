"""The operators around the activation used together, captured in graphs, on
streams of their own, and over buffers that a caller keeps."""
import math

import pytest
import torch

import ffn_gated_activation_b200 as pkg
from ffn_gated_activation_b200 import abi

from test_gpu_moe_few import check as check_moe
from test_gpu_moe_few import make as make_moe
from test_gpu_nvfp4_product import product_case, values

pytestmark = pytest.mark.gpu

EPS = 1e-6


def normal(*shape, seed, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def situ(g, u, w):
    return 4 * torch.tanh(g / 4) * torch.sigmoid(g) * 25 * torch.tanh(u / 25) * w


def test_a_decoding_block(cuda_device):
    """norm -> experts -> norm, the residual stream running through both; each
    operator against the formula in 64 bits on what the one before it gave."""
    s = make_moe(7, 256, 128, 6, 2, seed=21)
    stream, w = normal(7, 256, seed=1, std=2.0), 1 + 0.1 * normal(256, seed=2, dtype=torch.float32)
    d = {k: v.to(cuda_device) for k, v in s.items()}
    y, h = pkg.situ_glu_rms_norm_fwd(d["x"], w.to(cuda_device), EPS, residual=stream.to(cuda_device))
    out = pkg.situ_glu_moe_fwd(y, d["ids"], d["weights"], d["w1"], d["w2"])
    y2, h2 = pkg.situ_glu_rms_norm_fwd(out, w.to(cuda_device), EPS, residual=h)
    s["x"] = y.cpu()
    check_moe(out, s)
    ref = h2.cpu().double()
    ref = ref / torch.sqrt(ref.square().mean(-1, keepdim=True) + EPS) * w.double()
    assert bool(((y2.cpu().double() - ref).abs() <= (2.0 ** -8 + 31 * 2.0 ** -24) * ref.abs()).all())
    total = out.cpu().double() + h.cpu().double()
    assert bool(((h2.cpu().double() - total).abs() <= (2.0 ** -8 + 2.0 ** -23) * total.abs()).all())


def test_an_nvfp4_feed_forward(cuda_device):
    """norm -> NVFP4 rows -> FC1 product -> SiTU-GLU with NVFP4 rows -> FC2
    product, rows grouped by expert.  The end is compared with 64-bit arithmetic
    on the same codes from the activation's codes on, and the activation's codes
    with the values they stand for (half a step of E2M1, and of its scale)."""
    T, H, I, offsets = 300, 512, 256, [0, 90, 90, 300]
    off = torch.tensor(offsets, device=cuda_device)
    x, w = normal(T, H, seed=3), torch.ones(H, device=cuda_device)
    y, _ = pkg.situ_glu_rms_norm_fwd(x.to(cuda_device), w, EPS)
    rows = pkg.situ_glu_nvfp4_quantize(y)

    def weights(n, k, seed):
        parts = [pkg.situ_glu_nvfp4_quantize(normal(n, k, seed=seed + e, std=1 / math.sqrt(k)).to(cuda_device))
                 for e in range(3)]
        return (torch.stack([p[0] for p in parts]), torch.stack([p[1].view(torch.uint8) for p in parts]),
                torch.cat([p[2] for p in parts]))

    w1, w2 = weights(2 * I, H, 30), weights(H, I, 40)
    gate_up = pkg.situ_glu_nvfp4_gemm(rows, w1, off)
    rw = torch.rand(T, 1, generator=torch.Generator().manual_seed(5)).to(cuda_device)
    act = pkg.situ_glu_fwd_nvfp4(gate_up, rw)
    out = pkg.situ_glu_nvfp4_gemm(act, w2, off, out_dtype=torch.float32)
    gu = gate_up.cpu().double()
    exact_act = situ(gu[:, :I], gu[:, I:], rw.cpu().double())
    held = values(*act)
    unit = act[1].cpu().double().repeat_interleave(16, -1) * (act[2].cpu().double() / 2688)
    assert bool(((held - exact_act).abs() <= torch.maximum(unit * 0.251, exact_act.abs() * 0.2) + unit * 0.01).all())
    for e in range(3):
        lo, hi = offsets[e], offsets[e + 1]
        for got, a, b in ((gate_up, values(*rows), w1), (out, held, w2)):
            wv = values(b[0][e], b[1][e], b[2][e])
            ref, mag = a[lo:hi] @ wv.T, a[lo:hi].abs() @ wv.abs().T
            half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
            assert bool(((got[lo:hi].cpu().double() - ref).abs() <= (half + 2.0 ** -23) * ref.abs() + 2.0 ** -18 * mag).all())


def test_graph_replays_equal_eager_calls(cuda_device):
    """All operators in one graph, replayed on refilled inputs, twice."""
    s = make_moe(9, 128, 64, 5, 2, seed=31)
    d = {k: v.to(cuda_device) for k, v in s.items()}
    w = torch.linspace(0.5, 1.5, 128, device=cuda_device)
    res = normal(9, 128, seed=32).to(cuda_device)
    gy, gh = normal(9, 128, seed=33).to(cuda_device), normal(9, 128, seed=34).to(cuda_device)
    big = normal(2600, 1024, seed=35).to(cuda_device)  # 2600 x 1544: two-SM tiles; more blocks than one launch takes
    wq = pkg.situ_glu_nvfp4_quantize(normal(1544, 1024, seed=36).to(cuda_device))

    def step():
        y, h = pkg.situ_glu_rms_norm_fwd(d["x"], w, EPS, residual=res)
        codes, scale, _ = pkg.situ_glu_rms_norm_fwd_mxfp8(d["x"], w, EPS, residual=res)
        m = pkg.situ_glu_moe_fwd(y, d["ids"], d["weights"], d["w1"], d["w2"])
        dx, dw = pkg.situ_glu_rms_norm_bwd(gy, h, w, EPS, grad_h=gh)
        q, qs = pkg.situ_glu_nvfp4_quantize(big), pkg.situ_glu_nvfp4_quantize(y)
        p = pkg.situ_glu_nvfp4_gemm(q, wq)
        return [y, h, codes.view(torch.uint8), scale, m, dx, dw, q[0], q[1].view(torch.uint8), q[2], qs[0], p,
                pkg.situ_glu_nvfp4_dequantize(*qs)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (41, 42):
        d["x"].copy_(normal(9, 128, seed=seed))
        d["ids"].copy_(torch.randint(-1, 5, (9, 2), generator=torch.Generator().manual_seed(seed)))
        big.copy_(normal(2600, 1024, seed=seed + 10, std=seed - 40.0))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    assert abi.situ_glu_device_status(0) == 0


def test_autograd_in_a_graph(cuda_device):
    """A training step's forward and backward captured together."""
    x, r = normal(33, 256, seed=51).to(cuda_device), normal(33, 256, seed=52).to(cuda_device)
    w = torch.ones(256, device=cuda_device)
    gy = normal(33, 256, seed=53).to(cuda_device)

    def step():
        leaves = [t.detach().requires_grad_(True) for t in (x, r, w)]
        y, h = pkg.add_rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1])
        return list(torch.autograd.grad((y, h), leaves, (gy, gy)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(normal(33, 256, seed=54))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)


def test_two_streams_at_once(cuda_device):
    """Calls that overlap on the GPU, each with its own scratch, give what they
    give alone."""
    cases = [make_moe(16, 512, 256, 8, 4, seed=60 + i) for i in range(2)]
    dev = [{k: v.to(cuda_device) for k, v in s.items()} for s in cases]
    h, gy = normal(3000, 1024, seed=70).to(cuda_device), normal(3000, 1024, seed=71).to(cuda_device)
    w = torch.ones(1024, device=cuda_device)
    run = [lambda st, i=i: pkg.situ_glu_moe_fwd(dev[i]["x"], dev[i]["ids"], dev[i]["weights"], dev[i]["w1"], dev[i]["w2"],
                                                stream=st) for i in range(2)]
    run.append(lambda st: pkg.situ_glu_rms_norm_bwd(gy, h, w, EPS, stream=st)[1])
    run.append(lambda st: pkg.situ_glu_nvfp4_quantize(h, stream=st)[0])
    alone = [f(None) for f in run]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in run]
    got = [[] for _ in run]
    for _ in range(20):
        for i, f in enumerate(run):
            got[i].append(f(streams[i]))
    torch.cuda.synchronize()
    for a, many in zip(alone, got):
        assert all(torch.equal(a, b) for b in many)
    assert abi.situ_glu_device_status(0) == 0


def test_a_stream_of_another_device_is_refused(cuda_device):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=cuda_device)

    class Other:
        device = torch.device("cuda", 7)

    with pytest.raises(ValueError, match="stream is on"):
        pkg.situ_glu_rms_norm_fwd(x, torch.ones(64, device=cuda_device), EPS, stream=Other())


@pytest.mark.parametrize("rows", [1, 2])
def test_offsets_past_32_bits(rows, cuda_device):
    """Matrices whose bytes and elements pass 2^32: the last rows are the same as alone."""
    hidden = 16384
    n = 2 ** 32 // hidden // 2 + 40  # 4 GiB and a little of bf16 rows
    big = torch.empty(n, hidden, dtype=torch.bfloat16, device=cuda_device)
    tail = normal(rows, hidden, seed=80).to(cuda_device)
    big.zero_()
    big[-rows:] = tail
    w = torch.ones(hidden, device=cuda_device)
    y, _ = pkg.situ_glu_rms_norm_fwd(big, w, EPS)
    assert torch.equal(y[-rows:], pkg.situ_glu_rms_norm_fwd(tail, w, EPS)[0]) and bool((y[0] == 0).all())
    del y
    data, scale, amax = pkg.situ_glu_nvfp4_quantize(big)
    alone = pkg.situ_glu_nvfp4_quantize(tail)
    assert torch.equal(amax, alone[2]) and torch.equal(data[-rows:], alone[0])
    back = pkg.situ_glu_nvfp4_dequantize(data, scale, amax)
    assert torch.equal(back[-rows:], pkg.situ_glu_nvfp4_dequantize(*alone))


def test_products_of_two_calls_do_not_share_anything(cuda_device):
    a, w = product_case(700, 512, 320, [0, 700], seed=90, device=cuda_device)
    b, v = product_case(500, 768, 256, [0, 500], seed=95, device=cuda_device)
    first, second = pkg.situ_glu_nvfp4_gemm(a, w), pkg.situ_glu_nvfp4_gemm(b, v)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        x, y = pkg.situ_glu_nvfp4_gemm(a, w, stream=s1), pkg.situ_glu_nvfp4_gemm(b, v, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(x, first) and torch.equal(y, second)
