"""The whole expert layer for a few tokens against the formula in 64 bits.

Tolerance of an output, counted from the arithmetic (u = 2^-24):
  * G and U are fp32 sums on the tensor cores, within 2^-18 of their sums of
    magnitudes (as the fused FC1's); through the activation that is E_i = 2^-18
    (|da/dG| sum |x w_g| + |da/dU| sum |x w_u|);
  * the activation's own arithmetic is within 1e-5 and its two-part rounding
    within 2^-17 of |a|;
  * the second sum is within 2^-18 of its sum of magnitudes, and the result is
    rounded to bf16 once (2^-8).
So |y - ref| <= 2^-8 |ref| + sum_i |w2_i| ((1e-5 + 2^-17 + 2^-18) |a_i| + E_i).
"""
import pytest
import torch

import ffn_gated_activation_b200 as pkg
from ffn_gated_activation_b200 import abi

pytestmark = pytest.mark.gpu


def make(tokens, hidden, inter, experts, topk, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(torch.bfloat16)
    p, ids = torch.softmax(torch.randn(tokens, experts, generator=g), -1).topk(topk, -1)
    return {"x": n(tokens, hidden), "ids": ids, "weights": p, "w1": n(experts, 2 * inter, hidden, std=3 / hidden ** 0.5),
            "w2": n(experts, hidden, inter, std=1 / inter ** 0.5)}


def reference(s, beta, lb):
    """(y, bound) in float64."""
    x, ids = s["x"].double(), s["ids"]
    tokens, hidden = x.shape
    experts, inter = s["w2"].shape[0], s["w2"].shape[2]
    w = s["weights"].double() if s["weights"] is not None else torch.ones(ids.shape, dtype=torch.float64)
    y, bound = torch.zeros(tokens, hidden, dtype=torch.float64), torch.zeros(tokens, hidden, dtype=torch.float64)
    for e in range(experts):
        share = (w * (ids == e)).sum(1)
        rows = (ids == e).any(1).nonzero().flatten()
        if not rows.numel():
            continue
        w1, w2 = s["w1"][e].double(), s["w2"][e].double()
        gu, mag = x[rows] @ w1.T, x[rows].abs() @ w1.abs().T
        G, Uu = gu[:, :inter].requires_grad_(True), gu[:, inter:].requires_grad_(True)
        up = lb * torch.tanh(Uu / lb) if lb is not None else Uu
        act = beta * torch.tanh(G / beta) * torch.sigmoid(G) * up * share[rows, None]
        dG, dU = torch.autograd.grad(act.sum(), (G, Uu))
        act = act.detach()
        err = 2.0 ** -18 * (dG.abs() * mag[:, :inter] + dU.abs() * mag[:, inter:])
        y[rows] += act @ w2.T
        bound[rows] += ((1e-5 + 2.0 ** -17 + 2.0 ** -18) * act.abs() + err) @ w2.abs().T
    return y, bound + 2.0 ** -8 * y.abs() + 1e-37


def run(s, device, beta=4.0, lb=25.0, **kw):
    d = {k: v.to(device) if v is not None else None for k, v in s.items()}
    return pkg.situ_glu_moe_fwd(d["x"], d["ids"], d["weights"], d["w1"], d["w2"], beta, lb, **kw)


def check(got, s, beta=4.0, lb=25.0):
    ref, bound = reference(s, beta, lb)
    bad = ~((got.cpu().double() - ref).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


# tokens per expert of one tile, two, four, eight; one chunk of k; more experts than CTAs' threads
@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", [
    (1, 64, 64, 1, 1), (1, 448, 192, 16, 8), (2, 128, 64, 3, 2), (7, 256, 128, 8, 2), (8, 320, 64, 2, 1),
    (9, 64, 320, 2, 2), (17, 192, 128, 3, 3), (33, 128, 64, 2, 1), (64, 128, 128, 1, 1), (64, 256, 64, 5, 4),
    (64, 64, 64, 1024, 16), (5, 1024, 512, 40, 6)])
def test_shapes(tokens, hidden, inter, experts, topk, cuda_device):
    s = make(tokens, hidden, inter, experts, topk, seed=tokens * 31 + experts)
    check(run(s, cuda_device), s)


@pytest.mark.parametrize("beta,lb", [(4.0, None), (2.0, 25.0), (1.0, 3.0), (3.5, 10.0), (3.5, None)])
def test_activation_forms(beta, lb, cuda_device):
    s = make(6, 128, 128, 4, 2, seed=5)
    check(run(s, cuda_device, beta, lb), s, beta, lb)


def test_routing_weights(cuda_device):
    s = make(6, 128, 64, 4, 2, seed=6)
    s["weights"] = None
    check(run(s, cuda_device), s)
    s["weights"] = torch.rand(6, 2, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    check(run(s, cuda_device), s)
    s["weights"] = -s["weights"].float()
    check(run(s, cuda_device), s)


def test_empty_slots_repeats_and_strangers(cuda_device):
    """Slots without an expert, ids outside the range, an expert named twice."""
    s = make(9, 128, 64, 6, 3, seed=7)
    s["ids"][0], s["ids"][4] = -1, torch.tensor([-1, 2, -1])
    s["ids"][5] = torch.tensor([3, 3, 1])
    s["ids"][6] = torch.tensor([5, 5, 5])
    s["ids"][7] = torch.tensor([6, 1 << 40, 0])
    got = run(s, cuda_device)
    check(got, s)
    assert bool((got[0] == 0).all())
    s["ids"][:] = -1
    out = torch.full((9, 128), 3.0, dtype=torch.bfloat16, device=cuda_device)
    run(s, cuda_device, out=out)
    assert bool((out == 0).all())


def test_special_values_stay_with_their_token(cuda_device):
    s = make(10, 128, 64, 3, 2, seed=8)
    clean = run(s, cuda_device)
    s["x"][4, 9] = float("nan")
    s["weights"][6, 0] = float("inf")
    got = run(s, cuda_device).cpu()
    rows = [i for i in range(10) if i not in (4, 6)]
    assert torch.equal(got[rows], clean.cpu()[rows])
    assert torch.isnan(got[4]).all() and not torch.isfinite(got[6]).any()


def test_a_token_alone_and_the_launch_size(cuda_device):
    """The same bits under any launch cap, on a second call, and in a workspace of the caller's."""
    s = make(20, 256, 128, 8, 4, seed=9)
    first = run(s, cuda_device)
    nbytes = abi.situ_glu_moe_workspace_bytes(20, 4, 256, 128)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=cuda_device)
    assert torch.equal(run(s, cuda_device, workspace=ws), first)
    assert torch.equal(run(s, cuda_device, workspace=ws), first)
    for cap in (1, 5):
        prev = abi.situ_glu_set_max_ctas(cap)
        try:
            assert torch.equal(run(s, cuda_device), first)
        finally:
            abi.situ_glu_set_max_ctas(prev)


def test_strides_and_buffers(cuda_device):
    s = make(5, 128, 64, 4, 2, seed=10)
    first = run(s, cuda_device)
    wide = {"x": torch.zeros(5, 192, dtype=torch.bfloat16), "w1": torch.zeros(4, 128, 144, dtype=torch.bfloat16),
            "w2": torch.zeros(4, 128, 72, dtype=torch.bfloat16), "ids": torch.zeros(5, 7, dtype=torch.int64),
            "weights": torch.zeros(5, 3)}
    d = {k: v.to(cuda_device) for k, v in wide.items()}
    cut = {"x": d["x"][:, 64:], "w1": d["w1"][:, :, 8:136], "w2": d["w2"][:, :, :64], "ids": d["ids"][:, 2:4],
           "weights": d["weights"][:, 1:]}
    for k, v in cut.items():
        v.copy_(s[k])
    out = torch.full((5, 256), 9.0, dtype=torch.bfloat16, device=cuda_device)
    pkg.situ_glu_moe_fwd(cut["x"], cut["ids"], cut["weights"], cut["w1"], cut["w2"], out=out[:, 64:192])
    assert torch.equal(out[:, 64:192], first)
    assert bool((out[:, :64] == 9).all()) and bool((out[:, 192:] == 9).all())
    e = pkg.situ_glu_moe_fwd(cut["x"][:0], cut["ids"][:0], cut["weights"][:0], cut["w1"], cut["w2"])
    assert e.shape == (0, 128)
    with pytest.raises(abi.SituError, match="exceeds 64"):
        pkg.situ_glu_moe_fwd(torch.zeros(65, 128, dtype=torch.bfloat16, device=cuda_device),
                             torch.zeros(65, 1, dtype=torch.int64, device=cuda_device), None, cut["w1"], cut["w2"])
    with pytest.raises(ValueError, match="workspace"):
        run(s, cuda_device, workspace=torch.empty(16, dtype=torch.uint8, device=cuda_device))
