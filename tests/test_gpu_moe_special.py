"""Infinite and NaN weights in the expert layer: what IEEE sums of the exact activations give."""
import pytest
import torch

import ffn_gated_activation_b200 as pkg

from test_gpu_moe_few import check, make, run

pytestmark = pytest.mark.gpu

INF = float("inf")


def activations(s, e, t, beta=4.0, lb=25.0):
    """Expert e's activations of token t with the routing weight, in float64."""
    inter = s["w2"].shape[2]
    G, U = (s["w1"][e].double() @ s["x"][t].double()).split(inter)
    w = float((s["weights"][t] * (s["ids"][t] == e)).sum())
    return beta * torch.tanh(G / beta) * torch.sigmoid(G) * lb * torch.tanh(U / lb) * w


@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (9, 3, 2), (40, 2, 1)])
def test_infinite_w2(tokens, experts, topk, cuda_device):
    """An infinite entry makes its row of y infinite, with the activation's sign; nothing else changes."""
    s = make(tokens, 128, 64, experts, topk, seed=40)
    clean = run(s, cuda_device).cpu()
    rows = {5: (3, INF), 17: (10, -INF), 100: (63, INF)}
    for n, (k, v) in rows.items():
        s["w2"][0, n, k] = v
    got = run(s, cuda_device).cpu()
    has = (s["ids"] == 0).any(1)
    assert bool(has.any())
    for t in range(tokens):
        if not has[t]:
            assert torch.equal(got[t], clean[t])
            continue
        a = activations(s, 0, t)
        for n, (k, v) in rows.items():
            assert float(got[t, n]) == v * float(torch.sign(a[k])), (t, n)
    others = [n for n in range(128) if n not in rows]
    assert torch.equal(got[:, others], clean[:, others])


def test_infinities_of_both_signs_and_nan(cuda_device):
    """inf - inf over the activations is NaN, as is a NaN weight."""
    s = make(4, 128, 64, 1, 1, seed=41)
    a = torch.stack([activations(s, 0, t) for t in range(4)])
    s["w2"][0, 7, 2] = s["w2"][0, 7, 9] = INF
    s["w2"][0, 8, 30] = float("nan")
    got = run(s, cuda_device).cpu()
    for t in range(4):
        same = bool(torch.sign(a[t, 2]) == torch.sign(a[t, 9]))
        assert float(got[t, 7]) == float(torch.sign(a[t, 2])) * INF if same else bool(torch.isnan(got[t, 7])), t
    assert bool(torch.isnan(got[:, 8]).all())


def test_activations_that_are_exact_in_bf16(cuda_device):
    """Remainders of zero: a gate far out and an up value with few bits."""
    s = make(3, 128, 64, 2, 1, seed=42)
    s["ids"][:] = torch.tensor([[0], [1], [0]])
    s["weights"][:] = 0.5
    s["x"][:] = 0
    s["x"][:, 0], s["x"][:, 1] = 1, 1
    s["w1"][:] = 0
    s["w1"][:, :64, 0] = 64  # T_g = 4 to fp32's precision
    s["w1"][:, 64:, 1] = 1.5
    y = pkg.situ_glu_moe_fwd(*(s[k].to(cuda_device) for k in ("x", "ids", "weights", "w1", "w2")), 4.0, None)
    ref = 4 * 1.5 * 0.5 * s["w2"][s["ids"][:, 0]].double().sum(2)
    assert bool(((y.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4).all())
    s["w2"][0, 3, 5], s["w2"][0, 4, 6] = INF, -INF
    y = pkg.situ_glu_moe_fwd(*(s[k].to(cuda_device) for k in ("x", "ids", "weights", "w1", "w2")), 4.0, None).cpu()
    assert float(y[0, 3]) == INF and float(y[2, 4]) == -INF and bool(torch.isfinite(y[1]).all())


def test_infinite_w1(cuda_device):
    """An infinite gate or up weight saturates or overflows as the formula does, for the expert's tokens alone."""
    s = make(6, 128, 64, 2, 1, seed=43)
    s["ids"][:] = torch.tensor([0, 0, 0, 1, 1, 1])[:, None]
    clean = run(s, cuda_device).cpu()
    s["w1"][0, 4, 9] = INF  # gate: T_g = 4 or 0 by the sign of x
    s["w1"][0, 64 + 8, 3] = -INF  # up: T_u = +-25
    got = run(s, cuda_device).cpu()
    assert torch.equal(got[3:], clean[3:])
    ref = torch.stack([s["w2"][0].double() @ activations(s, 0, t) for t in range(3)])
    assert bool(torch.isfinite(ref).all())
    mag = torch.stack([s["w2"][0].double().abs() @ activations(s, 0, t).abs() for t in range(3)])
    # the file's bound of the activations (1e-5 + 2^-17 + 2^-18) and of G and U (2^-18 of ten times their size)
    assert bool(((got[:3].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4 * mag).all())


def test_long_sums_are_not_cut_off(cuda_device):
    """7168 terms a sum.  An error of d, relative to y, moves a share of about 0.8 d 2^8 3 of the outputs
    over a border of bf16 (0.8: the mean of a normal error's size; 3: outputs near zero have narrower
    steps).  The activations' 16 bits and the arithmetic's 1e-6 are an rms of 3e-6, a share of 0.2 %;
    448 additions that cut off instead of rounding would be 1.2e-5, 0.7 %.  The border between: 0.4 %."""
    s = make(4, 7168, 256, 2, 1, seed=44)
    got = run(s, cuda_device).cpu()
    ref = torch.stack([s["w2"][e].double() @ activations(s, e, t) for t, e in enumerate(s["ids"][:, 0].tolist())])
    assert float((got != ref.to(torch.bfloat16)).float().mean()) <= 0.004
    assert bool(((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2e-5 * ref.abs().mean()).all())
