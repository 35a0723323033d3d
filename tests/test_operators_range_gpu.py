"""Operators at the ends of fp32's range, against 64 bits (GPU): scores and powers of two that leave the range
of fp32 (or of 64 bits) although the results do not.

Tolerances: 4e-6 of a weight and 2e-5 of the largest incoming gradient, as derived at the head of
test_operators_gpu.py; codes, scale bytes and values are equal.
"""
import math

import pytest
import torch

from sparse_mixture_experts_gate_b200 import operators as ops

pytestmark = pytest.mark.gpu

W_TOL, G_TOL = 4e-6, 2e-5
LOWEST = torch.finfo(torch.float32).min


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def small_weights(logits, idx):
    """Renormalised sigmoid weights of a selection, by the scores' logarithms, in 64 bits."""
    return torch.softmax(torch.nn.functional.logsigmoid(logits.double()).gather(1, idx.long()), 1)


@pytest.mark.parametrize("at", [-60.0, -95.0, -700.0, -745.0, -800.0, -1e4, LOWEST])
def test_renormalised_weights_of_small_sigmoid_scores(at):
    """They sum to the scale, even where every score is 0 in 64 bits."""
    g = gen(2)
    logits = at + torch.randn(30, 24, generator=g, device="cuda") * (1.0 if at > LOWEST else 0.0)
    w, idx, n = ops.route(logits, ops.RouteConfig(24, 5, "sigmoid", scale=2.5))
    assert torch.equal(idx.long(), logits.sort(dim=1, descending=True, stable=True).indices[:, :5]) and n.sum() == 150
    want = 2.5 * small_weights(logits, idx)
    assert ((w.double() - want).abs() <= W_TOL * want).all()


@pytest.mark.parametrize("gap", [50.0, 200.0, 800.0, 1e5])
def test_renormalised_weights_far_below_the_largest_score(gap):
    """A bias selects experts whose softmax scores are next to nothing, or nothing in 64 bits."""
    g = gen(3)
    logits = torch.randn(30, 32, generator=g, device="cuda")
    logits[:, :28] += gap
    bias = torch.zeros(32, device="cuda")
    bias[28:] = torch.tensor([8.0, 7.0, 6.0, 5.0])
    w, idx, _ = ops.route(logits, ops.RouteConfig(32, 3, "softmax"), bias=bias)
    assert (idx == torch.tensor([28, 29, 30], dtype=torch.int32, device="cuda")).all()
    want = torch.softmax(logits.double()[:, 28:31], 1)
    assert ((w.double() - want).abs() <= W_TOL * want).all()
