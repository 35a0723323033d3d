"""Selections that fp32 keys decide wrongly if their error is taken too small, against keys in 64 bits (GPU).

The selection is the one of 64-bit keys (include/moe.h), so indices and counts have to be equal. The inputs
put the border of the selection where fp32 keys are off: groups whose two highest keys cancel, a lane that
holds most of the choices, small scores close together.
"""
import math

import pytest
import torch

from sparse_mixture_experts_gate_b200 import operators as ops

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def select(logits, k, score, groups=1, top_groups=1, group_top=2, bias=None):
    """Indices [T][k] by 64-bit keys, -1 where nothing is left; for all tokens at once."""
    T, E = logits.shape
    l = logits.double()
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        s = torch.exp(l - l.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    key = s + bias.double() if bias is not None else (s if groups > 1 else l)
    key = torch.where(l.isneginf(), -math.inf, key)
    if groups > 1:
        best = key.view(T, groups, E // groups).sort(dim=2, descending=True).values[:, :, :group_top]
        total = torch.where(best.isneginf(), 0.0, best).sum(2)
        total = torch.where(best[:, :, 0].isneginf(), -math.inf, total)
        chosen = total.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=l.device).scatter_(1, chosen, True)
        key = key.masked_fill(~keep.repeat_interleave(E // groups, 1), -math.inf)
    best = key.sort(dim=1, descending=True, stable=True)
    return torch.where(best.values[:, :k].isneginf(), -1, best.indices[:, :k])


def check(logits, k, score, groups=1, top_groups=1, group_top=2, bias=None):
    cfg = ops.RouteConfig(logits.shape[1], k, score, groups, top_groups, group_top)
    _, idx, n = ops.route(logits, cfg, bias=bias)
    want = select(logits, k, score, groups, top_groups, group_top, bias)
    off = (idx.long() != want).any(1)
    assert not off.any(), f"{int(off.sum())} of {len(off)} tokens, the first {idx[off][0].tolist()} for {want[off][0].tolist()}"
    assert torch.equal(n.long(), torch.bincount(want[want >= 0], minlength=logits.shape[1]))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size,groups,top", [(2, 32, 9), (8, 8, 4), (32, 8, 4), (20, 5, 2)])
@pytest.mark.parametrize("B", [16.0, 100.0, 1000.0, 10000.0])
def test_groups_of_keys_of_both_signs(B, size, groups, top, score):
    """One expert of each group is forced up by its bias and the others down: a group's score is a small sum
    of two large keys, which were rounded at their own size."""
    g = gen(int(B) + size)
    E = size * groups
    logits = torch.randn(200000, E, generator=g, device="cuda")
    bias = torch.full((E,), -B, device="cuda")
    bias[::size] = B
    check(logits, min(8, top * size), score, groups, top, 2, bias)


@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_forced_in_and_out(group_top):
    """Groups far above and far below the others, of which two are close."""
    g = gen(7)
    logits = torch.randn(50000, 64, generator=g, device="cuda")
    bias = torch.zeros(64, device="cuda")
    bias[:8], bias[8:16], bias[16:24] = 1e4, -1e4, 3e6
    bias[60] = math.inf
    check(logits, 8, "sigmoid", 8, 4, group_top, bias)


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_groups_of_the_lowest_numbers(score, group_top):
    """Experts that the lowest finite number takes out come before those that are not there, also as groups."""
    g = gen(8)
    logits = torch.randn(400, 64, generator=g, device="cuda")
    logits[:, :16] = -math.inf
    logits[200:, 16:24] = -math.inf
    bias = torch.zeros(64, device="cuda")
    bias[16:56] = torch.finfo(torch.float32).min
    for top in (1, 2, 3, 5):
        check(logits, min(12, 8 * top), score, 8, top, group_top, bias)


def test_border_hidden_behind_a_lanes_other_choices():
    """Experts 0, 32 and 64 lead; the fourth choice is one of 1, 96 and 128, whose fp32 keys share the bits that
    are sorted. 96 and 128 are the fourth and fifth of one lane's experts."""
    key = torch.full((256,), 0.5, dtype=torch.float64)
    for e, v in ((0, 0.92), (32, 0.91), (64, 0.90), (1, 0.750003), (96, 0.750001), (128, 0.750008)):
        key[e] = v
    logits = torch.zeros(3, 256, device="cuda")
    bias = (key - 0.5).float().cuda()
    check(logits, 4, "sigmoid", bias=bias)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("E", [200, 256, 384, 512])
@pytest.mark.parametrize("k", [4, 6, 8, 12])
def test_near_ties_of_experts_32_apart(k, E, groups, score):
    """The highest keys of a token belong to experts that are congruent modulo 32, all but the first three
    within the bits that fp32 keys are sorted without."""
    g = gen(E + k)
    T = 4096
    first = torch.randint(0, 32, (T, 1), generator=g, device="cuda")
    lanes = torch.arange(E, device="cuda") % 32 == first
    close = lanes | (torch.rand(T, E, generator=g, device="cuda") < 4.0 / E)
    u = torch.rand(T, E, generator=g, device="cuda", dtype=torch.float64)
    key = torch.where(close, 0.75 + 2.0 ** -15 * u, 0.1 + 0.4 * u)
    # Three of the lane's experts stand clear of the others.
    high = torch.where(lanes, u, -1.0).topk(3, dim=1).indices
    key.scatter_(1, high, 0.8 + 0.1 * torch.rand(T, 3, generator=g, device="cuda", dtype=torch.float64))
    logits = (torch.log(key / (1 - key)) if score == "sigmoid" else torch.log(key)).float()
    check(logits, k, score, groups, groups, 2, torch.zeros(E, device="cuda"))


@pytest.mark.parametrize("groups,top", [(2, 2), (8, 4), (16, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_sigmoid_scores_close_together(dtype, groups, top):
    """Scores without a bias between e^-16 and e^-12, apart by about the error that fp32 has there."""
    g = gen(groups)
    T, E = 20000, 128
    base = -16 + 4 * torch.rand(T, 1, generator=g, device="cuda")
    step = torch.randint(-40, 41, (T, E), generator=g, device="cuda") * 2.0 ** -20
    logits = torch.where(torch.rand(T, E, generator=g, device="cuda") < 0.3, base * (1 + step / 16), base - 3)
    check(logits.to(dtype), 8, "sigmoid", groups, top)
