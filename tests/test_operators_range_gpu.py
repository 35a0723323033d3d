"""Operators at the ends of fp32's range, against 64 bits (GPU): scores and powers of two that leave the range
of fp32 (or of 64 bits) although the results do not.

Tolerances: 4e-6 of a weight and 2e-5 of the largest incoming gradient, as derived at the head of
test_operators_gpu.py; codes, scale bytes and values are equal.
"""
import math

import pytest
import torch

import operators_ref as ref
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [-60.0, -87.5, -95.0, -104.0, -300.0, -1e4])
def test_gradient_of_small_sigmoid_scores(at, dtype):
    """Renormalised weights have a gradient of ordinary size however small their scores are."""
    g = gen(1)
    logits = (at + torch.randn(40, 16, generator=g, device="cuda")).to(dtype)
    cfg = ops.RouteConfig(16, 4, "sigmoid", scale=2.5)
    idx = logits.float().topk(4, dim=1).indices.to(torch.int32)
    gw = torch.randn(40, 4, generator=g, device="cuda")
    d = ops.route_backward(gw, logits, idx, cfg)
    l = logits.double().requires_grad_()
    (2.5 * small_weights(l, idx) * gw).sum().backward()
    tol = G_TOL * 2.5 * gw.abs().max() + (2.0 ** -8 * l.grad.abs() if dtype == torch.bfloat16 else 0)
    assert ((d.double() - l.grad).abs() <= tol).all()


def test_gradient_of_sigmoid_scores_of_every_size():
    """Scores next to 0 and next to 1 in one selection, and selections of masked logits only."""
    logits = torch.tensor([[-120.0, -118.5, -3.0, 2.0], [50.0, 90.0, 130.0, 88.0], [-89.0, -90.0, -91.0, 0.0],
                           [-math.inf, -100.0, -101.0, -math.inf], [-math.inf] * 4], device="cuda")
    idx = torch.tensor([[0, 1], [0, 2], [0, 1], [1, 2], [0, 3]], dtype=torch.int32, device="cuda")
    gw = torch.tensor([[1.0, -2.0]], device="cuda").expand(5, 2).contiguous()
    d = ops.route_backward(gw, logits, idx, ops.RouteConfig(4, 2, "sigmoid"))
    l = logits[:4].double().requires_grad_()
    (small_weights(l, idx[:4]) * gw[:4]).sum().backward()
    assert ((d[:4].double() - l.grad).abs() <= G_TOL * 2).all() and (d[4] == 0).all()


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


def test_mxfp4_borders_below_the_normal_numbers():
    """x 2^-60 lies among fp32's subnormals: the code is still that of the exact quotient."""
    unit = 2.0 ** -67  # a scale of 2^-127 times 2^60
    row = []
    for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        bits = torch.tensor([border * unit]).view(torch.int32)
        row += [(bits + s).view(torch.float32).item() for s in (-1, 0, 1)]
    x = torch.zeros(2, 32)
    x[0, :21], x[0, 31] = torch.tensor(row), 6 * unit
    x[1] = -x[0]
    x = x.cuda()
    v = torch.empty_like(x)
    q = ops.mx_quantize(x, "mxfp4", scale_exp=60, values=v)
    codes, byte, want = ref.quantize(x, "mxfp4", 60)
    assert torch.equal(ref.scale_bytes(q.scales, 2, 32, "mxfp4"), byte)
    assert torch.equal(ref.unpack(q.codes), codes)
    assert torch.equal(v.double(), want) and torch.equal(ops.mx_dequantize(q).double(), want)


@pytest.mark.parametrize("exp", [-60, -1, 0, 60])
def test_values_of_the_smallest_numbers(exp):
    """Multiples of fp32's smallest number: their scales times 2^exp may be smaller than it, their values are not."""
    x = torch.arange(1, 65, dtype=torch.float32).view(2, 32).repeat(3, 1)
    x[2:4] = x[2:4].remainder(3)
    x[4:6] = 1.0
    x = (x.double() * 2.0 ** -149).float().cuda()
    v = torch.empty_like(x)
    q = ops.mx_quantize(x, "mxfp4", scale_exp=exp, values=v)
    codes, byte, want = ref.quantize(x, "mxfp4", exp)
    assert torch.equal(ref.unpack(q.codes), codes) and torch.equal(ref.scale_bytes(q.scales, 6, 32, "mxfp4"), byte)
    assert torch.equal(v.double(), want.float().double()) and torch.equal(ops.mx_dequantize(q), v)


def test_values_of_the_largest_scales():
    """2^127 times 2^60 is out of range: zero codes are still zeros, and small exponents bring the others back."""
    codes = torch.arange(16, dtype=torch.uint8).repeat(4)
    packed = (codes[0::2] | codes[1::2] << 4).view(1, 32).cuda()
    byte = torch.full((1, 1, 2), 254, dtype=torch.uint8, device="cuda")
    for exp in (-60, 0, 60):
        q = ops.MxTensor("mxfp4", packed, ops.mx_tile_scales(byte), 1, 64, scale_exp=exp)
        want = ref.values(codes[None].cuda(), byte[0], "mxfp4", exp).float()
        assert torch.equal(ops.mx_dequantize(q), want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_finite_numbers_that_an_exponent_takes_out_of_range(fmt, dtype):
    """x 2^60 is finite where fp32 does not hold it: scales go to their largest, codes to 6; infinities stay NaN."""
    x = torch.zeros(8, 64, dtype=dtype)
    for r, v in enumerate((2.0 ** 67, 1.5 * 2.0 ** 68, 2.0 ** 69, 1.75 * 2.0 ** 69, 2.0 ** 70, -2.0 ** 100, torch.finfo(dtype).max,
                           math.inf)):
        x[r, 3], x[r, 7], x[r, 40] = v, -v / 4, 2.0 ** -61
    x = x.cuda()
    v = torch.empty_like(x)
    q = ops.mx_quantize(x, fmt, scale_exp=-60, values=v)
    codes, byte, want = ref.quantize(x, fmt, -60)
    assert torch.equal(ref.scale_bytes(q.scales, 8, 64, fmt), byte)
    assert torch.equal(ref.unpack(q.codes), codes)
    assert torch.equal(v.double().nan_to_num(-7.0), want.nan_to_num(-7.0))
    assert v[7, 3].isnan() and not v[:7].isnan().any()
