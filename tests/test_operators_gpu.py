"""Routing from logits and microscaled 4-bit rows and products against plain 64-bit
implementations (GPU).

Tolerances, from the arithmetic:
  * indices, counts, codes, scale bytes and values: equal;
  * weights: fp32 scores. exp of l - m with |l - m| <= 32 is off by 2^-20 from the rounded
    difference and 2^-22 by itself, a sum of 512 terms by 25 x 2^-24, a division by 2^-24:
    below 4e-6 of the weight in all;
  * gradients: w (g - sum g w) and the like, weights and their sums off by 4e-6 of
    themselves, so 2e-5 x scale x max|g|; bf16 gradients half a step (2^-8 of the value) more;
  * products: each of the K / 64 accumulations of the tensor cores may lose 2^-22 of the
    partial sum, which is below sum |a w|; the epilogue 2^-20 of the result; bf16 outputs half
    a step (2^-8 of the value) more. The activations' slopes are below 1.13.
"""
import math

import pytest
import torch

import operators_ref as ref
from sparse_mixture_experts_gate_b200 import operators as ops
from sparse_mixture_experts_gate_b200.binding import MoEError

pytestmark = pytest.mark.gpu

W_TOL, G_TOL = 4e-6, 2e-5
HALF_BF16 = 2.0 ** -8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# ------------------------------------------------------------------ quantisation


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,exp", [(1, 32, 0), (3, 64, -3), (130, 96, 2), (33, 1408, 0), (257, 4096, -8),
                                           (5, 2080, 0)])
def test_quantize_equals_the_definition(fmt, dtype, rows, cols, exp):
    g = gen(rows * 7 + cols)
    x = (randn(g, rows, cols) * torch.exp(2 * randn(g, rows, 1)) * 2.0 ** exp).to(dtype)
    v = torch.full_like(x, 7)
    q = ops.mx_quantize(x, fmt, scale_exp=exp, values=v)
    codes, byte, want = ref.quantize(x, fmt, exp)
    assert torch.equal(ref.scale_bytes(q.scales, rows, cols, fmt), byte)
    assert torch.equal(ref.unpack(q.codes), codes)
    assert torch.equal(v.double(), want)
    assert torch.equal(ops.mx_dequantize(q).double(), want)
    assert torch.equal(ops.mx_dequantize(q, torch.bfloat16).double(), want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_borders(fmt, dtype):
    """Every border between two levels, from both sides and exactly, for many scales."""
    B = ref.BLOCK[fmt]
    rows = []
    for m in list(range(8, 16)):  # block maxima of every E4M3 mantissa
        top = 6.0 * m if fmt == "nvfp4" else 4.0 * m / 8
        for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            t = border * (m if fmt == "nvfp4" else 1)
            for step in (-1, 0, 1):
                v = torch.tensor([t], dtype=dtype)
                bits = v.view(torch.int16 if dtype == torch.bfloat16 else torch.int32) + step
                rows.append([top, bits.view(dtype).double().item()] + [-0.0] * (B - 2))
    x = torch.tensor(rows, dtype=torch.float64).to(dtype).cuda()
    if x.shape[1] < 32:
        x = torch.cat((x, x.roll(1, 0)), 1).contiguous()
    v = torch.empty_like(x)
    q = ops.mx_quantize(x, fmt, values=v)
    codes, byte, want = ref.quantize(x, fmt)
    assert torch.equal(ref.scale_bytes(q.scales, *x.shape, fmt), byte)
    assert torch.equal(ref.unpack(q.codes), codes)
    assert torch.equal(v.double(), want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_extremes(fmt, dtype):
    """Zeros, the types' largest and smallest numbers, infinities and NaN, each in a block of its own."""
    big = torch.finfo(dtype).max
    x = torch.zeros(9, 64, dtype=dtype, device="cuda")
    for r, v in enumerate((0.0, -0.0, 2.0 ** -133, torch.finfo(dtype).tiny, 1.0, big / 8, math.inf, -math.inf, math.nan)):
        x[r, 5] = v
    x[4, 40] = 3e4
    v = torch.empty_like(x)
    q = ops.mx_quantize(x, fmt, values=v)
    codes, byte, want = ref.quantize(x, fmt)
    assert torch.equal(ref.scale_bytes(q.scales, 9, 64, fmt), byte)
    assert torch.equal(ref.unpack(q.codes), codes)
    assert torch.equal(v.double().nan_to_num(-7.0), want.nan_to_num(-7.0))
    for r in (6, 7, 8):
        assert v[r, 5].isnan() and not v[r, 40].isnan()


def test_quantize_gathers_rows_and_leaves_the_others():
    g = gen(3)
    x = randn(g, 50, 160).bfloat16()
    index = torch.tensor([4, -1, 4, 49, 0, 50, 2 ** 31 - 1, -5, 17] + [-1] * 125 + [33], dtype=torch.int32, device="cuda")
    n = index.numel()
    for fmt in ("mxfp4", "nvfp4"):
        v = torch.full((n, 160), 9.0, dtype=torch.bfloat16, device="cuda")
        codes = torch.full((n, 80), 0xAB, dtype=torch.uint8, device="cuda")
        need = ops.B.moe_mx_scales_bytes(ops.B.MOE_MX[fmt], n, 160)
        out = ops.MxTensor(fmt, codes, torch.full((need,), 0xCD, dtype=torch.uint8, device="cuda"), n, 160)
        q = ops.mx_quantize(x, fmt, row_index=index, values=v, out=out)
        live = (index >= 0) & (index < 50)
        c, b, want = ref.quantize(x[index[live].long()], fmt)
        assert torch.equal(ref.unpack(q.codes)[live], c)
        assert torch.equal(ref.scale_bytes(q.scales, n, 160, fmt)[live], b)
        assert torch.equal(v[live].double(), want)
        assert (v[~live] == 9).all() and (q.codes[~live] == 0xAB).all()
        assert (ref.scale_bytes(q.scales, n, 160, fmt)[~live] == 0xCD).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,src,cols", [(1, 1, 32), (300, 70, 96), (513, 200, 2080), (5000, 9, 1408), (2100, 1000, 7168),
                                           (3100, 1000, 7168)])
def test_gathered_rows_are_the_rows(fmt, rows, src, cols):
    """Rows copied after quantisation, and quantised by index (which does so from a size on), with rows left out."""
    g = gen(rows)
    x = randn(g, src, cols).bfloat16()
    index = torch.randint(-2, src + 2, (rows,), generator=g, device="cuda", dtype=torch.int32)
    live = (index >= 0) & (index < src)
    c, b, _ = ref.quantize(x[index.clamp(0, src - 1).long()], fmt)
    need = ops.B.moe_mx_scales_bytes(ops.B.MOE_MX[fmt], rows, cols)

    def blank():
        return ops.MxTensor(fmt, torch.full((rows, cols // 2), 0xAB, dtype=torch.uint8, device="cuda"),
                            torch.full((need,), 0xCD, dtype=torch.uint8, device="cuda"), rows, cols)

    for q in (ops.mx_gather(ops.mx_quantize(x, fmt), index, out=blank()), ops.mx_quantize(x, fmt, row_index=index, out=blank())):
        assert torch.equal(ref.unpack(q.codes)[live], c[live]) and (q.codes[~live] == 0xAB).all()
        s = ref.scale_bytes(q.scales, rows, cols, fmt)
        assert torch.equal(s[live], b[live]) and (s[~live] == 0xCD).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,src,cols,exp", [(1, 1, 32, 0), (7, 3, 96, -4), (700, 130, 160, 3), (513, 200, 2080, 0), (90, 257, 4128, 0)])
def test_quantize_once_is_quantize(fmt, dtype, rows, src, cols, exp):
    """Rows quantised once and copied, through the C ABI and its workspace, and rows that are none left alone."""
    g = gen(rows + cols)
    x = randn(g, src, cols + 5).to(dtype)[:, 3:cols + 3]
    index = torch.randint(-1, src + 1, (rows,), generator=g, device="cuda", dtype=torch.int32)
    f, B = ops.B.MOE_MX[fmt], ops.B
    need, ws = B.moe_mx_scales_bytes(f, rows, cols), B.moe_mx_once_bytes(f, src, cols)
    got = []
    for once in (True, False):
        codes = torch.full((rows, cols // 2), 0xAB, dtype=torch.uint8, device="cuda")
        scales = torch.full((need,), 0xCD, dtype=torch.uint8, device="cuda")
        space = torch.full((ws + 16,), 0x5A, dtype=torch.uint8, device="cuda")
        head = (f, x.data_ptr(), B.MOE_DTYPE["bf16" if dtype is torch.bfloat16 else "fp32"], cols + 5, src, cols,
                index.data_ptr(), rows, exp, codes.data_ptr(), scales.data_ptr())
        s = torch.cuda.current_stream().cuda_stream
        if once:
            B.moe_mx_quantize_once(*head, space.data_ptr(), ws, s)
            assert (space[ws:] == 0x5A).all()
        else:
            B.moe_mx_quantize(*head, None, 0, s)
        got.append((codes, scales))
    assert torch.equal(got[0][0], got[1][0])
    a, b = (ref.scale_bytes(s, rows, cols, fmt) for _, s in got)
    live = (index >= 0) & (index < src)
    assert torch.equal(a, b) and (a[~live] == 0xCD).all() and (got[0][0][~live] == 0xAB).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_strided_rows(dtype):
    """Row strides and starts that no vector load can take."""
    g = gen(11)
    big = randn(g, 20, 203).to(dtype)
    x = big[:, 3:3 + 96]
    vb = torch.zeros(20, 101, dtype=dtype, device="cuda")
    v = vb[:, 5:]
    for fmt in ("mxfp4", "nvfp4"):
        q = ops.mx_quantize(x, fmt, values=v)
        codes, byte, want = ref.quantize(x.contiguous(), fmt)
        assert torch.equal(ref.unpack(q.codes), codes) and torch.equal(v.double(), want)
        assert torch.equal(ref.scale_bytes(q.scales, 20, 96, fmt), byte)
        assert (vb[:, :5] == 0).all()


def test_tiled_scales_are_the_layout():
    for fmt, rows, cols in (("mxfp4", 200, 416), ("nvfp4", 77, 96)):
        s = torch.randint(0, 256, (3, rows, cols // ref.BLOCK[fmt]), dtype=torch.uint8, device="cuda")
        t = ops.mx_tile_scales(s)
        for g in range(3):
            assert torch.equal(ref.scale_bytes(t, rows, cols, fmt, g), s[g])


# ------------------------------------------------------------------ routing

ROUTES = [
    # T, E, k, score, groups, top_groups, group_top, renorm, scale, bias
    (1, 1, 1, "softmax", 1, 1, 2, True, 1.0, False),
    (5, 2, 2, "sigmoid", 1, 1, 2, True, 1.0, True),
    (37, 8, 2, "softmax", 1, 1, 2, True, 1.0, False),
    (64, 7, 3, "softmax", 1, 1, 2, False, 2.5, False),
    (33, 60, 6, "softmax", 4, 2, 1, False, 16.0, False),
    (129, 64, 6, "softmax", 8, 3, 1, True, 1.0, False),
    (70, 128, 8, "softmax", 1, 1, 2, True, 1.0, True),
    (100, 160, 6, "softmax", 8, 3, 2, False, 16.0, True),
    (130, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, True),
    (65, 256, 8, "sigmoid", 1, 1, 2, True, 2.5, True),
    (40, 384, 8, "sigmoid", 1, 1, 2, True, 2.827, True),
    (40, 512, 32, "softmax", 32, 9, 2, True, 1.0, False),
    (31, 100, 10, "sigmoid", 20, 10, 2, False, 1.0, True),
    (17, 16, 16, "sigmoid", 16, 16, 2, True, 1.0, False),
    (50, 128, 8, "sigmoid", 4, 2, 2, True, 1.0, True),
    (50, 64, 4, "softmax", 2, 1, 1, False, 1.0, False),
    (45, 512, 8, "sigmoid", 16, 4, 2, True, 2.5, True),
    (45, 32, 5, "sigmoid", 32, 7, 2, True, 1.0, True),
]


def _route_case(T, E, dtype, with_bias, seed, masked=0):
    g = gen(seed)
    logits = (1.5 * randn(g, T, E) + 0.5 * randn(g, E))
    if masked:
        logits[torch.rand(T, E, generator=g, device="cuda") < masked] = -math.inf
    bias = 0.1 * randn(g, E) if with_bias else None
    return logits.to(dtype), bias


def _check_route(logits, bias, k, score, groups, top, gtop, renorm, scale):
    cfg = ops.RouteConfig(logits.shape[1], k, score, groups, top, gtop, renorm, scale)
    w, idx, n = ops.route(logits, cfg, bias=bias)
    rw, ri, rn = ref.route(logits, k, score, groups, top, gtop, renorm, scale, bias)
    assert torch.equal(idx.cpu(), ri)
    assert torch.equal(n.cpu(), rn)
    assert ((w.cpu().double() - rw).abs() <= W_TOL * rw.abs()).all()
    return w, idx, n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "T%d_E%d_k%d_%s_g%d" % c[:5])
def test_route(case, dtype):
    T, E, k, score, groups, top, gtop, renorm, scale, with_bias = case
    logits, bias = _route_case(T, E, dtype, with_bias, T + E)
    _check_route(logits, bias, k, score, groups, top, gtop, renorm, scale)


@pytest.mark.parametrize("masked", [0.3, 0.9, 1.1])
@pytest.mark.parametrize("case", [c for c in ROUTES if c[0] > 30], ids=lambda c: "T%d_E%d_k%d_%s_g%d" % c[:5])
def test_route_masked_experts(case, masked):
    """-inf logits; rows that keep fewer experts than choices, or none."""
    T, E, k, score, groups, top, gtop, renorm, scale, with_bias = case
    logits, bias = _route_case(T, E, torch.float32, with_bias, 5 * T + E, masked)
    w, idx, _ = _check_route(logits, bias, k, score, groups, top, gtop, renorm, scale)
    assert torch.equal(idx < 0, (idx < 0) & (w == 0))
    assert not w.isnan().any()


def test_route_nan_and_lowest_values():
    """NaN logits count as masked; the lowest finite number is a logit like others."""
    logits = torch.full((4, 40), torch.finfo(torch.float32).min, device="cuda")
    logits[0, 7] = math.nan
    logits[1, :] = math.nan
    logits[2, 3], logits[2, 9] = -math.inf, 0.0
    logits[3, 39] = 80.0
    for score in ("softmax", "sigmoid"):
        cfg = ops.RouteConfig(40, 3, score)
        w, idx, n = ops.route(logits, cfg)
        assert idx.tolist() == [[0, 1, 2], [-1, -1, -1], [9, 0, 1], [39, 0, 1]]
        assert not w.isnan().any() and (w[1] == 0).all()
        assert n.sum() == 9


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_route_ties_go_to_the_lower_index(score, groups, top):
    g = gen(1)
    logits = torch.randint(-1, 2, (200, 64), generator=g, device="cuda").float()
    bias = torch.where(torch.arange(64, device="cuda") % 2 == 0, 0.125, 0.0)
    for b in (None, bias):
        _check_route(logits, b, 6, score, groups, top, 2, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (8, 3)])
def test_route_near_ties_are_decided_in_64_bits(score, groups, top):
    """Keys that differ by less than fp32 scores can tell apart."""
    g = gen(2)
    base = randn(g, 300, 8).repeat_interleave(8, 1)[:, torch.randperm(64, generator=torch.Generator().manual_seed(0))]
    logits = base * (1 + 2.0 ** -22 * torch.randint(-2, 3, (300, 64), generator=g, device="cuda"))
    bias = (0.25 * randn(g, 8)).repeat(8)
    for b in (None, bias):
        _check_route(logits, b, 8, score, groups, top, 2, True, 1.0)


def test_route_scores_far_apart():
    """Large logits, biases that outweigh every score, biases that take experts out."""
    g = gen(9)
    logits = 12 * randn(g, 60, 96)
    bias = torch.zeros(96, device="cuda")
    bias[:10], bias[10:20], bias[20] = 1000.0, -math.inf, math.nan
    for score in ("softmax", "sigmoid"):
        cfg = ops.RouteConfig(96, 12, score, renormalize=False)
        w, idx, n = ops.route(logits, cfg, bias=bias)
        rw, ri, rn = ref.route(logits, 12, score, renorm=False, bias=bias)
        assert torch.equal(idx.cpu(), ri) and torch.equal(n.cpu(), rn)
        # |l - m| goes to 100 here, whose rounding is 2^-18.
        assert ((w.cpu().double() - rw).abs() <= 4 * W_TOL * rw.abs() + 1e-37).all()
        assert not ((idx >= 10) & (idx <= 20)).any()


def test_route_strided_logits_and_given_outputs():
    g = gen(4)
    big = randn(g, 30, 300)
    logits = big[:, 7:7 + 130]
    cfg = ops.RouteConfig(130, 5, "sigmoid")
    out = (torch.full((30, 5), 9.0, device="cuda"), torch.full((30, 5), 9, dtype=torch.int32, device="cuda"),
           torch.full((130,), 9, dtype=torch.int32, device="cuda"))
    w, idx, n = ops.route(logits, cfg, out=out)
    rw, ri, rn = ref.route(logits, 5, "sigmoid")
    assert torch.equal(idx.cpu(), ri) and torch.equal(n.cpu(), rn) and w is out[0]
    assert ((w.cpu().double() - rw).abs() <= W_TOL * rw).all()
    w2, idx2, none = ops.route(logits, cfg, counts=False)
    assert none is None and torch.equal(w2, w) and torch.equal(idx2, idx)


def test_route_no_tokens():
    cfg = ops.RouteConfig(16, 2)
    w, idx, n = ops.route(torch.empty(0, 16, device="cuda"), cfg)
    assert w.shape == (0, 2) and idx.shape == (0, 2) and (n == 0).all()
    assert ops.route_backward(w, torch.empty(0, 16, device="cuda"), idx, cfg).shape == (0, 16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,scale", [(1, 1, 1, 1.0), (9, 7, 3, 2.5), (40, 64, 6, 1.0), (33, 100, 32, 1.0),
                                         (20, 256, 8, 2.5), (11, 512, 10, 1.0)])
def test_route_backward(T, E, k, scale, score, renorm, dtype):
    logits, _ = _route_case(T, E, dtype, False, T * E)
    cfg = ops.RouteConfig(E, k, score, renormalize=renorm, scale=scale)
    _, idx, _ = ops.route(logits, cfg)
    g = randn(gen(5), T, k)
    d = ops.route_backward(g, logits, idx, cfg)
    l = logits.double().requires_grad_()
    ref.route_weights(l, idx, score, renorm, scale).backward(g.double())
    tol = G_TOL * scale * g.abs().max() + (HALF_BF16 * l.grad.abs() if dtype == torch.bfloat16 else 0)
    assert d.dtype == dtype and ((d.double() - l.grad).abs() <= tol).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(score, renorm):
    """Central differences of the 64-bit weights: their own error is h^2 / 6 times the third
    derivative (below 2 for these scores) and 2^-53 / h: 1e-6 at h = 1e-3."""
    logits, _ = _route_case(3, 12, torch.float32, False, 77)
    cfg = ops.RouteConfig(12, 4, score, renormalize=renorm)
    _, idx, _ = ops.route(logits, cfg)
    g = randn(gen(6), 3, 4)
    d = ops.route_backward(g, logits, idx, cfg).double()
    h, l = 1e-3, logits.double()
    for e in range(12):
        step = torch.zeros_like(l)
        step[:, e] = h
        up, dn = (ref.route_weights(l + s, idx, score, renorm, 1.0) for s in (step, -step))
        want = ((up - dn) * g.double()).sum(1) / (2 * h)
        assert ((d[:, e] - want).abs() <= G_TOL * g.abs().max() + 4e-6 * g.abs().sum(1)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_absent_and_repeated_choices(score, renorm):
    """Index -1 and indices outside the experts count as absent, a repeated one adds up; masked
    logits have no gradient, and a row without any choice none at all."""
    g = gen(8)
    logits = randn(g, 6, 20)
    logits[2, 4:9] = -math.inf
    logits[4] = -math.inf
    idx = torch.randint(0, 4, (6, 5), generator=g, device="cuda", dtype=torch.int32)
    idx[0] = torch.tensor([3, 3, 1, 3, 19])
    idx[1, 2:] = torch.tensor([-1, 20, 7], dtype=torch.int32)
    idx[3], idx[4] = -1, -1
    gw = randn(g, 6, 5)
    gw[3], gw[1, 2:4] = math.nan, math.nan  # never read
    cfg = ops.RouteConfig(20, 5, score, renormalize=renorm)
    d = ops.route_backward(gw, logits, idx, cfg)
    assert (d[3] == 0).all() and (d[4] == 0).all() and (d[2, 4:9] == 0).all()
    clean = torch.where((idx < 0) | (idx >= 20), -1, idx)
    keep = [0, 1, 2, 5]
    l = logits.double()[keep].requires_grad_()
    w = ref.route_weights(l, clean[keep], score, renorm, 1.0)
    (w * gw.double()[keep].nan_to_num(0.0)).sum().backward()
    assert ((d.double()[keep] - l.grad).abs() <= G_TOL * gw.nan_to_num(0.0).abs().max()).all()


def test_route_backward_strided():
    g = gen(12)
    big = randn(g, 10, 99)
    logits = big[:, 1:71]
    cfg = ops.RouteConfig(70, 4, "softmax", renormalize=False)
    _, idx, _ = ops.route(logits, cfg)
    gw = randn(g, 10, 4)
    buf = torch.full((10, 75), 5.0, device="cuda")
    d = ops.route_backward(gw, logits, idx, cfg, out=buf[:, 2:72])
    assert torch.equal(d, ops.route_backward(gw, logits.contiguous(), idx, cfg))
    assert (buf[:, :2] == 5).all() and (buf[:, 72:] == 5).all()


# ------------------------------------------------------------------ products


def _operands(g, fmt, R, G, N, K, exps=(0, 0)):
    a = ops.mx_quantize((randn(g, R, K) * 2.0 ** exps[0]).bfloat16(), fmt, scale_exp=exps[0])
    parts = [ops.mx_quantize(randn(g, N, K) * 2.0 ** exps[1] / math.sqrt(K), fmt, scale_exp=exps[1]) for _ in range(G)]
    w = ops.MxTensor(fmt, torch.stack([p.codes for p in parts]), torch.stack([p.scales for p in parts]), N, K, groups=G,
                     scale_exp=exps[1])
    return a, w, ops.mx_dequantize(a).double(), torch.stack([ops.mx_dequantize(p).double() for p in parts])


def _check_product(got, want, mass, K, act, bf16):
    tol = 1.13 * (K / 64 + 8) * 2.0 ** -22 * mass + 2.0 ** -20 * want.abs() + 1e-30
    if bf16:
        tol = tol + HALF_BF16 * (want.abs() + tol)
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (off / tol).max().item()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("R,N,K", [(1, 128, 256), (8, 128, 64), (16, 256, 128), (128, 128, 256), (3, 5, 32), (1, 1, 32), (130, 1, 96), (130, 77, 96),
                                   (65, 129, 320), (191, 64, 1056), (192, 384, 512), (193, 130, 2048), (500, 257, 416),
                                   (1000, 640, 7168)])
def test_product_of_one_group(fmt, R, N, K):
    a, w, av, wv = _operands(gen(R + N + K), fmt, R, 1, N, K)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        out = ops.mx_gemm(a, w, dtype=dtype, status=st)
        _check_product(out, av @ wv[0].T, av.abs() @ wv[0].abs().T, K, None, dtype == torch.bfloat16)
    assert st.item() == 0


def _plan(rows, extra=0):
    start, at = [], 0
    for r in rows:
        start.append(at)
        at += -(-r // 128) * 128
    return (torch.tensor(start, dtype=torch.int32, device="cuda"), torch.tensor(rows, dtype=torch.int32, device="cuda"),
            at + extra)


@pytest.mark.parametrize("fmt,act,bias,alpha", [("mxfp4", "gelu", True, False), ("mxfp4", None, False, True),
                                                ("nvfp4", "swish", True, True), ("nvfp4", "relu", False, False)])
@pytest.mark.parametrize("rows,N,K,extra", [([5, 0, 1, 33, 128, 0, 300, 17], 200, 512, 0), ([0, 0], 64, 64, 256),
                                            ([1] * 40, 96, 1024, 128), ([700, 2, 129, 1300], 384, 640, 64),
                                            ([0] * 199 + [3], 33, 96, 0), ([64, 65, 192, 193], 128, 288, 7)])
def test_product_of_groups(fmt, act, bias, alpha, rows, N, K, extra):
    g = gen(len(rows) + N + K)
    start, n, R = _plan(rows, extra)
    R = max(R, 1)
    exps = (0, 0) if fmt == "mxfp4" else (1, -4)
    a, w, av, wv = _operands(g, fmt, R, len(rows), N, K, exps)
    b = randn(g, len(rows), N) if bias else None
    al = torch.rand(len(rows), generator=g, device="cuda") + 0.5 if alpha else None
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((R, N), 77.0, dtype=dtype, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.mx_gemm(a, w, start, n, bias=b, alpha=al, activation=act, out=out, status=st)
        assert st.item() == 0
        live = torch.zeros(R, dtype=torch.bool, device="cuda")
        for e, r in enumerate(rows):
            s = slice(int(start[e]), int(start[e]) + r)
            live[s] = True
            c = 1.0 if al is None else al[e].double()
            z, mass = c * (av[s] @ wv[e].T), c * (av[s].abs() @ wv[e].abs().T)
            if b is not None:
                z, mass = z + b[e].double(), mass + b[e].double().abs()
            _check_product(out[s], ref.activate(z, act), mass, K, act, dtype == torch.bfloat16)
        assert (out[~live] == 77).all()


@pytest.mark.parametrize("fmt,G,N,K", [("mxfp4", 1024, 40, 96), ("nvfp4", 577, 33, 288), ("mxfp4", 90, 264, 4096),
                                       ("nvfp4", 17, 520, 4128)])
def test_product_of_many_groups(fmt, G, N, K):
    """Segments of every size around a tile's, in the forms for long ones: each row is there once."""
    g = gen(G)
    sizes = torch.tensor([0, 1, 31, 32, 33, 100, 191, 192, 193, 300, 383, 384, 385, 400], device="cuda")
    rows = sizes[torch.randint(0, 14, (G,), generator=g, device="cuda")].tolist()
    start, n, R = _plan(rows)
    exps = (0, 0) if fmt == "mxfp4" else (1, -4)
    a, w, av, wv = _operands(g, fmt, R, G, N, K, exps)
    out = torch.full((R, N), 77.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.mx_gemm(a, w, start, n, out=out, status=st)
    assert st.item() == 0
    live = torch.zeros(R, dtype=torch.bool, device="cuda")
    for e, (s, r) in enumerate(zip(start.tolist(), rows)):
        live[s:s + r] = True
        _check_product(out[s:s + r], av[s:s + r] @ wv[e].T, av[s:s + r].abs() @ wv[e].abs().T, K, None, True)
    assert (out[~live] == 77).all()


def test_product_of_extreme_scales():
    """Scales from one end of each format to the other: the sum is right where fp32 holds it."""
    for fmt, lo, hi in (("mxfp4", 100, 150), ("nvfp4", 1, 126)):
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        R, N, K = 100, 140, 384
        ca, cw = (torch.randint(0, 256, (n, K // 2), generator=g, device="cuda", dtype=torch.uint8) for n in (R, N))
        sa, sw = (torch.randint(lo, hi + 1, (1, n, K // ref.BLOCK[fmt]), generator=g, device="cuda",
                                dtype=torch.uint8) for n in (R, N))
        a = ops.MxTensor(fmt, ca, ops.mx_tile_scales(sa), R, K)
        w = ops.MxTensor(fmt, cw, ops.mx_tile_scales(sw), N, K)
        av = ref.values(ref.unpack(ca), sa[0], fmt)
        wv = ref.values(ref.unpack(cw), sw[0], fmt)
        out = ops.mx_gemm(a, w, dtype=torch.float32)
        _check_product(out, av @ wv.T, av.abs() @ wv.abs().T, K, None, False)


def test_product_keeps_nan_in_its_rows():
    """A NaN block of one row, or of one weight row, makes NaN of the outputs it is part of, and of no others."""
    g = gen(21)
    for fmt in ("mxfp4", "nvfp4"):
        x, wt = randn(g, 200, 256), randn(g, 150, 256)
        x[70, 100], wt[131, 3] = math.inf, math.nan
        a, w = ops.mx_quantize(x, fmt), ops.mx_quantize(wt, fmt)
        out = ops.mx_gemm(a, w, dtype=torch.float32)
        want = torch.zeros(200, 150, dtype=torch.bool, device="cuda")
        want[70], want[:, 131] = True, True
        assert torch.equal(out.isnan(), want)


def test_product_refuses_segments_outside_the_rows():
    """A segment that does not start at a multiple of 128 or leaves the rows is skipped and reported."""
    g = gen(22)
    a, w, av, wv = _operands(g, "mxfp4", 384, 5, 64, 128)
    start = torch.tensor([0, 64, 256, -128, 2 ** 31 - 128], dtype=torch.int32, device="cuda")
    n = torch.tensor([10, 5, 129, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = torch.full((384, 64), 77.0, dtype=torch.float32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.mx_gemm(a, w, start, n, out=out, status=st)
    assert st.item() == 2
    _check_product(out[:10], av[:10] @ wv[0].T, av[:10].abs() @ wv[0].abs().T, 128, None, False)
    assert (out[10:] == 77).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("off,ld,N", [(1, 301, 99), (2, 302, 99), (3, 401, 256), (0, 300, 98), (8, 304, 128)])
def test_product_into_strided_rows(dtype, off, ld, N):
    a, w, av, wv = _operands(gen(ld), "nvfp4", 140, 1, N, 160)
    buf = torch.full((140, ld), 5.0, dtype=dtype, device="cuda")
    out = ops.mx_gemm(a, w, out=buf[:, off:off + N])
    _check_product(out, av @ wv[0].T, av.abs() @ wv[0].abs().T, 160, None, dtype == torch.bfloat16)
    assert (buf[:, :off] == 5).all() and (buf[:, off + N:] == 5).all()


def test_product_repeats_bit_for_bit():
    a, w, _, _ = _operands(gen(30), "mxfp4", 700, 1, 500, 2048)
    first = ops.mx_gemm(a, w)
    for _ in range(5):
        assert torch.equal(ops.mx_gemm(a, w), first)


# ------------------------------------------------------------------ together


def _experts(logits, x, cfg, w1, w2, b1, bias=None):
    """Tokens through 4-bit experts: routing, rows by expert, two products, weighted sum."""
    wts, idx, counts = ops.route(logits, cfg, bias=bias)
    T, k = idx.shape
    G = cfg.num_experts
    e = idx.reshape(-1).long()
    start = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
    start[1:] = ((counts + 127) // 128 * 128).cumsum(0)
    order = e.argsort(stable=True)
    first = counts.cumsum(0) - counts
    row = torch.empty_like(e)
    row[order] = start[e[order]] + torch.arange(T * k, device="cuda") - first[e[order]]
    R = (T * k + G * 127) // 128 * 128
    index = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    index[row] = (torch.arange(T * k, device="cuda") // k).to(torch.int32)
    s32 = start.to(torch.int32)
    a = ops.mx_quantize(x, w1.format, row_index=index)
    h = ops.mx_gemm(a, w1, s32, counts, bias=b1, activation="swish")
    o = ops.mx_gemm(ops.mx_quantize(h, w2.format), w2, s32, counts, dtype=torch.float32)
    return (o[row].view(T, k, -1) * wts[..., None]).sum(1), idx, wts, h[row]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T", [1, 77])
def test_route_quantize_and_products_together(fmt, T):
    g = gen(40 + T)
    E, k, d, F = 16, 4, 256, 320
    logits, x = randn(g, T, E), randn(g, T, d).bfloat16()
    _, w1, _, v1 = _operands(g, fmt, 1, E, F, d, (0, -4 if fmt == "nvfp4" else 0))
    _, w2, _, v2 = _operands(g, fmt, 1, E, d, F, (0, -4 if fmt == "nvfp4" else 0))
    b1 = 0.1 * randn(g, E, F)
    cfg = ops.RouteConfig(E, k, "sigmoid", 4, 2, scale=2.5)
    y, idx, wts, h = _experts(logits, x, cfg, w1, w2, b1)
    rw, ri, _ = ref.route(logits, k, "sigmoid", 4, 2, scale=2.5)
    assert torch.equal(idx.cpu(), ri)
    # From the hidden activations as they were stored: what follows is exact up to fp32 sums.
    _, _, xv = ref.quantize(x, fmt)
    _, _, hv = ref.quantize(h, fmt)
    want, mass = torch.zeros(T, d, dtype=torch.float64, device="cuda"), 0
    for t in range(T):
        for r in range(k):
            e = int(ri[t, r])
            z = v1[e] @ xv[t] + b1[e].double()
            hw = ref.activate(z, "swish")
            m1 = v1[e].abs() @ xv[t].abs() + b1[e].double().abs()
            tol = 1.13 * (d / 64 + 8) * 2.0 ** -22 * m1
            assert ((h[t * k + r].double() - hw).abs() <= tol + HALF_BF16 * (hw.abs() + tol) + 2.0 ** -20 * hw.abs()).all()
            want[t] += rw[t, r].item() * (v2[e] @ hv[t * k + r])
            mass = max(mass, (v2[e].abs() @ hv[t * k + r].abs()).max().item())
    assert ((y.double() - want).abs() <= 2.5 * mass * ((F / 64 + 8) * 2.0 ** -22 + 2 * W_TOL)).all()


def test_captured_and_replayed_on_two_streams():
    """Everything in a CUDA graph, and two graphs at once on streams of their own."""
    g = gen(50)
    cfg = ops.RouteConfig(64, 6, "sigmoid", 8, 4)
    runs = []
    for i in range(2):
        logits, x, bias = randn(g, 200, 64), randn(g, 200, 512).bfloat16(), 0.1 * randn(g, 64)
        _, w, _, _ = _operands(g, "mxfp4", 1, 1, 300, 512)

        def step(logits=logits, x=x, bias=bias, w=w):
            wts, idx, n = ops.route(logits, cfg, bias=bias)
            d = ops.route_backward(wts, logits, idx, cfg)
            return wts, idx, n, d, ops.mx_gemm(ops.mx_quantize(x, "mxfp4"), w)

        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            got = step()
        runs.append((graph, stream, got, want, step))  # `step` keeps the inputs
    for _ in range(3):
        for graph, stream, got, _, _ in runs:
            with torch.cuda.stream(stream):
                for t in got:
                    t.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for _, _, got, want, _ in runs:
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_replays_read_what_was_just_quantised():
    """Rows quantised once, copied and multiplied, each kernel started while the one before it runs: a
    graph replayed on changing inputs gives what separate calls give."""
    g = gen(51)
    cols, N, G = 4096, 256, 4
    x = torch.empty(1100, cols, dtype=torch.bfloat16, device="cuda")
    index = torch.randint(0, 1100, (4 * 896,), generator=g, device="cuda", dtype=torch.int32)
    start = torch.arange(4, device="cuda", dtype=torch.int32) * 896
    count = torch.tensor([640, 0, 513, 1], device="cuda", dtype=torch.int32)
    _, w, _, _ = _operands(g, "nvfp4", 1, G, N, cols)
    out = torch.zeros(4 * 896, N, dtype=torch.bfloat16, device="cuda")

    def step():
        return ops.mx_gemm(ops.mx_quantize(x, "nvfp4", row_index=index), w, start, count, out=out)

    x.copy_(randn(g, 1100, cols))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        x.copy_(randn(g, 1100, cols))
        index.copy_(torch.randint(0, 1100, (4 * 896,), generator=g, device="cuda"))
        out.zero_()
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        q = ops.mx_quantize(x[index.long()], "nvfp4")
        torch.cuda.synchronize()
        want = ops.mx_gemm(q, w, start, count, out=torch.zeros_like(out))
        assert torch.equal(got, want)


# ------------------------------------------------------------------ offsets past 32 bits


def _ends(n, m=300):
    """The first and the last rows of n."""
    return torch.cat([torch.arange(m), torch.arange(n - m, n)]).cuda()


@pytest.mark.parametrize("E,score", [(256, "sigmoid"), (40, "softmax")])
def test_route_of_many_tokens(E, score):
    """More than 2^31 logits: the last tokens are routed as they are alone."""
    T = 2 ** 31 // E + 12345
    x = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(60))
    cfg = ops.RouteConfig(E, 2, score, renormalize=False)
    w, idx, n = ops.route(x, cfg)
    at = _ends(T)
    lw, li, _ = ops.route(x[at], cfg)
    assert torch.equal(idx[at], li) and torch.equal(w[at], lw)
    assert torch.equal(n.long(), torch.bincount(idx.reshape(-1), minlength=E))
    d = ops.route_backward(w, x, idx, cfg, out=torch.full_like(x, 7))
    assert torch.equal(d[at], ops.route_backward(w[at], x[at], idx[at], cfg))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_rows_and_products_past_32_bits(fmt):
    """More than 2^31 elements of x, 2^31 bytes of codes and 2^31 outputs."""
    g = gen(61)
    rows, cols = 2 ** 31 // 14336 + 40, 28672
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    at = _ends(rows)
    q, few = ops.mx_quantize(x, fmt), ops.mx_quantize(x[at], fmt)
    del x
    back = ops.mx_gather(q, at.to(torch.int32))
    assert torch.equal(back.codes, few.codes)
    assert torch.equal(ref.scale_bytes(back.scales, 600, cols, fmt), ref.scale_bytes(few.scales, 600, cols, fmt))
    assert torch.equal(ops.mx_dequantize(q, torch.bfloat16)[at], ops.mx_dequantize(few, torch.bfloat16))
    _, w, _, _ = _operands(g, fmt, 1, 1, 100, cols)
    assert torch.equal(ops.mx_gemm(q, w)[at], ops.mx_gemm(few, w))
    rows = 2 ** 31 // 640 + 77
    x = torch.empty(rows, 32, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    at = _ends(rows)
    _, w, _, _ = _operands(g, fmt, 1, 1, 640, 32)
    assert torch.equal(ops.mx_gemm(ops.mx_quantize(x, fmt), w)[at], ops.mx_gemm(ops.mx_quantize(x[at], fmt), w))


def test_errors_reach_python():
    with pytest.raises(MoEError):
        ops.route(torch.zeros(2, 6, device="cuda"), ops.RouteConfig(6, 2, num_groups=4))
    with pytest.raises(ValueError):
        ops.route(torch.zeros(2, 6, device="cuda").half(), ops.RouteConfig(6, 2))
    with pytest.raises(ValueError):
        ops.mx_quantize(torch.zeros(2, 64, device="cuda").t())
    with pytest.raises(ValueError):
        ops.mx_quantize(torch.zeros(2, 40, device="cuda"))
    with pytest.raises(MoEError):
        ops.mx_quantize(torch.zeros(2, 64, device="cuda"), scale_exp=99)
