"""Argument checks of the layer-free operators, on the host, before anything is enqueued (no GPU)."""
import copy
import ctypes
import pickle
import math

import pytest
import torch

import operators_ref as ref
from sparse_mixture_experts_gate_b200 import binding as B
from sparse_mixture_experts_gate_b200 import build
from sparse_mixture_experts_gate_b200 import operators as ops

P = 0x10000  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return B.lib()


def _route(L, c, logits=P, ld=None, T=4, bias=None, w=P, idx=P, n=None):
    return L.moe_route(ctypes.byref(c), logits, c.num_experts if ld is None else ld, T, bias, w, idx, n, None)


def _backward(L, c, g=P, logits=P, idx=P, T=4, out=P, ld=None, gld=None):
    return L.moe_route_backward(ctypes.byref(c), g, logits, c.num_experts if ld is None else ld, idx, T, out,
                                c.num_experts if gld is None else gld, None)


def test_route_default(L):
    c = B.moe_route_config_default()
    assert (c.num_experts, c.num_active, c.num_groups, c.top_groups, c.group_top, c.renormalize) == (8, 2, 1, 1, 2, 1)
    assert c.scale == 1.0 and c.dtype == B.MOE_DTYPE["fp32"] and c.score == B.MOE_SCORE["softmax"]


@pytest.mark.parametrize("change,code", [
    (dict(num_experts=0), B.MOE_ERR_INVALID_ARG), (dict(num_experts=513), B.MOE_ERR_UNSUPPORTED),
    (dict(num_active=0), B.MOE_ERR_INVALID_ARG), (dict(num_active=9), B.MOE_ERR_INVALID_ARG),
    (dict(num_experts=64, num_active=33), B.MOE_ERR_UNSUPPORTED), (dict(score=2), B.MOE_ERR_INVALID_ARG),
    (dict(num_groups=3), B.MOE_ERR_INVALID_ARG), (dict(num_groups=0), B.MOE_ERR_INVALID_ARG),
    (dict(num_experts=64, num_groups=64), B.MOE_ERR_UNSUPPORTED), (dict(num_groups=4, top_groups=5), B.MOE_ERR_INVALID_ARG),
    (dict(top_groups=0), B.MOE_ERR_INVALID_ARG), (dict(group_top=3), B.MOE_ERR_INVALID_ARG),
    (dict(num_groups=8, top_groups=1), B.MOE_ERR_INVALID_ARG), (dict(renormalize=2), B.MOE_ERR_INVALID_ARG),
    (dict(scale=math.inf), B.MOE_ERR_INVALID_ARG), (dict(dtype=7), B.MOE_ERR_INVALID_ARG)])
def test_route_config_refusals(L, change, code):
    c = B.moe_route_config_default()
    for k, v in change.items():
        setattr(c, k, v)
    assert _route(L, c) == code and B.moe_last_error()
    assert _backward(L, c) == code


def test_route_argument_refusals(L):
    c = B.moe_route_config_default()
    bad = B.MOE_ERR_INVALID_ARG
    assert L.moe_route(None, P, 8, 4, None, P, P, None, None) == bad
    assert _route(L, c, T=-1) == bad and _route(L, c, logits=None) == bad and _route(L, c, ld=7) == bad
    assert _route(L, c, w=None) == bad and _route(L, c, idx=None) == bad and _route(L, c, logits=P + 2) == bad
    assert _route(L, c, bias=P + 1) == bad and _route(L, c, n=P + 2) == bad
    assert _backward(L, c, g=None) == bad and _backward(L, c, logits=None) == bad and _backward(L, c, idx=None) == bad
    assert _backward(L, c, out=None) == bad and _backward(L, c, gld=7) == bad and _backward(L, c, T=-2) == bad
    assert _backward(L, c, out=P + 1) == bad


def _quantize(L, fmt=0, x=P, dtype=0, ld=64, x_rows=3, cols=64, index=None, rows=3, exp=0, codes=P, scales=P, values=None,
              vld=0):
    return L.moe_mx_quantize(fmt, x, dtype, ld, x_rows, cols, index, rows, exp, codes, scales, values, vld, None)


def test_quantize_refusals(L):
    bad = B.MOE_ERR_INVALID_ARG
    for kw in (dict(fmt=2), dict(dtype=3), dict(cols=0, ld=64), dict(cols=48), dict(cols=-32), dict(ld=63), dict(x_rows=-1),
               dict(rows=-1), dict(rows=4), dict(exp=61), dict(exp=-61), dict(x=None), dict(codes=None), dict(scales=None),
               dict(x=P + 1), dict(codes=P + 8), dict(scales=P + 4), dict(values=P + 1, vld=64), dict(values=P, vld=63),
               dict(index=P + 2)):
        assert _quantize(L, **kw) == bad, kw
        assert B.moe_last_error()
    assert _quantize(L, rows=0, x_rows=0) == B.MOE_OK
    ok = [0, P, P, 4, 64, P, 3, P, P, None]
    for i, v in ((0, 7), (1, None), (2, P + 4), (3, -1), (4, 48), (5, None), (5, P + 2), (6, -1), (7, None), (7, P + 8), (8, None)):
        a = list(ok)
        a[i] = v
        assert L.moe_mx_gather(*a) == bad, i
    assert L.moe_mx_gather(0, None, None, 0, 64, P, 3, P, P, None) == B.MOE_OK
    assert L.moe_mx_dequantize(0, P, P, 3, 64, 0, None, 0, 64, None) == bad
    assert L.moe_mx_dequantize(0, P, P, 3, 64, 0, P, 0, 60, None) == bad
    assert L.moe_mx_dequantize(0, P + 4, P, 3, 64, 0, P, 0, 64, None) == bad
    assert L.moe_mx_dequantize(1, P, P, 3, 40, 0, P, 0, 64, None) == bad
    assert L.moe_mx_dequantize(1, P, P, 0, 64, 0, None, 0, 64, None) == B.MOE_OK


def test_quantize_once_refusals(L):
    ok = dict(fmt=0, x=P, dtype=0, ld=64, x_rows=3, cols=64, index=P, rows=9, exp=0, codes=P, scales=P, ws=P, n=3 * 36)
    for change, code in ((dict(fmt=2), B.MOE_ERR_INVALID_ARG), (dict(x=None), B.MOE_ERR_INVALID_ARG), (dict(ld=63), B.MOE_ERR_INVALID_ARG),
                         (dict(dtype=2), B.MOE_ERR_INVALID_ARG), (dict(cols=48), B.MOE_ERR_INVALID_ARG),
                         (dict(index=None), B.MOE_ERR_INVALID_ARG), (dict(index=P + 2), B.MOE_ERR_INVALID_ARG),
                         (dict(rows=-1), B.MOE_ERR_INVALID_ARG), (dict(x_rows=-1), B.MOE_ERR_INVALID_ARG),
                         (dict(codes=None), B.MOE_ERR_INVALID_ARG), (dict(scales=P + 8), B.MOE_ERR_INVALID_ARG),
                         (dict(ws=None), B.MOE_ERR_INVALID_ARG), (dict(ws=P + 8), B.MOE_ERR_INVALID_ARG),
                         (dict(n=3 * 36 - 1), B.MOE_ERR_WORKSPACE), (dict(exp=61), B.MOE_ERR_INVALID_ARG),
                         (dict(rows=2 ** 31 - 1), B.MOE_ERR_UNSUPPORTED), (dict(rows=0), B.MOE_OK)):
        assert L.moe_mx_quantize_once(*{**ok, **change}.values(), None) == code, change
    assert B.moe_mx_once_bytes(0, 3, 64) == 3 * 36 and B.moe_mx_once_bytes(1, 5, 96) == 5 * (48 + 8)
    assert B.moe_mx_once_bytes(2, 3, 64) == 0 and B.moe_mx_once_bytes(0, -1, 64) == 0 and B.moe_mx_once_bytes(0, 3, 40) == 0


def test_sizes(L):
    assert B.moe_mx_codes_bytes(3, 64) == 96 and B.moe_mx_codes_bytes(3, 40) == 0 and B.moe_mx_codes_bytes(-1, 64) == 0
    assert B.moe_mx_scales_bytes(0, 1, 128) == 512 and B.moe_mx_scales_bytes(0, 129, 160) == 2048
    assert B.moe_mx_scales_bytes(1, 128, 128) == 1024 and B.moe_mx_scales_bytes(2, 1, 128) == 0
    assert B.moe_mx_scales_bytes(0, 0, 64) == 0


def test_product_refusals(L):
    ok = dict(format=0, rows=4, n=8, k=64, groups=1, scale_exp=0, activation=-1, out_dtype=0, out_ld=8, a_codes=P,
              a_scales=P, w_codes=P, w_scales=P, group_start=None, group_rows=None, bias=None, alpha=None, out=P,
              status=None)
    bad, no = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED
    for change, code in ((dict(format=5), bad), (dict(rows=-1), bad), (dict(n=0), bad), (dict(k=48), bad), (dict(k=0), bad),
                         (dict(groups=0), bad), (dict(groups=2), bad), (dict(groups=1025, group_start=P, group_rows=P), no),
                         (dict(group_start=P), bad), (dict(group_rows=P), bad), (dict(activation=3), bad),
                         (dict(activation=-2), bad), (dict(out_dtype=2), bad), (dict(out_ld=7), bad),
                         (dict(scale_exp=121), bad), (dict(a_codes=None), bad), (dict(w_scales=None), bad),
                         (dict(out=None), bad), (dict(a_codes=P + 8), bad), (dict(out=P + 1), bad),
                         (dict(status=P + 2), bad), (dict(bias=P + 2), bad),
                         (dict(groups=1024, group_start=P, group_rows=P, n=2 ** 21, out_ld=2 ** 21), no)):
        a = B.MoeMxGemm(**{**ok, **change})
        assert L.moe_mx_gemm(ctypes.byref(a), None) == code, change
        assert B.moe_last_error()
    assert L.moe_mx_gemm(None, None) == bad
    assert L.moe_mx_gemm(ctypes.byref(B.MoeMxGemm(**{**ok, "rows": 0})), None) == B.MOE_OK


def test_layer_calls_without_a_layer(L):
    c = B.moe_route_config_default()
    assert L.moe_set_routing(None, ctypes.byref(c)) == B.MOE_ERR_INVALID_ARG
    assert L.moe_prepare_experts_mx(None, 0, 0, 0, P, 1 << 20, None) == B.MOE_ERR_INVALID_ARG
    assert B.moe_experts_mx_bytes(None, 0) == 0


def test_python_refusals():
    with pytest.raises(ValueError):
        ops.RouteConfig(8, 2, score="tanh")
    cfg = ops.RouteConfig(8, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ops.route(torch.zeros(2, 8), cfg)
    with pytest.raises(ValueError, match="columns"):
        ops.route(torch.zeros(2, 7), cfg)
    with pytest.raises(ValueError, match="contiguous"):
        ops.route(torch.zeros(8, 2).t(), cfg)
    with pytest.raises(ValueError, match="out"):
        ops.route(torch.zeros(2, 8), cfg, out=(torch.zeros(2, 2), None, None))
    with pytest.raises(ValueError, match="bf16 or fp32"):
        ops.route(torch.zeros(2, 8, dtype=torch.float16), cfg)
    with pytest.raises(ValueError, match="bias"):
        ops.route(torch.zeros(2, 8), cfg, bias=torch.zeros(7))
    with pytest.raises(ValueError, match="row_index"):
        ops.mx_quantize(torch.zeros(2, 64), row_index=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="values"):
        ops.mx_quantize(torch.zeros(2, 64), values=torch.zeros(2, 32))
    with pytest.raises(ValueError, match="multiple of 32"):
        ops.mx_quantize(torch.zeros(2, 40))
    with pytest.raises(ValueError, match="grad_weights"):
        ops.route_backward(torch.zeros(2, 3), torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32), cfg)
    with pytest.raises(ValueError, match="format"):
        ops.mx_quantize(torch.zeros(2, 64), "fp4")
    with pytest.raises(ValueError, match="codes"):
        ops.MxTensor("mxfp4", torch.zeros(10, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 1, 64)
    codes, scales = torch.zeros(64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    a, w = ops.MxTensor("mxfp4", codes, scales, 2, 64), ops.MxTensor("nvfp4", codes, scales, 2, 64)
    with pytest.raises(ValueError, match="differ"):
        ops.mx_gemm(a, w)


def test_copies_of_a_routing_are_whole():
    cfg = ops.RouteConfig(60, 6, "sigmoid", 4, 2, 1, False, 2.5)
    for c in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg))):
        assert c._at == ctypes.addressof(c.struct) != cfg._at and bytes(c.struct) == bytes(cfg.struct)


def test_reference_rounds_as_the_formats_say():
    """The tests' own 64-bit rounding at every border (ties to the even code)."""
    u = torch.tensor([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] + [0.0] * 24], dtype=torch.float64)
    codes, byte, v = ref.quantize(u, "mxfp4")
    assert byte.tolist() == [[127]]
    assert v[0, :8].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]
    assert codes[0, :8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    assert ref.quantize(u * 1.3, "mxfp4")[2][0, 7] == 6.0
    _, byte, v = ref.quantize(torch.full((1, 32), 6.0 * 17, dtype=torch.float64), "nvfp4")
    assert v[0, 0] == 6.0 * 16  # 17 lies between the scales 16 and 18: the even one


def test_sizes_that_32_bits_do_not_hold(L):
    no, top = B.MOE_ERR_UNSUPPORTED, 2 ** 31 - 1
    assert _quantize(L, x_rows=top, rows=top) == no and _quantize(L, cols=2 ** 30 + 32, ld=2 ** 31) == no
    assert L.moe_mx_gather(0, P, P, 4, 64, P, top, P, P, None) == no
    assert L.moe_mx_dequantize(0, P, P, top, 64, 0, P, 0, 64, None) == no
    g = dict(format=0, k=64, scale_exp=0, activation=-1, out_dtype=0, a_codes=P, a_scales=P, w_codes=P, w_scales=P,
             group_start=P, group_rows=P, bias=None, alpha=None, out=P, status=None)
    for size in (dict(rows=top, n=8, groups=1), dict(rows=2 ** 28, n=1024, groups=512), dict(rows=2 ** 30, n=2 ** 18, groups=1),
                 dict(rows=4, n=2 ** 21, groups=1023 + 1)):
        a = B.MoeMxGemm(**g, **size, out_ld=size["n"])
        assert L.moe_mx_gemm(ctypes.byref(a), None) == no, size


def test_gather_refuses_its_own_rows(L):
    bad, n = B.MOE_ERR_INVALID_ARG, 1 << 20
    assert L.moe_mx_gather(0, P, P + n, 8, 64, P, 8, P, P + 2 * n, None) == bad
    assert L.moe_mx_gather(0, P, P + n, 8, 64, P, 8, P + 16, P + 2 * n, None) == bad
    assert L.moe_mx_gather(0, P, P + n, 8, 64, P, 300, P + 2 * n, P + n - 512, None) == bad
