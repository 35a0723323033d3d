"""The layer's forwards with routing by scores (moe_set_routing) and with 4-bit experts
(moe_prepare_experts_mx), on the GPU.

Routing is compared with a plain 64-bit implementation on the layer's own logits. 4-bit
experts are compared with the layer-free operators, which have their own tests against 64
bits, on the layer's own routing: the experts' outputs are the same bits, so y is off by the
combine's fp32 sums (2^-20 of the sum of magnitudes) and half a bf16 step (2^-8 of y).
"""
import math

import pytest
import torch

import operators_ref as ref
from sparse_mixture_experts_gate_b200 import binding
from sparse_mixture_experts_gate_b200 import operators as ops
from sparse_mixture_experts_gate_b200.binding import MoEError, MoELayer, StepGraph
from sparse_mixture_experts_gate_b200.workloads import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu


def forward(layer, inp, poison=True):
    x = inp["x"].cuda()
    ws, _ = layer.workspace(x.shape[0])
    if poison:
        ws.fill_(0xFF)
    out = layer.forward(x, noise=None if inp.get("noise") is None else inp["noise"].cuda())
    tl = inp.get("token_loss")
    layer.aux_stats(out, token_loss=None if tl is None else tl.cuda())
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    return out


def bf16_experts(layer, inp, out):
    """y in 64 bits from the layer's routing: hidden activations and outputs rounded to bf16, as stored."""
    w, W = layer.w, layer.weights
    x = inp["x"].cuda().double()
    y = torch.zeros(x.shape[0], w.O, dtype=torch.float64, device="cuda")
    for e in range(w.E + w.S):
        if e < w.E:
            t, r = ((out["topk_idx"] == e) & (out["slot"] >= 0)).nonzero(as_tuple=True)
            g = out["gates"][t, r].double()
        else:
            t, g = torch.arange(x.shape[0], device="cuda"), torch.ones(x.shape[0], dtype=torch.float64, device="cuda")
        h = ref.activate(x[t] @ W["w1"][e].double().T + W["b1"][e].double(), w.activation).bfloat16().double()
        y.index_add_(0, t, g[:, None] * (h @ W["w2"][e].double().T + W["b2"][e].double()).bfloat16().double())
    return y


ROUTINGS = [dict(score="sigmoid", num_groups=8, top_groups=4, scale=2.5), dict(score="sigmoid", renormalize=False),
            dict(score="softmax", num_groups=4, top_groups=2, group_top=1), dict(score="softmax", renormalize=False, scale=16.0)]


@pytest.mark.parametrize("kw", ROUTINGS, ids=lambda k: "_".join(str(v) for v in k.values()))
@pytest.mark.parametrize("name,T", [("e64", 300), ("default", 1000), ("e64", 1), ("tiny", 37)])
def test_layer_routes_by_scores(name, T, kw):
    w = WORKLOADS[name].with_(T=T)
    if w.E < 16:
        kw = {**kw, "num_groups": min(kw.get("num_groups", 1), 2), "top_groups": 1 if w.E == 4 else min(kw.get("top_groups", 1), 2)}
    inp = make_inputs(w, "cpu", seed=31, random_biases=True)
    layer = MoELayer(w, inp)
    before = {k: v.clone() for k, v in forward(layer, inp).items()}
    cfg = ops.RouteConfig(w.E, w.k, **kw)
    layer.set_routing(cfg)
    out = forward(layer, inp)
    assert torch.equal(out["logits"], before["logits"]) and torch.equal(out["p_mean"], before["p_mean"])
    assert torch.equal(out["l_z"], before["l_z"])
    bias = layer.weights["sel_bias"] if w.use_selection_bias else None
    rw, ri, rn = ref.route(out["logits"], w.k, kw["score"], kw.get("num_groups", 1), kw.get("top_groups", 1),
                           kw.get("group_top", 2), kw.get("renormalize", True), kw.get("scale", 1.0), bias)
    assert torch.equal(out["topk_idx"].cpu(), ri) and torch.equal(out["count_pre"].cpu(), rn)
    assert ((out["gates"].cpu().double() - rw).abs() <= 4e-6 * rw.abs()).all()
    # y: bf16 storage of H, the experts' outputs and y, as for the other routing (2e-2), scaled gates as they are.
    want = bf16_experts(layer, inp, out) if w.dtype == "bf16" else None
    if want is not None:
        assert ((out["y"].double() - want).abs() <= 2e-2 * (1 + want.abs()) * max(1.0, kw.get("scale", 1.0))).all()
    layer.set_routing(None)
    back = forward(layer, inp)
    for k in ("y", "topk_idx", "gates", "slot", "count_pre", "credit", "l_aux", "f"):
        assert torch.equal(back[k].nan_to_num(-7.0), before[k].nan_to_num(-7.0)), k


def test_layer_fills_choices_that_are_left_over():
    """Biases that leave 3 of 64 experts: the other choices are the lowest free experts, with gate 0."""
    w = WORKLOADS["e64"].with_(T=150)
    inp = make_inputs(w, "cpu", seed=5)
    inp["sel_bias"] = torch.full((64,), -math.inf)
    inp["sel_bias"][[2, 40, 63]] = 0.5
    layer = MoELayer(w, inp)
    layer.set_routing(ops.RouteConfig(64, 6, "sigmoid", 4, 3))
    out = forward(layer, inp)
    idx, gates = out["topk_idx"].cpu(), out["gates"].cpu()
    assert sorted(set(idx[:, :3].flatten().tolist())) == [2, 40, 63]
    assert (idx[:, 3:] == torch.tensor([0, 1, 3])).all() and (gates[:, 3:] == 0).all()
    assert ((gates.sum(1) - 1).abs() < 1e-5).all() and out["y"].isfinite().all()


def mx_experts(layer, inp, out, fmt, exps):
    """y from the layer-free operators on the layer's routing, and the experts' outputs by assignment."""
    w, W = layer.w, layer.weights
    x = inp["x"].cuda()
    T, G = x.shape[0], w.E + w.S
    kept = torch.cat((out["count_kept"].long(), torch.full((w.S,), T, device="cuda")))
    start = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
    start[1:] = ((kept + 127) // 128 * 128).cumsum(0)
    R = max(int(start[-1]), 1)
    index = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    live = out["slot"] >= 0
    row = start[out["topk_idx"].long()] + out["slot"]
    tok = torch.arange(T, device="cuda")
    index[row[live]] = tok[:, None].expand(T, w.k)[live].to(torch.int32)
    for s in range(w.S):
        index[start[w.E + s] + tok] = tok.to(torch.int32)

    def weights(v, e):
        parts = [ops.mx_quantize(v[g], fmt, scale_exp=e) for g in range(G)]
        return ops.MxTensor(fmt, torch.stack([p.codes for p in parts]), torch.stack([p.scales for p in parts]), v.shape[1],
                            v.shape[2], groups=G, scale_exp=e)

    s32, n32 = start.to(torch.int32), kept.to(torch.int32)
    a = ops.mx_quantize(x, fmt, row_index=index)
    h = ops.mx_gemm(a, weights(W["w1"], exps[0]), s32, n32, bias=W["b1"], activation=w.activation)
    o = ops.mx_gemm(ops.mx_quantize(h, fmt), weights(W["w2"], exps[1]), s32, n32, bias=W["b2"]).double()
    part = torch.where(live[..., None], o[row.clamp_min(0)], 0.0)
    terms = [out["gates"].double()[..., None] * part] + [o[start[w.E + s] + tok][:, None] for s in range(w.S)]
    terms = torch.cat(terms, 1)
    return terms.sum(1), terms.abs().sum(1), part


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("name,T,kw", [("default", 1000, {}), ("e64", 700, {}), ("e64", 1, {}), ("decode", 128, {}), ("e64", 2100, {}),
                                       ("default", 260, dict(S=2, capacity_factor=0.3, activation="relu")),
                                       ("e64", 150, dict(capacity_factor=0.0, credit_norm="hidden")),
                                       ("default", 300, dict(E=1, k=1, capacity_factor=0.0))])
def test_layer_with_4_bit_experts(name, T, kw, fmt):
    w = WORKLOADS[name].with_(T=T, **kw)
    inp = make_inputs(w, "cpu" if name != "decode" else "cuda", seed=12, random_biases=True)
    layer = MoELayer(w, inp)
    before = {k: v.clone() for k, v in forward(layer, inp).items()}
    layer.prepare_experts_mx(fmt)
    out = forward(layer, inp)
    for k in ("logits", "topk_idx", "gates", "slot", "count_pre", "count_kept", "f", "p_mean", "l_aux", "l_z"):
        assert torch.equal(out[k], before[k]), k
    exps = [round(-0.5 * math.log2(n)) if fmt == "nvfp4" else 0 for n in (w.d, w.F)]
    want, mass, part = mx_experts(layer, inp, out, fmt, exps)
    assert ((out["y"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * mass + 2.0 ** -8 * 2.0 ** -20 * mass).all()
    if w.credit_norm == "output":
        credit = out["gates"].double() * part.norm(dim=2)
        assert ((out["credit"].double() - credit).abs() <= 1e-5 * (1 + credit)).all()
    layer.prepare_experts_mx(None)
    back = forward(layer, inp)
    assert torch.equal(back["y"], before["y"]) and torch.equal(back["credit"], before["credit"])


def test_layer_with_both_replayed_from_a_graph():
    w = WORKLOADS["e64"].with_(T=500)
    inp = make_inputs(w, "cpu", seed=3)
    layer = MoELayer(w, inp)
    layer.set_routing(ops.RouteConfig(w.E, w.k, "sigmoid", 8, 4, scale=2.5))
    layer.prepare_experts_mx("mxfp4")
    eager = {k: v.clone() for k, v in forward(layer, inp, poison=False).items()}
    g = StepGraph(layer, inp["x"].cuda())
    for _ in range(3):
        g.out["y"].zero_()
        out = g.replay()
        torch.cuda.synchronize()
        for k in ("y", "topk_idx", "gates", "credit", "l_total"):
            assert torch.equal(out[k], eager[k]), k


def test_layer_refusals():
    w = WORKLOADS["default"].with_(T=8)
    inp = make_inputs(w, "cpu")
    layer = MoELayer(w, inp)
    for cfg in (ops.RouteConfig(16, 2), ops.RouteConfig(8, 3), ops.RouteConfig(8, 2, num_groups=3)):
        with pytest.raises(MoEError):
            layer.set_routing(cfg)
    c = ops.RouteConfig(8, 2)
    c.struct.dtype = binding.MOE_DTYPE["bf16"]
    with pytest.raises(MoEError):
        layer.set_routing(c)
    c.struct.dtype = binding.MOE_DTYPE["fp32"]
    n = binding.moe_experts_mx_bytes(layer.handle, 0)
    buf = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    for fmt, e1, at, size in ((2, 0, 0, n), (0, 99, 0, n), (0, 0, 0, n - 1), (0, 0, 128, n)):
        with pytest.raises(MoEError):
            binding.moe_prepare_experts_mx(layer.handle, fmt, e1, 0, buf.data_ptr() + at, size, s)
    noisy = WORKLOADS["default"].with_(T=8, top_k_method="noisy", noise=True)
    with pytest.raises(MoEError, match="NOISY"):
        MoELayer(noisy, make_inputs(noisy, "cpu")).set_routing(c)
    tiny = WORKLOADS["tiny"]
    fp32 = MoELayer(tiny, make_inputs(tiny, "cpu"))
    assert binding.moe_experts_mx_bytes(fp32.handle, 0) == 0
    with pytest.raises(MoEError):
        binding.moe_prepare_experts_mx(fp32.handle, 0, 0, 0, buf.data_ptr(), n, s)
    # A statistics call needs a forward of the layout that is in force.
    forward(layer, inp)
    out = layer.alloc_outputs(8)
    layer.prepare_experts_mx("nvfp4")
    with pytest.raises(MoEError):
        layer.aux_stats(out)
