"""Layers routed by scores, against 64 bits (GPU).

The experts' arithmetic is made exact: tokens, weights and biases are small whole numbers, few of them not 0, so
that with ReLU every hidden activation and every expert's output is a whole number below 256, which bf16 holds. What
is left is the combine: y is off by (k + S + 2) 2^-23 of the sum of its terms' magnitudes, and by half a step of the
layer's type (2^-8 for bf16, 2^-24 for fp32) of itself. Gates are the layer's own, which are compared with 64 bits by
themselves (4e-6 of a weight, see test_operators_gpu.py).
"""
import pytest
import torch

import operators_ref as ref
from sparse_mixture_experts_gate_b200 import operators as ops
from sparse_mixture_experts_gate_b200.binding import MoELayer, StepGraph, ep_send_splits
from sparse_mixture_experts_gate_b200.workloads import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu

def whole(w, seed):
    """Inputs of the workload with experts and tokens of small whole numbers."""
    inp = make_inputs(w, "cpu", seed=seed, random_biases=True)
    g = torch.Generator().manual_seed(seed)

    def few(like, n):  # about n of each row's elements are -1 or 1
        r = torch.rand(like.shape, generator=g)
        p = n / like.shape[-1] / 2
        return torch.where(r < p, -1.0, torch.where(r < 2 * p, 1.0, 0.0)).to(like.dtype)

    inp["x"] = torch.randint(-2, 3, inp["x"].shape, generator=g).to(inp["x"].dtype)
    inp["w1"], inp["w2"] = few(inp["w1"], 6), few(inp["w2"], 6)
    inp["b1"], inp["b2"] = (torch.randint(-3, 4, inp[n].shape, generator=g).to(inp[n].dtype) for n in ("b1", "b2"))
    return inp


def experts(w, W, x, out):
    """(y, how far it may be off) in 64 bits from the layer's routing."""
    u = 2.0 ** -8 if w.dtype == "bf16" else 2.0 ** -24
    x = x.double()
    T = x.shape[0]
    y = torch.zeros(T, w.O, dtype=torch.float64, device="cuda")
    mass = torch.zeros_like(y)
    for e in range(w.E + w.S):
        if e < w.E:
            t, r = ((out["topk_idx"] == e) & (out["slot"] >= 0)).nonzero(as_tuple=True)
            g = out["gates"][t, r].double()[:, None]
        else:
            t, g = torch.arange(T, device="cuda"), torch.ones(T, 1, dtype=torch.float64, device="cuda")
        w1, b1, w2, b2 = (W[n][e].cuda().double() for n in ("w1", "b1", "w2", "b2"))
        h = (x[t] @ w1.T + b1).clamp_min(0)
        o = h @ w2.T + b2
        if len(t):
            assert h.max() < 256 and o.abs().max() < 256  # what makes the sums exact
        y.index_add_(0, t, g * o)
        mass.index_add_(0, t, (g * o).abs())
    off = (w.k + w.S + 2) * 2.0 ** -23 * mass
    return y, off + u * (y.abs() + off)


def check(w, W, x, out, kw, bias=None):
    rw, ri, rn = ref.route(out["logits"], w.k, kw["score"], kw.get("num_groups", 1), kw.get("top_groups", 1),
                           kw.get("group_top", 2), kw.get("renormalize", True), kw.get("scale", 1.0), bias)
    assert torch.equal(out["topk_idx"].cpu(), ri) and torch.equal(out["count_pre"].cpu(), rn)
    assert ((out["gates"].cpu().double() - rw).abs() <= 4e-6 * rw.abs()).all()
    y, off = experts(w, W, x, out)
    assert ((out["y"].double() - y).abs() <= off).all()
    return y, off


@pytest.mark.parametrize("kw", [dict(score="sigmoid", num_groups=4, top_groups=2, scale=2.5), dict(score="sigmoid", renormalize=False),
                                dict(score="softmax", renormalize=False, scale=16.0)], ids=lambda k: "_".join(str(v) for v in k.values()))
@pytest.mark.parametrize("name,T,more", [("default", 400, {}), ("e64", 77, {}), ("default", 130, dict(S=2, capacity_factor=0.5)),
                                         ("tiny", 37, {})])
def test_outputs_of_layers_routed_by_scores(name, T, more, kw):
    w = WORKLOADS[name].with_(T=T, activation="relu", **more)
    if w.E < 8:
        kw = {**kw, "num_groups": min(kw.get("num_groups", 1), 2), "top_groups": 1}
    inp = whole(w, 17)
    layer = MoELayer(w, inp)
    x = inp["x"].cuda()
    layer.set_routing(ops.RouteConfig(w.E, w.k, **kw))
    out = layer.forward(x)
    y, off = check(w, layer.weights, x, out, kw, layer.weights["sel_bias"] if w.use_selection_bias else None)
    # The bound tells the gates from others: those of the choices the other way round are outside it.
    other = dict(out, gates=out["gates"].flip(1))
    assert ((experts(w, layer.weights, x, other)[0] - y).abs() > off).any(1).float().mean() > 0.5
    # Twice the scale is twice every gate and, without shared experts, twice y, bit for bit.
    if w.S == 0:
        once = {n: out[n].clone() for n in ("y", "gates")}
        layer.set_routing(ops.RouteConfig(w.E, w.k, **{**kw, "scale": 2 * kw.get("scale", 1.0)}))
        twice = layer.forward(x)
        assert torch.equal(twice["gates"], 2 * once["gates"]) and torch.equal(twice["y"], 2 * once["y"])


def test_two_expert_parallel_ranks_route_by_scores():
    """The phases of two ranks in one process (the exchange by slicing): each rank's tokens are routed by scores
    with its own capacity and come out as with all experts in one place."""
    G = 2
    kw = dict(score="sigmoid", num_groups=4, top_groups=2, scale=2.5)
    w = WORKLOADS["e64"].with_(T=300, E=16, k=4, S=1, d=256, F=384, O=320, capacity_factor=1.0, activation="relu")
    inp = whole(w, 52)
    El = w.E // G
    layers, xs, first = [], [], []
    for r in range(G):
        local = dict(inp)
        for key in ("w1", "b1", "w2", "b2"):
            local[key] = torch.cat([inp[key][r * El:(r + 1) * El], inp[key][w.E:]])
        layers.append(MoELayer(w, local, ep_size=G, ep_rank=r))
        layers[r].set_routing(ops.RouteConfig(w.E, w.k, **kw))
        xs.append(whole(w, 310 + r)["x"].cuda())
        first.append(layers[r].ep_dispatch(xs[r]))

    def exchange(rows, splits):
        return [torch.cat([rows[r][sum(splits[r][:q]):sum(splits[r][:q + 1])] for r in range(G)]) for q in range(G)]

    there = [ep_send_splits(f[3], G) for f in first]
    recv = exchange([f[1] for f in first], there)
    done = []
    for q in range(G):
        counts = torch.tensor([first[r][3][q * El:(q + 1) * El] for r in range(G)], dtype=torch.int32).cuda()
        done.append(layers[q].ep_experts(recv[q], counts))
    back = exchange(done, [[there[r][q] for r in range(G)] for q in range(G)])
    for r in range(G):
        out = first[r][0]
        first[r][2][:back[r].shape[0]].copy_(back[r])
        layers[r].ep_combine(out)
        torch.cuda.synchronize()
        assert layers[r].device_status() == 0
        check(w, inp, xs[r], out, kw, layers[r].weights["sel_bias"] if w.use_selection_bias else None)


def test_a_captured_step_keeps_its_routing():
    """set_routing is for forwards that are enqueued after it: a graph replays what it was captured with."""
    w = WORKLOADS["e64"].with_(T=100)
    inp = make_inputs(w, "cpu", seed=4)
    layer = MoELayer(w, inp)
    x = inp["x"].cuda()
    plain = StepGraph(layer, x)
    before = {n: plain.replay()[n].clone() for n in ("y", "gates", "topk_idx")}
    cfg = ops.RouteConfig(w.E, w.k, "sigmoid", 8, 4, scale=2.5)
    layer.set_routing(cfg)
    scored = StepGraph(layer, x)
    layer.set_routing(None)
    got = scored.replay()
    gates, idx, _ = ops.route(got["logits"], cfg, bias=layer.weights["sel_bias"] if w.use_selection_bias else None)
    assert torch.equal(got["gates"], gates) and torch.equal(got["topk_idx"], idx)
    again = plain.replay()
    assert all(torch.equal(again[n], before[n]) for n in before)
