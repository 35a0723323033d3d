"""Routing to experts and the experts' products in microscaled 4-bit floating point: cases to measure them on.

Four operators, each with its plain form in elementary torch operations:

  route           scores of the router's logits (softmax or sigmoid), a balance bias that takes part in the selection
                  only, selection of groups, top-k, renormalised and scaled weights, selections per expert
  route_backward  the gradient of those weights with respect to the logits
  quantize        rows to 4-bit codes with a scale per block: "mxfp4" (32 elements, power-of-two scales) and "nvfp4"
                  (16 elements, E4M3 scales, and one power of two for the whole tensor)
  experts         the tokens' rows gathered by expert, quantised, and multiplied with 4-bit expert weights, with bias
                  and activation

Sizes are those of the named workloads (default, e64, decode, e256) or lie around them.
"""
import math

import torch

own = False

# ------------------------------------------------------------------ the cases


def listed():
    return [
        # The decode workload's routing: latency, one token per sequence, 128 sequences.
        dict(name="route_decode", op="route", T=128, E=128, k=8, score="softmax", bias=False, groups=1, top_groups=1,
             renorm=True, scale=1.0, dtype="fp32", masked=0),
        # One sequence being answered: a single token, grouped sigmoid routing with a balance bias.
        dict(name="route_single", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             renorm=True, scale=2.5, dtype="fp32", masked=0),
        # A prefill or training batch of the e256 workload, grouped sigmoid routing with a balance bias.
        dict(name="route_e256", op="route", T=32768, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             renorm=True, scale=2.5, dtype="fp32", masked=0),
        # Training the e64 workload's router: the renormalised softmax, three experts taken out of service.
        dict(name="backward_e64", op="route_backward", T=8192, E=64, k=6, score="softmax", bias=False, groups=1,
             top_groups=1, renorm=True, scale=1.0, dtype="fp32", masked=3),
        # Training at the e256 sizes: the gradient of weights that are not renormalised reaches every logit.
        dict(name="backward_e256", op="route_backward", T=32768, E=256, k=8, score="softmax", bias=False, groups=1,
             top_groups=1, renorm=False, scale=1.0, dtype="fp32", masked=0),
        # The activations of one decode step.
        dict(name="quantize_decode", op="quantize", rows=128, cols=4096, format="mxfp4", exp=0, dtype="bf16"),
        # The activations of an e256 batch.
        dict(name="quantize_e256", op="quantize", rows=32768, cols=7168, format="nvfp4", exp=0, dtype="bf16"),
        # fp32 master weights of a width of 1408, an odd number of rows.
        dict(name="quantize_odd", op="quantize", rows=8191, cols=1408, format="mxfp4", exp=-6, dtype="fp32"),
        # One token through its 8 experts of the decode workload: the weights' bytes are all there is.
        dict(name="experts_single", op="experts", T=1, G=128, k=8, K=4096, N=1536, format="mxfp4", act="gelu",
             bias=True, zipf=True),
        # A decode step of 128 tokens, skewed popularity: few rows for each expert.
        dict(name="experts_decode", op="experts", T=128, G=128, k=8, K=4096, N=1536, format="mxfp4", act="gelu",
             bias=True, zipf=True),
        # The e64 workload's first layer: ragged segments, a width of 1408.
        dict(name="experts_e64", op="experts", T=8192, G=64, k=6, K=2048, N=1408, format="nvfp4", act="swish",
             bias=False, zipf=False),
        # An eighth of the e256 workload's experts with the rows that one of eight ranks gets.
        dict(name="experts_e256", op="experts", T=32768, G=32, k=1, K=7168, N=2048, format="mxfp4", act="swish",
             bias=False, zipf=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "quantize", "experts"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.choice([4, 7, 8, 12, 16, 20, 24, 32]) if groups > 1 else rng.randint(2, 256)
        E = groups * per
        top = rng.randint(1, groups)
        renorm = rng.random() < 0.7
        # One weight alone is 1 after renormalising, whatever its logit.
        k = rng.randint(2 if renorm else 1, min(16, top * per))
        free = E - k if groups == 1 else 0
        return dict(op=op, T=_log_int(rng, 1, 32768), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=op == "route" and rng.random() < 0.5, groups=groups, top_groups=top,
                    renorm=renorm, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "fp32", "bf16"]),
                    masked=min(free, rng.randint(0, 3)))
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op == "quantize":
        return dict(op=op, rows=_log_int(rng, 1, 16384), cols=32 * _log_int(rng, 1, 256), format=fmt,
                    exp=rng.randint(-8, 4), dtype=rng.choice(["bf16", "fp32"]))
    G = _log_int(rng, 1, 64)
    return dict(op=op, T=_log_int(rng, 1, 4096), G=G, k=rng.randint(1, min(4, G)), K=32 * _log_int(rng, 2, 128),
                N=_log_int(rng, 16, 2048), format=fmt, act=rng.choice(["none", "relu", "gelu", "swish"]),
                bias=rng.random() < 0.5, zipf=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs

_TORCH = {"fp32": torch.float32, "bf16": torch.bfloat16}
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _routing_inputs(case, gen):
    """Logits with a popularity of each expert, as a router in use has them; the last `masked` experts are out."""
    T, E = case["T"], case["E"]
    logits = 1.5 * _normal(gen, T, E) + 0.5 * _normal(gen, E)
    if case["masked"]:
        logits[:, E - case["masked"]:] = -math.inf
    bias = 0.1 * _normal(gen, E) if case["bias"] else None
    return logits.to(_TORCH[case["dtype"]]), bias


def _tile_scales(s):
    """Scales [G][N][S] in the order in which the product reads them: [G][N / 128][S / 4] tiles of 512 bytes, in each
    the byte of row n and scale j at (n % 32) * 16 + (n % 128 / 32) * 4 + j % 4; zeros past N and S."""
    G, N, S = s.shape
    nb, sb = -(-N // 128), -(-S // 4)
    p = torch.zeros(G, nb * 128, sb * 4, dtype=torch.uint8, device=s.device)
    p[:, :N, :S] = s
    return p.view(G, nb, 4, 32, sb, 4).permute(0, 1, 4, 3, 2, 5).contiguous()


def _weight_exp(case):
    """The power of two that is taken out of nvfp4 weights of variance 1 / K before their E4M3 scales."""
    return round(-0.5 * math.log2(case["K"])) if case["format"] == "nvfp4" else 0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "route":
        st["logits"], st["bias"] = _routing_inputs(case, gen)
    elif op == "route_backward":
        st["logits"], _ = _routing_inputs(case, gen)
        T, E, groups = case["T"], case["E"], case["groups"]
        # The forward's selection: the highest logits of the groups with the highest logits.
        key = st["logits"].float()
        if groups > 1:
            best = key.view(T, groups, E // groups).amax(2)
            out = torch.ones_like(best, dtype=torch.bool)
            out.scatter_(1, best.topk(case["top_groups"], dim=1).indices, False)
            key = key.masked_fill(out.repeat_interleave(E // groups, dim=1), -math.inf)
        st["idx"] = key.topk(case["k"], dim=1).indices.to(torch.int32)
        st["grad"] = _normal(gen, T, case["k"])
    elif op == "quantize":
        # Activations: normal, rows of different size, a few outlying columns.
        x = _normal(gen, case["rows"], case["cols"]) * torch.exp(0.5 * _normal(gen, case["rows"], 1))
        x *= torch.where(torch.rand(case["cols"], generator=gen, device="cuda") < 0.01, 12.0, 1.0)
        if case["exp"]:
            x *= 2.0 ** case["exp"]
        st["x"] = x.to(_TORCH[case["dtype"]])
    else:
        T, G, k, K, N = (case[n] for n in ("T", "G", "k", "K", "N"))
        st["x"] = _normal(gen, T, K).to(torch.bfloat16)
        # Which experts a token goes to: distinct ones, evenly or by a Zipf popularity.
        pop = torch.arange(1, G + 1, device="cuda", dtype=torch.float32).log().neg() if case["zipf"] else 0.0
        u = torch.rand(T, G, generator=gen, device="cuda").clamp_min(1e-20)
        choice = (pop - (-u.log()).log()).topk(k, dim=1).indices.reshape(-1)
        rows = torch.bincount(choice, minlength=G)
        # Each expert's rows in token order from a multiple of 128 on: the plan that a dispatch leaves.
        start = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
        start[1:] = ((rows + 127) // 128 * 128).cumsum(0)
        by_expert = choice.argsort(stable=True)
        first = rows.cumsum(0) - rows
        e = choice[by_expert]
        at = start[e] + torch.arange(T * k, device="cuda") - first[e]
        R = (T * k + G * 127) // 128 * 128
        st["row_index"] = torch.full((R,), -1, dtype=torch.int32, device="cuda")
        st["row_index"][at] = (by_expert // k).to(torch.int32)
        st["group_start"], st["group_rows"] = start.to(torch.int32), rows.to(torch.int32)
        st["most"] = int(rows.max())
        w = _normal(gen, G * N, K) / math.sqrt(K)
        codes, scales = _plain_quantize(w, case["format"], _weight_exp(case))
        del w
        st["w_codes"] = (codes[:, 0::2] | codes[:, 1::2] << 4).view(G, N, K // 2)
        st["w_scales"] = scales.view(G, N, K // BLOCK[case["format"]])
        st["w_tiles"] = _tile_scales(st["w_scales"])
        st["bias"] = 0.5 * _normal(gen, G, N) if case["bias"] else None
        # The user's output buffer: rows that no token fills stay as they are.
        st["out"] = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ the plain forms


def _plain_scores(logits, score):
    # In 64 bits: the selection is decided between neighbouring scores.
    l = logits.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    p = torch.exp(l - l.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _plain_route(logits, bias, case):
    T, E = logits.shape
    groups, k = case["groups"], case["k"]
    s = _plain_scores(logits, case["score"])
    if bias is not None:
        key = s + bias.double()
    else:
        key = s if groups > 1 else logits.double()
    key = torch.where(logits.isneginf(), -math.inf, key)
    if groups > 1:
        best = key.view(T, groups, E // groups).sort(dim=2, descending=True).values[:, :, :2]
        total = torch.where(best.isneginf(), 0.0, best).sum(2)
        total = torch.where(best[:, :, 0].isneginf(), -math.inf, total)
        chosen = total.sort(dim=1, descending=True, stable=True).indices[:, : case["top_groups"]]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=key.device).scatter_(1, chosen, True)
        key = torch.where(keep.repeat_interleave(E // groups, dim=1), key, -math.inf)
    best = key.sort(dim=1, descending=True, stable=True)
    idx, found = best.indices[:, :k], ~best.values[:, :k].isneginf()
    w = torch.where(found, s.gather(1, idx), 0.0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    counts = torch.zeros(E, dtype=torch.int32, device=key.device)
    counts.index_add_(0, idx.reshape(-1), found.reshape(-1).to(torch.int32))
    return {"weights": (w * case["scale"]).float(), "idx": torch.where(found, idx, -1).to(torch.int32),
            "counts": counts}


def _plain_route_backward(grad, logits, idx, case):
    l, c = logits.float(), case["scale"]
    at = idx.long()
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
        r = s.gather(1, at)
        ds = 1 - r
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        s = p / p.sum(1, keepdim=True)
        r = s.gather(1, at)
    if case["renorm"]:
        q = r / r.sum(1, keepdim=True)
        d = c * q * (grad - (grad * q).sum(1, keepdim=True))
        if case["score"] == "sigmoid":
            d = d * ds
        return torch.zeros_like(l).scatter_(1, at, d).to(logits.dtype)
    if case["score"] == "sigmoid":
        return torch.zeros_like(l).scatter_(1, at, c * grad * r * ds).to(logits.dtype)
    g = torch.zeros_like(l).scatter_(1, at, grad)
    return (c * s * (g - (grad * r).sum(1, keepdim=True))).to(logits.dtype)


def _pow2(e):
    """2^e of whole numbers in -252..254, exactly, from the bits of two 32-bit numbers."""
    h = e // 2
    return ((h + 127) << 23).view(torch.float32) * ((e - h + 127) << 23).view(torch.float32)


def _plain_scale_values(scales, fmt, exp):
    """The scale bytes' values, in 32 bits."""
    if fmt == "mxfp4":
        return _pow2(scales.to(torch.int32) - 127)
    return scales.view(torch.float8_e4m3fn).float() * 2.0 ** exp


def _plain_quantize(x, fmt, exp):
    """Codes [rows][cols] (one in each byte) and scale bytes [rows][cols / block]. Powers of two come out of 32-bit
    numbers exactly, and so does everything that a code depends on."""
    R, C = x.shape
    b = x.float().view(R, C // BLOCK[fmt], BLOCK[fmt])
    top = b.abs().amax(2)
    if fmt == "mxfp4":
        e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
        u = b * _pow2(-e)[:, :, None]
        scales = (e + 127).to(torch.uint8)
    else:
        s = (top * 2.0 ** -exp / 6).clamp_max(448.0).to(torch.float8_e4m3fn)
        scales, s = s.view(torch.uint8), s.float()[:, :, None]
        u = torch.where(s > 0, b * 2.0 ** -exp / s, 0.0)
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp_max(6.0)
    code = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
    code = torch.where(b.signbit(), code | 8, code)
    return code.view(R, C), scales


def _plain_values(codes, scales, fmt, exp):
    """What codes (one in each byte) and scale bytes stand for, in 32 bits."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = table[codes.int()].view(*scales.shape, BLOCK[fmt])
    return (v * _plain_scale_values(scales, fmt, exp)[..., None]).view(codes.shape)


def _plain_act(z, act):
    if act == "relu":
        return torch.clamp_min(z, 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "swish":
        return z / (1 + torch.exp(-z))
    return z


def _plain_experts(st, case):
    G, N, K, fmt = case["G"], case["N"], case["K"], case["format"]
    codes, scales = _plain_quantize(st["x"], fmt, 0)
    a = _plain_values(codes, scales, fmt, 0)
    wc = torch.stack((st["w_codes"] & 15, st["w_codes"] >> 4), 3).view(G, N, K)
    w = _plain_values(wc, st["w_scales"], fmt, _weight_exp(case))
    # Every expert's rows, filled up to the longest segment: one batched product.
    R = st["row_index"].shape[0]
    at = torch.arange(st["most"], device=a.device)
    live = at < st["group_rows"][:, None]
    row = torch.where(live, st["group_start"][:-1, None] + at, 0)
    token = torch.where(live, st["row_index"][row], 0)
    z = torch.bmm(a[token], w.transpose(1, 2))
    if st["bias"] is not None:
        z += st["bias"][:, None]
    y = _plain_act(z, case["act"]).to(torch.bfloat16)
    out = torch.zeros(R + 1, N, dtype=torch.bfloat16, device=a.device)
    out[torch.where(live, row, R).reshape(-1)] = y.view(-1, N)
    return out[:R]


# ------------------------------------------------------------------ one pass


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from sparse_mixture_experts_gate_b200 import operators as ops
        if op == "route":
            cfg = _config(ops, state)
            w, idx, counts = ops.route(state["logits"], cfg, bias=state["bias"])
            return {"weights": w, "idx": idx, "counts": counts}
        if op == "route_backward":
            return ops.route_backward(state["grad"], state["logits"], state["idx"], _config(ops, state))
        if op == "quantize":
            values = torch.empty_like(state["x"])
            ops.mx_quantize(state["x"], case["format"], scale_exp=case["exp"], values=values)
            return values
        if "w" not in state:
            state["w"] = ops.MxTensor(case["format"], state["w_codes"], state["w_tiles"], case["N"], case["K"],
                                      groups=case["G"], scale_exp=_weight_exp(case))
        a = ops.mx_quantize(state["x"], case["format"], row_index=state["row_index"])
        return ops.mx_gemm(a, state["w"], group_start=state["group_start"], group_rows=state["group_rows"],
                           bias=state["bias"], activation=case["act"], out=state["out"])
    if op == "route":
        return _plain_route(state["logits"], state["bias"], case)
    if op == "route_backward":
        return _plain_route_backward(state["grad"], state["logits"], state["idx"], case)
    if op == "quantize":
        codes, scales = _plain_quantize(state["x"], case["format"], case["exp"])
        return _plain_values(codes, scales, case["format"], case["exp"]).to(state["x"].dtype)
    return _plain_experts(state, case)


def _config(ops, state):
    """The routing's configuration, which a program makes once."""
    if "config" not in state:
        c = state["case"]
        state["config"] = ops.RouteConfig(c["E"], c["k"], score=c["score"], num_groups=c["groups"],
                                          top_groups=c["top_groups"], renormalize=c["renorm"], scale=c["scale"])
    return state["config"]


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_route(st, case):
    l = st["logits"].double()
    T, E = l.shape
    out = l == -math.inf
    if case["score"] == "sigmoid":
        s = torch.where(l >= 0, 1 / (1 + torch.exp(-l.abs())), torch.exp(-l.abs()) / (1 + torch.exp(-l.abs())))
    else:
        s = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    if case["bias"]:
        key = s + st["bias"].double()
    else:
        key = l.clone() if case["groups"] == 1 else s.clone()
    key[out] = -math.inf
    gs = E // case["groups"]
    number = torch.arange(E, device=l.device)
    if case["groups"] > 1:
        total = []
        for g in range(case["groups"]):
            part = key[:, g * gs:(g + 1) * gs].clone()
            m1, a1 = part.max(1)
            part[torch.arange(T, device=l.device), a1] = -math.inf
            m2 = part.max(1).values
            total.append(torch.where(m2 == -math.inf, m1, m1 + m2))
        total = torch.stack(total, 1)
        # A group is in when fewer than top_groups groups are before it: higher, or as high with a lower number.
        gn = torch.arange(case["groups"], device=l.device)
        before = (total[:, None, :] > total[:, :, None]) | (
            (total[:, None, :] == total[:, :, None]) & (gn[None, None, :] < gn[None, :, None]))
        inside = before.sum(2) < case["top_groups"]
        key[~inside.repeat_interleave(gs, 1)] = -math.inf
    picks, weights = [], []
    for _ in range(case["k"]):
        top = key.max(1, keepdim=True).values
        e = torch.where(key == top, number, E).min(1).values
        none = top[:, 0] == -math.inf
        picks.append(torch.where(none, -1, e))
        weights.append(torch.where(none, 0.0, s[torch.arange(T, device=l.device), e]))
        key[torch.arange(T, device=l.device), e] = -math.inf
    idx, w = torch.stack(picks, 1), torch.stack(weights, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    counts = torch.bincount(idx[idx >= 0], minlength=E)
    return {"weights": w * case["scale"], "idx": idx.to(torch.int32), "counts": counts.to(torch.int32)}


def _exact_route_backward(st, case):
    l, g, at = st["logits"].double(), st["grad"].double() * case["scale"], st["idx"].long()
    r = l.gather(1, at)
    if case["score"] == "softmax":
        if case["renorm"]:  # the softmax over the selected logits alone
            q = torch.softmax(r, 1)
            return torch.zeros_like(l).scatter_(1, at, q * g - q * (q * g).sum(1, keepdim=True))
        p = torch.softmax(l, 1)
        m = (p.gather(1, at) * g).sum(1, keepdim=True)
        return (-p * m).scatter_add_(1, at, p.gather(1, at) * g)
    s = torch.sigmoid(r)
    if case["renorm"]:
        total = s.sum(1, keepdim=True)
        g = g / total - (g * s).sum(1, keepdim=True) / total ** 2
    return torch.zeros_like(l).scatter_(1, at, g * s * torch.sigmoid(-r))


_MIDDLES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _floor_pow2(v, lo, hi):
    """The largest power of two up to v, between 2^lo and 2^hi, from a table: exact at the powers themselves."""
    table = torch.tensor([2.0 ** i for i in range(lo, hi + 1)], dtype=torch.float64, device=v.device)
    return table[(torch.bucketize(v, table, right=True) - 1).clamp_min(0)]


def _exact_values(x, fmt, exp):
    """What the rows of x are after quantisation, in 64 bits: the nearest of the eight levels, the even one of two."""
    R, C = x.shape
    b = x.double().view(R, -1, BLOCK[fmt])
    top = b.abs().amax(2, keepdim=True)
    if fmt == "mxfp4":
        scale = _floor_pow2(top / 4, -127, 127)
    else:
        v = top * 2.0 ** -exp / 6
        step = _floor_pow2(v, -6, 8) / 8
        scale = (torch.round(v / step) * step).clamp_max(448.0) * 2.0 ** exp
    u = b.abs() / torch.where(scale > 0, scale, 1.0)
    n = torch.zeros_like(u, dtype=torch.int64)
    for i, m in enumerate(_MIDDLES):
        n += (u >= m) if i % 2 else (u > m)
    level = torch.tensor(_LEVELS, dtype=torch.float64, device=x.device)[n]
    return (torch.sign(b) * level * scale).view(R, C)


def _exact_experts(st, case):
    G, N, K, fmt = case["G"], case["N"], case["K"], case["format"]
    a = _exact_values(st["x"], fmt, 0)
    level = torch.tensor(_LEVELS, dtype=torch.float64, device=a.device)
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=a.device)
    start, rows = st["group_start"].tolist(), st["group_rows"].tolist()
    for g in range(G):
        if not rows[g]:
            continue
        c = torch.stack((st["w_codes"][g] & 15, st["w_codes"][g] // 16), 2).view(N, K).long()
        w = torch.where(c >= 8, -1.0, 1.0).double() * level[c % 8]
        s = st["w_scales"][g].long()
        if fmt == "mxfp4":
            values = [2.0 ** (i - 127) for i in range(255)] + [math.nan]
        else:
            values = [2.0 ** (max(i // 8, 1) - 10) * ((i // 8 > 0) * 8 + i % 8) for i in range(127)] + [math.nan] * 129
        s = torch.tensor(values, dtype=torch.float64, device=a.device)[s]
        if fmt == "nvfp4":
            s = s * 2.0 ** _weight_exp(case)
        w = w * s.repeat_interleave(BLOCK[fmt], 1)
        token = st["row_index"][start[g]:start[g] + rows[g]].long()
        z = a[token] @ w.T
        if case["bias"]:
            z = z + st["bias"][g].double()
        if case["act"] == "relu":
            z = torch.where(z > 0, z, 0.0)
        elif case["act"] == "gelu":
            z = 0.5 * z * torch.erfc(-z / math.sqrt(2))
        elif case["act"] == "swish":
            z = z * torch.sigmoid(z)
        out[start[g]:start[g] + rows[g]] = z
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st, case)
    if op == "route_backward":
        return _exact_route_backward(st, case)
    if op == "quantize":
        return _exact_values(st["x"], case["format"], case["exp"])
    return _exact_experts(st, case)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op = case["op"]
    if op in ("route", "route_backward"):
        size = 2 if case["dtype"] == "bf16" else 4
        T, E, k = case["T"], case["E"], case["k"]
        if op == "route":  # logits in; weights, indices and counts out; the scores' and the selection's operations
            return {"bytes": T * E * size + T * k * 8 + E * 4 + (E * 4 if case["bias"] else 0), "flops": T * E * 8}
        # Every logit is read only where the gradient needs it; the gradient is written whole.
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * (E if dense else k) * size + T * k * 8 + T * E * size, "flops": T * (E if dense else k) * 8}
    block = BLOCK[case["format"]]
    if op == "quantize":
        n, size = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * size * 2 + n // 2 + n // block, "flops": n * 4}
    T, G, k, K, N = (case[n] for n in ("T", "G", "k", "K", "N"))
    touched = min(G, T * k)
    w = touched * N * (K // 2 + K // block)
    return {"bytes": T * K * 2 + w + T * k * (4 + N * 2) + (touched * N * 4 if case["bias"] else 0),
            "flops": 2 * T * k * K * N}
