"""Plain 64-bit implementations of the routing and 4-bit operators, for their tests."""
import math

import torch

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
BLOCK = {"mxfp4": 32, "nvfp4": 16}
E4M3 = [2.0 ** (max(i // 8, 1) - 10) * ((i // 8 > 0) * 8 + i % 8) for i in range(127)]
E8M0 = [2.0 ** (i - 127) for i in range(255)]


def _nearest(v, levels):
    """Index of the nearest level for v >= 0, the even index of two, the last one above all."""
    t = torch.tensor(levels, dtype=torch.float64, device=v.device)
    hi = torch.bucketize(v, t).clamp(1, len(levels) - 1)  # first level >= v
    lo = hi - 1
    dl, dh = v - t[lo], t[hi] - v
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def quantize(x, fmt, exp=0):
    """(codes [R][C] one in each byte, scale bytes [R][C / block], values in 64 bits)."""
    R, C = x.shape
    b = x.double().view(R, C // BLOCK[fmt], BLOCK[fmt]) * 2.0 ** -exp
    top = b.abs().amax(2)
    fine = torch.isfinite(b).all(2)
    top = torch.where(fine, top, 1.0)
    if fmt == "mxfp4":
        table = torch.tensor(E8M0, dtype=torch.float64, device=x.device)
        byte = (torch.bucketize(top / 4, table, right=True) - 1).clamp(0, 254)
        nan = 255
    else:
        table = torch.tensor(E4M3, dtype=torch.float64, device=x.device)
        byte = _nearest(top / 6, E4M3)
        nan = 127
    s = table[byte]
    u = torch.where(s[..., None] > 0, b.abs() / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    u = torch.where(fine[..., None], u, 0.0)
    mag = _nearest(u, LEVELS)
    neg = b.signbit() & fine[..., None] & (s[..., None] > 0)
    codes = mag + 8 * neg
    v = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)[mag] * torch.where(neg, -1.0, 1.0) * s[..., None]
    v = torch.where(fine[..., None], v, math.nan) * 2.0 ** exp
    byte = torch.where(fine, byte, nan)
    return codes.view(R, C).to(torch.uint8), byte.to(torch.uint8), v.view(R, C)


def scale_bytes(tiles, rows, cols, fmt, group=0):
    """The scale bytes [rows][blocks] out of the tiles, by the layout's formula."""
    nb = cols // BLOCK[fmt]
    SB = -(-nb // 4)
    r = torch.arange(rows, device=tiles.device)[:, None]
    j = torch.arange(nb, device=tiles.device)[None, :]
    at = (r // 128 * SB + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4
    return tiles.reshape(-1)[at + group * -(-rows // 128) * SB * 512]


def unpack(codes):
    """Codes one in each byte."""
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def values(codes, byte, fmt, exp=0):
    table = torch.tensor(E8M0 + [math.nan] if fmt == "mxfp4" else E4M3 + [math.nan], dtype=torch.float64,
                         device=codes.device)
    lv = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=codes.device)
    return lv[codes.long()] * table[byte.long()].repeat_interleave(BLOCK[fmt], -1) * 2.0 ** exp


def activate(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "swish":
        return z * torch.sigmoid(z)
    return z


def route(logits, k, score, groups=1, top_groups=1, group_top=2, renorm=True, scale=1.0, bias=None):
    """(weights, idx, counts), token by token."""
    T, E = logits.shape
    l = logits.double().cpu()
    b = None if bias is None else bias.double().cpu()
    W, I = torch.zeros(T, k, dtype=torch.float64), torch.full((T, k), -1, dtype=torch.int32)
    counts = torch.zeros(E, dtype=torch.int32)
    for t in range(T):
        row = [float(v) for v in l[t]]
        live = [e for e in range(E) if row[e] != -math.inf and not math.isnan(row[e])]
        if not live:
            continue
        m = max(row[e] for e in live)
        if score == "sigmoid":
            s = {e: float(torch.sigmoid(l[t, e])) for e in live}
        else:
            z = math.fsum(math.exp(row[e] - m) for e in live)
            s = {e: math.exp(row[e] - m) / z for e in live}
        if b is not None:
            key = {e: s[e] + float(b[e]) for e in live}
        else:
            key = dict(s) if groups > 1 else {e: row[e] for e in live}
        key = {e: v for e, v in key.items() if v != -math.inf and not math.isnan(v)}
        if groups > 1:
            gs = E // groups
            total = {}
            for g in range(groups):
                inside = sorted((key[e] for e in key if e // gs == g), reverse=True)[:group_top]
                total[g] = sum(inside) if inside else -math.inf
            chosen = sorted(total, key=lambda g: (-total[g], g))[:top_groups]
            key = {e: v for e, v in key.items() if e // gs in chosen}
        order = sorted(key, key=lambda e: (-key[e], e))[:k]
        total = sum(s[e] for e in order)
        for r, e in enumerate(order):
            I[t, r] = e
            W[t, r] = scale * s[e] / (total if renorm else 1.0)
            counts[e] += 1
    return W, I, counts


def route_weights(logits, idx, score, renorm, scale):
    """The weights of a given selection, differentiable, in 64 bits; absent choices weigh 0."""
    l = logits.double()
    live = idx >= 0
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    w = torch.where(live, s.gather(1, idx.clamp_min(0).long()), 0.0)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return w * scale
