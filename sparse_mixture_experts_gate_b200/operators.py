"""The operators of libmoe.so that need no layer, on torch tensors.

Routing to experts from given logits and its gradient (`route`, `route_backward`),
and microscaled 4-bit floating point: rows of codes and scales (`MxTensor`), made by
`mx_quantize` (and `mx_gather`), read back by `mx_dequantize`, and multiplied with 4-bit expert
weights by `mx_gemm`. Checks and pointer marshalling only; the work is done by the
kernels behind the C ABI (include/moe.h has the definitions). Every call runs on the
current stream of its tensors' device; nothing is differentiable through autograd.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import binding as B

_DTYPE = {torch.bfloat16: 0, torch.float32: 1}
_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda device: torch.cuda.current_stream(device).cuda_stream
_current = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _call(device: int, where: str, fn, *args):
    """fn(*args, the current stream of `device`) with that device current."""
    if device < 0:
        raise ValueError("the operators take CUDA tensors")
    if device == _current():
        rc = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(device))
    if rc:
        raise B.MoEError(rc, where, B.moe_last_error())


# Contiguous tensors; of the ways to make them the one that takes the least host time.
_empty = torch.empty_strided


def _rows(name: str, t: torch.Tensor, cols: Optional[int] = None) -> int:
    """The row stride of a matrix whose rows are contiguous."""
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name}: a matrix{'' if cols is None else f' of {cols} columns'} is needed, "
                         f"got {tuple(t.shape)}")
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name}: bf16 or fp32, got {t.dtype}")
    rows, width = t.shape
    ld, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{name}: rows have to be contiguous")
    return ld if rows > 1 and ld >= width else (width if rows <= 1 else ld)


def _array(name: str, t: torch.Tensor, like: torch.Tensor, dtype, shape=None) -> int:
    """The address of a contiguous array."""
    if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != like.get_device() or \
            (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: a contiguous {dtype} tensor{'' if shape is None else f' of {tuple(shape)}'} on "
                         f"{like.device} is needed, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


class RouteConfig:
    """How tokens are routed: `score` "softmax" or "sigmoid"; with num_groups > 1 only the
    experts of the top_groups best groups (by the sum of their group_top highest keys);
    weights renormalised over the selection or not, times `scale`."""

    def __init__(self, num_experts: int, num_active: int, score: str = "softmax", num_groups: int = 1,
                 top_groups: int = 1, group_top: int = 2, renormalize: bool = True, scale: float = 1.0):
        if score not in B.MOE_SCORE:
            raise ValueError(f"unknown score {score!r}")
        self.num_experts, self.num_active = num_experts, num_active
        self._c = {d: B.MoeRouteConfig(num_experts, num_active, B.MOE_SCORE[score], num_groups, top_groups, group_top,
                                       int(renormalize), scale, code) for d, code in _DTYPE.items()}
        self._ref = {d: ctypes.byref(c) for d, c in self._c.items()}


def route(logits: torch.Tensor, cfg: RouteConfig, bias: Optional[torch.Tensor] = None, counts: bool = True,
          out=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Routes the tokens of logits [T][E] (bf16 or fp32). Returns (weights [T][k] fp32,
    topk_idx [T][k] int32, selections per expert [E] int32 or None); `out`: these
    three to write into. bias [E] fp32 takes part in the selection only."""
    E, k = cfg.num_experts, cfg.num_active
    ld = _rows("logits", logits, E)
    T, dev = logits.shape[0], logits.device
    b = None if bias is None else _array("bias", bias, logits, torch.float32, (E,))
    if out is None:
        w = _empty((T, k), (k, 1), dtype=torch.float32, device=dev)
        idx = _empty((T, k), (k, 1), dtype=torch.int32, device=dev)
        n = _empty((E,), (1,), dtype=torch.int32, device=dev) if counts else None
    else:
        w, idx, n = out
        _array("weights", w, logits, torch.float32, (T, k))
        _array("topk_idx", idx, logits, torch.int32, (T, k))
        if n is not None:
            _array("counts", n, logits, torch.int32, (E,))
    _call(logits.get_device(), "moe_route", B.lib().moe_route, cfg._ref[logits.dtype], logits.data_ptr(), ld, T, b,
          w.data_ptr(), idx.data_ptr(), None if n is None else n.data_ptr())
    return w, idx, n


def route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor, cfg: RouteConfig,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient with respect to logits, given that of route's weights [T][k] fp32."""
    ld = _rows("logits", logits, cfg.num_experts)
    T = logits.shape[0]
    shape = (T, cfg.num_active)
    g = _array("grad_weights", grad_weights, logits, torch.float32, shape)
    idx = _array("topk_idx", topk_idx, logits, torch.int32, shape)
    if out is None:
        out = _empty((T, cfg.num_experts), (cfg.num_experts, 1), dtype=logits.dtype, device=logits.device)
        out_ld = cfg.num_experts
    else:
        if out.dtype != logits.dtype or out.shape != logits.shape or out.device != logits.device:
            raise ValueError("out has to be like logits")
        out_ld = _rows("out", out)
    _call(logits.get_device(), "moe_route_backward", B.lib().moe_route_backward, cfg._ref[logits.dtype], g,
          logits.data_ptr(), ld, idx, T, out.data_ptr(), out_ld)
    return out


def _code_bytes(rows: int, cols: int) -> int:
    return rows * (cols // 2)


def _scale_bytes(fmt: str, rows: int, cols: int) -> int:
    tile_k = 4 * _BLOCK[fmt]
    return (rows + 127) // 128 * ((cols + tile_k - 1) // tile_k) * 512


class MxTensor:
    """Rows of microscaled 4-bit floating point: `groups` matrices of rows x cols ("mxfp4" or
    "nvfp4"), codes [groups * rows][cols / 2] and scale tiles as uint8 tensors on one device,
    and the power of two scale_exp that the values count in."""

    def __init__(self, fmt: str, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int, groups: int = 1,
                 scale_exp: int = 0):
        if fmt not in _BLOCK:
            raise ValueError(f"unknown format {fmt!r}")
        if cols < 32 or cols % 32:
            raise ValueError(f"a row needs a positive multiple of 32 elements, got {cols}")
        for name, t, need in (("codes", codes, groups * _code_bytes(rows, cols)),
                              ("scales", scales, groups * _scale_bytes(fmt, rows, cols))):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() < need or t.device != codes.device:
                raise ValueError(f"{name}: at least {need} contiguous bytes on one device are needed")
        self._set(fmt, codes, scales, rows, cols, groups, scale_exp)

    def _set(self, fmt, codes, scales, rows, cols, groups, scale_exp):
        self.format, self.codes, self.scales = fmt, codes, scales
        self.rows, self.cols, self.groups, self.scale_exp = rows, cols, groups, scale_exp


def mx_tile_scales(scales: torch.Tensor) -> torch.Tensor:
    """Scale bytes [groups][rows][blocks] (a checkpoint's plain order) as scale tiles."""
    G, N, S = scales.shape
    nb, sb = -(-N // 128), -(-S // 4)
    p = torch.zeros(G, nb * 128, sb * 4, dtype=torch.uint8, device=scales.device)
    p[:, :N, :S] = scales
    return p.view(G, nb, 4, 32, sb, 4).permute(0, 1, 4, 3, 2, 5).contiguous()


def _empty_mx(fmt: str, rows: int, cols: int, scale_exp: int, device) -> MxTensor:
    q = MxTensor.__new__(MxTensor)
    q._set(fmt, _empty((rows, cols // 2), (cols // 2, 1), dtype=torch.uint8, device=device),
           _empty((_scale_bytes(fmt, rows, cols),), (1,), dtype=torch.uint8, device=device), rows, cols, 1, scale_exp)
    return q


def mx_quantize(x: torch.Tensor, fmt: str = "mxfp4", row_index: Optional[torch.Tensor] = None, scale_exp: int = 0,
                values: Optional[torch.Tensor] = None, out: Optional[MxTensor] = None) -> MxTensor:
    """Rows of x (bf16 or fp32) to 4 bits. row_index [rows] int32: output row r is x's row
    row_index[r], and is left as it was where that is no row of x. `values`, in x's type,
    receives what the codes stand for; `out`: an MxTensor to write into."""
    ld = _rows("x", x)
    x_rows, cols = x.shape
    if fmt not in _BLOCK:
        raise ValueError(f"unknown format {fmt!r}")
    if cols < 32 or cols % 32:
        raise ValueError(f"a row needs a positive multiple of 32 elements, got {cols}")
    if row_index is None:
        rows, index = x_rows, None
    else:
        rows, index = row_index.numel(), _array("row_index", row_index, x, torch.int32)
    if out is None:
        out = _empty_mx(fmt, rows, cols, scale_exp, x.device)
    elif (out.format, out.rows, out.cols, out.groups, out.scale_exp) != (fmt, rows, cols, 1, scale_exp) or \
            out.codes.device != x.device:
        raise ValueError("out has another format, size, exponent or device")
    if index is not None and values is None and rows >= 2 * x_rows and rows * cols >= 1 << 22:
        # Rows that are wanted several times are quantised once and copied, where that is worth a launch.
        q = mx_quantize(x, fmt, scale_exp=scale_exp)
        _call(x.get_device(), "moe_mx_gather", B.lib().moe_mx_gather, B.MOE_MX[fmt], q.codes.data_ptr(),
              q.scales.data_ptr(), x_rows, cols, index, rows, out.codes.data_ptr(), out.scales.data_ptr())
        return out
    v = v_ld = 0
    if values is not None:
        if values.dtype != x.dtype or values.shape != (rows, cols) or values.device != x.device:
            raise ValueError(f"values: {x.dtype} {(rows, cols)} on {x.device} is needed")
        v, v_ld = values.data_ptr(), _rows("values", values)
    _call(x.get_device(), "moe_mx_quantize", B.lib().moe_mx_quantize, B.MOE_MX[fmt], x.data_ptr(), _DTYPE[x.dtype], ld,
          x_rows, cols, index, rows, scale_exp, out.codes.data_ptr(), out.scales.data_ptr(), v or None, v_ld)
    return out


def mx_gather(q: MxTensor, row_index: torch.Tensor, out: Optional[MxTensor] = None) -> MxTensor:
    """Rows row_index [rows] (int32) of q; a row is left as it was in `out` where row_index is
    no row of q."""
    if q.groups != 1:
        raise ValueError("one group at a time")
    rows = row_index.numel()
    index = _array("row_index", row_index, q.codes, torch.int32)
    if out is None:
        out = _empty_mx(q.format, rows, q.cols, q.scale_exp, q.codes.device)
    elif (out.format, out.rows, out.cols, out.groups, out.scale_exp) != (q.format, rows, q.cols, 1, q.scale_exp) or \
            out.codes.device != q.codes.device:
        raise ValueError("out has another format, size, exponent or device")
    _call(q.codes.get_device(), "moe_mx_gather", B.lib().moe_mx_gather, B.MOE_MX[q.format], q.codes.data_ptr(),
          q.scales.data_ptr(), q.rows, q.cols, index, rows, out.codes.data_ptr(), out.scales.data_ptr())
    return out


def mx_dequantize(q: MxTensor, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values of q, [rows][cols] (one group)."""
    if dtype not in _DTYPE:
        raise ValueError(f"bf16 or fp32, got {dtype}")
    if q.groups != 1:
        raise ValueError("one group at a time")
    out = torch.empty(q.rows, q.cols, dtype=dtype, device=q.codes.device)
    _call(out.get_device(), "moe_mx_dequantize", B.lib().moe_mx_dequantize, B.MOE_MX[q.format], q.codes.data_ptr(),
          q.scales.data_ptr(), q.rows, q.cols, q.scale_exp, out.data_ptr(), _DTYPE[dtype], q.cols)
    return out


def mx_gemm(a: MxTensor, w: MxTensor, group_start: Optional[torch.Tensor] = None,
            group_rows: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
            alpha: Optional[torch.Tensor] = None, activation: Optional[str] = None, out: Optional[torch.Tensor] = None,
            dtype: torch.dtype = torch.bfloat16, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act(alpha_g a w_g^T + bias_g) for the rows of every group g: rows group_start[g] ..
    + group_rows[g] of a (int32, starts multiples of 128), or all rows with one group and
    neither given. Rows of no group are left as they were in `out`, or hold anything where
    `out` is not given. status: an int32 tensor of one zero, whose bit 0 reports a wait that
    gave up and bit 1 a segment outside the rows."""
    if a.format != w.format or a.cols != w.cols:
        raise ValueError(f"operands differ: {a.format} of {a.cols} columns, {w.format} of {w.cols}")
    if a.groups != 1:
        raise ValueError("a has one group of rows")
    like = a.codes
    if w.codes.device != like.device:
        raise ValueError("operands on different devices")
    G, n = w.groups, w.rows
    start = rows = None
    if group_start is not None:
        start = _array("group_start", group_start, like, torch.int32)
    if group_rows is not None:
        rows = _array("group_rows", group_rows, like, torch.int32)
    if (start is not None and group_start.numel() < G) or (rows is not None and group_rows.numel() < G):
        raise ValueError(f"group_start and group_rows: one entry for each of {G} groups is needed")
    b = None if bias is None else _array("bias", bias, like, torch.float32, (G, n))
    al = None if alpha is None else _array("alpha", alpha, like, torch.float32, (G,))
    st = None if status is None else _array("status", status, like, torch.int32, (1,))
    if activation is None or activation == "none":
        act = B.MOE_ACT_NONE
    elif activation in B.MOE_ACT:
        act = B.MOE_ACT[activation]
    else:
        raise ValueError(f"unknown activation {activation!r}")
    if out is None:
        out = _empty((a.rows, n), (n, 1), dtype=dtype, device=like.device)
    elif out.device != like.device or out.shape[0] != a.rows:
        raise ValueError(f"out: {a.rows} rows on {like.device} are needed")
    ld = _rows("out", out, n)
    args = B.MoeMxGemm(B.MOE_MX[a.format], a.rows, n, a.cols, G, a.scale_exp + w.scale_exp, act, _DTYPE[out.dtype], ld,
                       like.data_ptr(), a.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(), start, rows, b, al,
                       out.data_ptr(), st)
    _call(like.get_device(), "moe_mx_gemm", B.lib().moe_mx_gemm, ctypes.byref(args))
    return out
