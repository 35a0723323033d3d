"""The operators of libmoe.so that need no layer, on torch tensors.

Routing to experts from given logits and its gradient (`route`, `route_backward`),
and microscaled 4-bit floating point: rows of codes and scales (`MxTensor`), made by
`mx_quantize` (and `mx_gather`), read back by `mx_dequantize`, and multiplied with 4-bit
expert weights by `mx_gemm`. include/moe.h has the definitions; the argument checks and
the calls are compiled (csrc/operators_torch.cpp), the work is done by the kernels behind
the C ABI. Every call runs on the current stream of its tensors' device; nothing is
differentiable through autograd. Wrong tensors raise ValueError, wrong values what the
C ABI says (binding.MoEError).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import binding as B

B.lib()  # says so if the library has not been built
from . import _operators as _C  # noqa: E402

_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_ACT = {None: B.MOE_ACT_NONE, "none": B.MOE_ACT_NONE, **B.MOE_ACT}


class RouteConfig:
    """How tokens are routed: `score` "softmax" or "sigmoid"; with num_groups > 1 only the
    experts of the top_groups best groups (by the sum of their group_top highest keys);
    weights renormalised over the selection or not, times `scale`."""

    def __init__(self, num_experts: int, num_active: int, score: str = "softmax", num_groups: int = 1,
                 top_groups: int = 1, group_top: int = 2, renormalize: bool = True, scale: float = 1.0):
        if score not in B.MOE_SCORE:
            raise ValueError(f"unknown score {score!r}")
        self.num_experts, self.num_active = num_experts, num_active
        self._args = (num_experts, num_active, score, num_groups, top_groups, group_top, renormalize, scale)
        self.struct = B.MoeRouteConfig(num_experts, num_active, B.MOE_SCORE[score], num_groups, top_groups, group_top,
                                       int(renormalize), scale, B.MOE_DTYPE["fp32"])
        self._at = ctypes.addressof(self.struct)

    def __reduce__(self):  # a copy has a struct, and so an address, of its own
        return RouteConfig, self._args


def route(logits: torch.Tensor, cfg: RouteConfig, bias: Optional[torch.Tensor] = None, counts: bool = True,
          out=(None, None, None)) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Routes the tokens of logits [T][E] (bf16 or fp32). Returns (weights [T][k] fp32,
    topk_idx [T][k] int32, selections per expert [E] int32 or None); `out`: these
    three to write into, the last one None for no counts (`counts` says whether they are
    made where `out` is not given). bias [E] fp32 takes part in the selection only."""
    return _C.route(logits, cfg._at, bias, counts, *out)


def route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor, cfg: RouteConfig,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient with respect to logits, given that of route's weights [T][k] fp32. `out` may
    not overlap logits."""
    return _C.route_backward(grad_weights, logits, topk_idx, cfg._at, out)


def _format(fmt: str) -> int:
    if fmt not in B.MOE_MX:
        raise ValueError(f"unknown format {fmt!r}")
    return B.MOE_MX[fmt]


def _code_bytes(rows: int, cols: int) -> int:
    return rows * (cols // 2)


def _scale_bytes(fmt: str, rows: int, cols: int) -> int:
    tile_k = 4 * _BLOCK[fmt]
    return (rows + 127) // 128 * ((cols + tile_k - 1) // tile_k) * 512


class MxTensor:
    """Rows of microscaled 4-bit floating point: `groups` matrices of rows x cols ("mxfp4" or
    "nvfp4"), codes [groups * rows][cols / 2] and scale tiles as uint8 tensors on one device,
    and the power of two scale_exp that the values count in."""

    __slots__ = ("format", "codes", "scales", "rows", "cols", "groups", "scale_exp")

    def __init__(self, fmt: str, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int, groups: int = 1,
                 scale_exp: int = 0):
        _format(fmt)
        if cols < 32 or cols % 32:
            raise ValueError(f"a row needs a positive multiple of 32 elements, got {cols}")
        if rows < 0 or groups < 1:
            raise ValueError(f"{groups} groups of {rows} rows")
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


def _given(out: Optional[MxTensor], fmt: str, rows: int, cols: int, scale_exp: int, like: torch.Tensor):
    if out is None:
        return None, None
    if (out.format, out.rows, out.cols, out.groups, out.scale_exp) != (fmt, rows, cols, 1, scale_exp) or \
            out.codes.device != like.device:
        raise ValueError("out has another format, size, exponent or device")
    return out.codes, out.scales


def mx_quantize(x: torch.Tensor, fmt: str = "mxfp4", row_index: Optional[torch.Tensor] = None, scale_exp: int = 0,
                values: Optional[torch.Tensor] = None, out: Optional[MxTensor] = None) -> MxTensor:
    """Rows of x (bf16 or fp32) to 4 bits. row_index [rows] int32: output row r is x's row
    row_index[r], and is left as it was where that is no row of x. `values`, in x's type,
    receives what the codes stand for; `out`: an MxTensor to write into."""
    f = _format(fmt)
    codes = scales = None
    if out is not None:
        codes, scales = _given(out, fmt, x.shape[0] if row_index is None else row_index.numel(), x.shape[1], scale_exp, x)
    q = MxTensor.__new__(MxTensor)
    codes, scales, rows, cols = _C.quantize(x, f, row_index, scale_exp, values, codes, scales)
    q._set(fmt, codes, scales, rows, cols, 1, scale_exp)
    return q if out is None else out


def mx_gather(q: MxTensor, row_index: torch.Tensor, out: Optional[MxTensor] = None) -> MxTensor:
    """Rows row_index [rows] (int32) of q; a row is left as it was in `out` where row_index is
    no row of q."""
    if q.groups != 1:
        raise ValueError("one group at a time")
    rows = row_index.numel()
    codes, scales = _given(out, q.format, rows, q.cols, q.scale_exp, q.codes)
    codes, scales = _C.gather(q.codes, q.scales, B.MOE_MX[q.format], q.rows, q.cols, row_index, codes, scales)
    return out if out is not None else MxTensor(q.format, codes, scales, rows, q.cols, scale_exp=q.scale_exp)


def mx_dequantize(q: MxTensor, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values of q, [rows][cols] (one group)."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"bf16 or fp32, got {dtype}")
    if q.groups != 1:
        raise ValueError("one group at a time")
    out = torch.empty(q.rows, q.cols, dtype=dtype, device=q.codes.device)
    _C.dequantize(q.codes, q.scales, B.MOE_MX[q.format], q.rows, q.cols, q.scale_exp, out)
    return out


def mx_gemm(a: MxTensor, w: MxTensor, group_start: Optional[torch.Tensor] = None,
            group_rows: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
            alpha: Optional[torch.Tensor] = None, activation: Optional[str] = None, out: Optional[torch.Tensor] = None,
            dtype: torch.dtype = torch.bfloat16, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act(alpha_g a w_g^T + bias_g) for the rows of every group g: rows group_start[g] ..
    + group_rows[g] of a (int32, starts multiples of 128), or all rows with one group and
    neither given. Rows of no group are left as they were in `out`, or hold anything where
    `out` is not given. status: an int32 tensor of one zero, whose bit 0 reports a wait that
    gave up and bit 1 a segment outside the rows; without it `mx_status` tells of both."""
    if a.format != w.format or a.cols != w.cols:
        raise ValueError(f"operands differ: {a.format} of {a.cols} columns, {w.format} of {w.cols}")
    if a.groups != 1:
        raise ValueError("a has one group of rows")
    if activation not in _ACT:
        raise ValueError(f"unknown activation {activation!r}")
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"bf16 or fp32, got {dtype}")
    return _C.gemm(a.codes, a.scales, w.codes, w.scales, B.MOE_MX[a.format], a.rows, w.rows, a.cols, w.groups,
                   a.scale_exp + w.scale_exp, group_start, group_rows, bias, alpha, _ACT[activation], out,
                   dtype is torch.float32, status)


def mx_status(device=None) -> None:
    """Waits for the current stream of `device` (the current one) and raises MoEError if a product on it that
    had no `status` gave up a wait (its output is incomplete) or skipped a segment outside its rows. Each
    report comes once. Not while a graph is captured."""
    with torch.cuda.device(device):
        B.moe_mx_status(torch.cuda.current_stream().cuda_stream)
