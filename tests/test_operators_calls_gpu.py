"""Calls of the layer-free operators that are allowed and out of the ordinary (GPU)."""
import pytest
import torch

from sparse_mixture_experts_gate_b200 import binding as B
from sparse_mixture_experts_gate_b200 import operators as ops
from sparse_mixture_experts_gate_b200.binding import MoEError

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_skipped_segments_are_told_of_without_a_status_word():
    """Once each, on whatever stream the product ran, and not where the caller has a word of their own."""
    g = gen(1)
    a = ops.mx_quantize(torch.randn(256, 128, generator=g, device="cuda"))
    w = ops.mx_quantize(torch.randn(64, 128, generator=g, device="cuda"))
    good = torch.tensor([[128], [20]], dtype=torch.int32, device="cuda")
    bad = torch.tensor([[128], [129]], dtype=torch.int32, device="cuda")
    ops.mx_status()
    out = ops.mx_gemm(a, w, good[0], good[1])
    ops.mx_status("cuda:0")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.mx_gemm(a, w, bad[0], bad[1], status=st)
    ops.mx_status()
    assert st.item() == 2
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = ops.mx_gemm(a, w, good[0], good[1])
        ops.mx_gemm(a, w, bad[0], bad[1])
        with pytest.raises(MoEError) as e:
            ops.mx_status()
    assert e.value.code == B.MOE_ERR_INVALID_ARG
    ops.mx_status()
    assert torch.equal(again[128:148], out[128:148])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.mx_gemm(a, w, bad[0], bad[1])
    ops.mx_status()
    for _ in range(2):
        graph.replay()
        with pytest.raises(MoEError):
            ops.mx_status()
    ops.mx_status()


@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_beside_its_logits(renormalize):
    """Columns of one buffer, and rows that lie between the logits' rows, do not overlap; the logits themselves do."""
    g = gen(2)
    cfg = ops.RouteConfig(24, 3, renormalize=renormalize)
    buf = torch.randn(40, 48, generator=g, device="cuda")
    logits, plain = buf[:, :24], buf[:, :24].clone()
    _, idx, _ = ops.route(plain, cfg)
    gw = torch.randn(40, 3, generator=g, device="cuda")
    want = ops.route_backward(gw, plain, idx, cfg)
    assert torch.equal(ops.route_backward(gw, logits, idx, cfg, out=buf[:, 24:]), want)
    assert torch.equal(logits, plain)
    last = ops.route_backward(gw[39:], logits[39:], idx[39:], cfg, out=buf[38:39, :24])
    assert torch.equal(last, want[39:])
    with pytest.raises(MoEError, match="overlap"):
        ops.route_backward(gw, plain, idx, cfg, out=plain)
