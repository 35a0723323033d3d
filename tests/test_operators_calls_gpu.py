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


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_the_bindings_calls_are_the_operators(fmt):
    """The ctypes functions on raw addresses, with the results that the tensors' functions have."""
    g = gen(3)
    f, s = B.MOE_MX[fmt], torch.cuda.current_stream().cuda_stream
    logits = torch.randn(50, 40, generator=g, device="cuda")
    cfg = ops.RouteConfig(40, 4, "sigmoid", 4, 2)
    want = ops.route(logits, cfg)
    w, idx, n = (torch.empty_like(t) for t in want)
    B.moe_route(cfg.struct, logits.data_ptr(), 40, 50, None, w.data_ptr(), idx.data_ptr(), n.data_ptr(), s)
    assert all(torch.equal(a, b) for a, b in zip((w, idx, n), want))
    d = torch.empty_like(logits)
    B.moe_route_backward(cfg.struct, w.data_ptr(), logits.data_ptr(), 40, idx.data_ptr(), 50, d.data_ptr(), 40, s)
    assert torch.equal(d, ops.route_backward(w, logits, idx, cfg))

    x, v = torch.randn(30, 96, generator=g, device="cuda"), torch.randn(20, 96, generator=g, device="cuda")
    a, wq = ops.mx_quantize(x, fmt), ops.mx_quantize(v, fmt)
    index = torch.randint(0, 30, (70,), generator=g, device="cuda", dtype=torch.int32)
    codes = torch.zeros(70, 48, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(B.moe_mx_scales_bytes(f, 70, 96), dtype=torch.uint8, device="cuda")
    B.moe_mx_gather(f, a.codes.data_ptr(), a.scales.data_ptr(), 30, 96, index.data_ptr(), 70, codes.data_ptr(),
                    scales.data_ptr(), s)
    q = ops.MxTensor(fmt, codes, scales, 70, 96)
    assert torch.equal(codes, ops.mx_gather(a, index).codes)
    val = torch.empty(70, 96, device="cuda")
    B.moe_mx_dequantize(f, codes.data_ptr(), scales.data_ptr(), 70, 96, 0, val.data_ptr(), B.MOE_DTYPE["fp32"], 96, s)
    assert torch.equal(val, ops.mx_dequantize(a)[index.long()])
    out = torch.empty(70, 20, device="cuda")
    B.moe_mx_gemm(B.MoeMxGemm(format=f, rows=70, n=20, k=96, groups=1, scale_exp=0, activation=B.MOE_ACT["gelu"],
                              out_dtype=B.MOE_DTYPE["fp32"], out_ld=20, a_codes=codes.data_ptr(), a_scales=scales.data_ptr(),
                              w_codes=wq.codes.data_ptr(), w_scales=wq.scales.data_ptr(), out=out.data_ptr()), s)
    assert torch.equal(out, ops.mx_gemm(q, wq, activation="gelu", dtype=torch.float32))
    B.moe_mx_status(s)


def test_calls_on_two_streams_at_once():
    """Products of every form, quantisation with its workspace and routing, queued on two streams without waiting
    for one another: each gives what it gives alone."""
    g = gen(4)
    cfg = ops.RouteConfig(256, 8, "sigmoid", 8, 4)
    work = []
    for fmt, rows, N, K, G in (("mxfp4", 2048, 512, 4096, 2), ("nvfp4", 2048, 512, 1024, 4), ("mxfp4", 1024, 640, 2048, 8)):
        x = torch.randn(700, K, generator=g, device="cuda").bfloat16()
        parts = [ops.mx_quantize(torch.randn(N, K, generator=g, device="cuda"), fmt) for _ in range(G)]
        w = ops.MxTensor(fmt, torch.stack([p.codes for p in parts]), torch.stack([p.scales for p in parts]), N, K, groups=G)
        index = torch.randint(0, 700, (rows * 2,), generator=g, device="cuda", dtype=torch.int32)
        start = (torch.arange(G, device="cuda") * (rows // G)).to(torch.int32)
        count = torch.full((G,), 9 if rows == 1024 else rows // G, dtype=torch.int32, device="cuda")
        logits = torch.randn(500, 256, generator=g, device="cuda")
        work.append((fmt, x, index, w, start, count, logits))

    def step(i):
        fmt, x, index, w, start, count, logits = work[i % len(work)]
        q = ops.mx_quantize(x, fmt, row_index=index)
        y = ops.mx_gemm(q, w, start, count, out=torch.zeros(index.numel(), w.rows, dtype=torch.bfloat16, device="cuda"))
        wts, idx, n = ops.route(logits, cfg)
        return y, wts, idx, n, ops.route_backward(wts, logits, idx, cfg)

    want = [step(i) for i in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(30):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i + j, step(i + j)))
    torch.cuda.synchronize()
    for i, outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i % 3]))
    ops.mx_status()
