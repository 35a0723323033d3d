"""4-bit experts prepared on a stream of their own (GPU): their memory is not another stream's.

`torch.cuda._sleep` keeps a stream busy for a while, so that what is queued behind it comes late.
"""
import pytest
import torch

from sparse_mixture_experts_gate_b200 import binding
from sparse_mixture_experts_gate_b200.binding import MoELayer
from sparse_mixture_experts_gate_b200.workloads import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu

LATE = 400_000_000  # clock cycles: about 0.2 s


def layer_of(T=200):
    w = WORKLOADS["default"].with_(T=T)
    inp = make_inputs(w, "cpu", seed=8)
    # Kernels that are loaded by their first launch would have the host wait for what is queued.
    torch.full((16,), 0xFF, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda._sleep(1)
    return MoELayer(w, inp), inp["x"].cuda()


def test_memory_the_current_stream_still_writes_is_not_taken():
    layer, x = layer_of()
    layer.prepare_experts_mx("mxfp4")
    want = layer.forward(x)["y"].clone()
    n = binding.moe_experts_mx_bytes(layer.handle, 0)
    layer.prepare_experts_mx(None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    out = layer.alloc_outputs(x.shape[0])
    layer.workspace(x.shape[0])
    t = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(LATE)
    t.fill_(0xFF)
    del t  # the current stream's to give out again, behind the write
    layer.prepare_experts_mx("mxfp4", stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(layer.forward(x, out=out)["y"], want)


@pytest.mark.parametrize("then", [None, "mxfp4"])
def test_a_forward_on_another_stream_keeps_its_weights(then):
    layer, x = layer_of()
    layer.prepare_experts_mx("mxfp4")
    want = layer.forward(x)["y"].clone()
    n = binding.moe_experts_mx_bytes(layer.handle, 0)
    out = layer.alloc_outputs(x.shape[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
    layer.forward(x, out=out, stream=side.cuda_stream)
    layer.prepare_experts_mx(then)
    t = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out["y"], want) and len(t) == 3


def test_weights_quantised_in_a_captured_graph():
    """A graph that quantises the weights and runs a forward, replayed on other weights; earlier weights stay."""
    layer, x = layer_of()
    layer.prepare_experts_mx("nvfp4")
    first = layer.forward(x)["y"].clone()
    out = layer.alloc_outputs(x.shape[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.prepare_experts_mx("nvfp4")
        layer.forward(x, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["y"], first)
    layer.weights["w1"].mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = out["y"].clone()
    layer.prepare_experts_mx("nvfp4")
    assert torch.equal(layer.forward(x)["y"], got) and not torch.equal(got, first)
