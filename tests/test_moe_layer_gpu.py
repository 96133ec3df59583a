"""The mixture-of-experts example: its operators together, against the layer in fp32.
E4M3 rounds a value by at most 2^-4 relative, uniformly spread: 2^-4 / sqrt(3) / 2 =
0.018 rms for the activations of each product (the weights are the same on both sides),
two products in a row and the gate's square root of two between them: 0.018 * sqrt(1 +
2 + 1) = 0.036; twice that is accepted."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,hidden,inner,experts,top", [(1, 256, 128, 8, 2), (33, 512, 272, 16, 4),
                                                             (700, 1040, 400, 8, 3)])
def test_layer(moe, tokens, hidden, inner, experts, top):
    layer = moe.MoeLayer(hidden, inner, experts, top, seed=tokens)
    x = torch.randn(tokens, hidden, generator=torch.Generator(device="cuda").manual_seed(2),
                    device="cuda").to(torch.bfloat16)
    out, ref = layer.forward(x).float(), layer.reference(x)
    assert moe.bs.fp8_status_query() == 0
    assert float((out - ref).norm() / ref.norm()) < 0.072


def test_layer_replays_in_a_graph(moe):
    """One capture serves other tokens: the routing is read on the device."""
    layer = moe.MoeLayer(256, 128, 8, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(20, 256, generator=g, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(x)
    for _ in range(2):
        x.copy_(torch.randn(20, 256, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer.forward(x))
    del graph
