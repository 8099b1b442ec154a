"""The block-128 FP8 MoE layer of examples/moe_block_fp8.py against float32
autograd, and its forward under graph capture.

Bounds: an E4M3 code is off by at most 2^-4 of its value, 2.6 % rms.  Each
quantised tensor on the way to a result adds its error in quadrature; SwiGLU and
its derivative amplify what lies before them by up to 1.4.  out: four tensors
(x, w1, a, w2), up to 6 %, dweights the same; dx: seven, up to 10 %; dw2: x,
w1, a, dy, up to 7 %; dw1: seven, up to 10 %.  The bounds are twice that."""
import importlib.util
import os

import pytest
import torch

import fp4_gemm_moe_amd as hq
from tests import _gpu as U

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUND = {"out": 0.12, "decode": 0.12, "dweights": 0.12, "dx": 0.20, "dw1": 0.20, "dw2": 0.14}


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block_fp8", os.path.join(ROOT, "examples", "moe_block_fp8.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", [(300, 512, 384, 8, 2), (65, 416, 160, 5, 5),
                                                              (1, 256, 128, 4, 2), (1000, 1024, 768, 16, 4)])
def test_layer_and_gradients(example, tokens, hidden, inter, experts, topk):
    U.banner(f"moe layer T={tokens} h={hidden} i={inter} E={experts} top{topk}")
    err, _ = example.compare(tokens, hidden, inter, experts, topk)
    for name, e in err.items():
        assert e <= BOUND[name], f"{name}: {e:.3f}"


def test_forward_replays_under_graph_capture(example):
    """Every call of the path captured: replays with eager work between them give
    the eager bits, also for new inputs written into the captured buffers."""
    U.banner("moe layer graph")
    torch.manual_seed(3)
    T, h, m, E, k = 200, 512, 256, 8, 2
    layer = example.MoeBlockFp8(torch.randn(E, 2 * m, h, device="cuda").mul_(0.05).bfloat16(),
                                torch.randn(E, h, m, device="cuda").mul_(0.05).bfloat16())
    x, ids = torch.randn(T, h, device="cuda").bfloat16(), torch.randint(0, E, (T, k), device="cuda")
    w = torch.rand(T, k, device="cuda")
    bufs = {}

    def once():
        # the dense product with its K split, a batch of quantised weights, the whole layer
        out, saved = layer.forward(x, ids, w)
        dy, dw = torch.empty_like(saved[6]), torch.empty_like(w)
        hq.hq_moe_combine_backward(out, saved[6], saved[2], w, saved[3], saved[4], dy, dw)
        q, s = hq.block_quantize(x, transpose=False)
        dense = torch.empty(T, 2 * m, device="cuda")
        hq.hq_block_gemm(q, s, layer.w1[0][0], layer.w1[1][0], dense, workspace=bufs["ws"])
        return out, dw, dense

    bufs["ws"] = torch.empty(hq.HQ_BLOCK_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = once()
    for i in range(4):
        x.copy_(torch.randn(T, h, device="cuda"))
        ids.copy_(torch.randint(-1, E, (T, k), device="cuda"))
        want = [v.clone() for v in once()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a, b), f"replay {i}"
