"""The network of examples/moe_half_lora.py: a frozen FP8 projection with low-rank
adapters and a MoE layer in 16 bits, forward and backward, against float32
autograd and under graph capture.

Bounds, relative in norm.  A rounding to 16 bits is off by at most u = 2^-8 of a
value (bf16; fp16 less).  out: gu, a, y and out itself are rounded, SwiGLU
amplifies by at most 1.4: 4.4 u.  dweights the same without out, and a product
with dout whose signs may cancel: the tokens' sums keep their norm within 2, 8 u.
dw2: dy and a rounded (a from a rounded gu): 3 u.  dh: dy, da, dgu (from a rounded
gu) and the rows of experts rounded, the derivative of SwiGLU amplifies three of
them by at most 1.4: 8 u.  dw1: the same without the last, 6 u.  h and dx hold an
E4M3 product: codes of the rows are off by at most 2^-4 of a value (the weight's
codes are the reference's), 2^-4 + 2 u; the transposed weight has codes of its
own in blocks with the same scales, so dx counts no more.  da, db: the inner
sums in FP32 and 16-bit operands as given, terms u / 4."""
import importlib.util
import os

import pytest
import torch

from tests import _gpu as U

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
UNIT = 2.0 ** -8
BOUND = {"out": 4.4 * UNIT, "dweights": 8 * UNIT, "dh": 8 * UNIT, "dw1": 6 * UNIT, "dw2": 3 * UNIT,
         "h": 2.0 ** -4 + 2 * UNIT, "dx": 2.0 ** -4 + 2 * UNIT, "da": UNIT / 4, "db": UNIT / 4}


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_half_lora", os.path.join(ROOT, "examples", "moe_half_lora.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk,adapters,rank", [
    (300, 512, 384, 8, 2, 3, 16), (65, 416, 160, 5, 5, 7, 8), (1, 256, 128, 4, 2, 1, 16), (1000, 1024, 768, 16, 4, 4, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_step(example, tokens, hidden, inter, experts, topk, adapters, rank, dtype):
    U.banner(f"half network T={tokens} h={hidden} i={inter} E={experts} top{topk} L={adapters} r={rank} {dtype}")
    err, _ = example.compare(tokens, hidden, inter, experts, topk, adapters, rank, dtype)
    for name, e in err.items():
        assert e <= BOUND[name], f"{name}: {e:.5f}"


def test_step_without_tokens(example):
    U.banner("half network of no tokens")
    layers, args = example.network(0, 256, 128, 4, 2, 3, 8)
    _, out, got = example.step(layers, *args, torch.empty_like(args[0]))
    torch.cuda.synchronize()
    assert out.shape == (0, 256) and got["dx"].shape == (0, 256)
    for name in ("dw1", "dw2", "da", "db"):
        assert torch.all(got[name] == 0), name


def test_step_replays_under_graph_capture(example):
    """Replays with eager work between them give the eager bits, also for new tokens,
    experts and adapters written into the captured buffers."""
    U.banner("half network graph")
    layers, (x, who, ids, weights) = example.network(200, 512, 256, 8, 2, 4, 16)
    dout = torch.randn_like(x)

    def once():
        h, out, got = example.step(layers, x, who, ids, weights, dout)
        return [h, out, *got.values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = once()
    for i in range(4):
        x.copy_(torch.randn_like(x))
        who.copy_(torch.randint(-1, 4, who.shape, device="cuda"))
        ids.copy_(torch.randint(-1, 8, ids.shape, device="cuda"))
        want = [v.clone() for v in once()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a, b), f"replay {i}"
