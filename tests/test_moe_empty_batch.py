"""The dispatch calls and the MoE layer without any token, as a rank or a
micro-batch can have it."""
import importlib.util
import os

import pytest
import torch

import fp4_gemm_moe_amd as hq
from tests import _gpu as U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


@pytest.mark.parametrize("T,rows", [(0, 0), (0, 3), (5, 20)])
def test_permute_passes_the_width_of_a_row(monkeypatch, T, rows):
    """The row's bytes come from the tensors' trailing shape, with or without rows."""
    class Library:
        def hq_moe_permute(self, stream, x, tokens, row_bytes, *rest):
            self.got = tokens, row_bytes
            return 0

    lib = Library()
    monkeypatch.setattr(hq, "load", lambda: lib)
    monkeypatch.setattr(hq, "_raw_stream", lambda t: 0)
    monkeypatch.setattr(hq, "_arg", lambda t, name, dtype, numel: 16)
    hq.hq_moe_permute(torch.zeros(T, 6, 8, dtype=BF16), torch.zeros(T, 4, dtype=torch.int32), None, None,
                      torch.zeros(rows, 6, 8, dtype=BF16))
    assert lib.got == (T, 96)


@pytest.mark.gpu
@pytest.mark.parametrize("align", [1, 128])
def test_dispatch_calls_without_tokens(align):
    U.banner(f"dispatch of no tokens, align {align}")
    T, topk, E, h = 0, 4, 8, 256
    row_map, row_pair, ends, counts = hq.moe_sort(torch.empty((T, topk), dtype=torch.int64, device="cuda"), E, align)
    assert row_map.shape == (0, topk) and row_pair.numel() == 0
    assert torch.all(ends == 0) and torch.all(counts == 0)
    x, rows = torch.empty((T, h), dtype=BF16, device="cuda"), torch.empty((0, h), dtype=BF16, device="cuda")
    q, sf = torch.empty((0, h), dtype=torch.uint8, device="cuda"), torch.empty((0, 2), device="cuda")
    w = torch.empty((T, topk), device="cuda")
    for pads in ((ends, counts), (None, None)):
        hq.hq_moe_permute(x, row_map, *pads, rows)
        hq.hq_moe_permute_block_quant(x, row_map, *pads, q, sf)
        hq.hq_moe_combine_backward(x, rows, row_map, w, *pads, rows, w)
    hq.hq_moe_combine(rows, row_map, w, x)
    hq.hq_moe_combine(rows, row_map, None, x)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_layer_without_tokens():
    """Forward gives no rows, backward no token gradients and zeros for the weights."""
    U.banner("moe layer of no tokens")
    spec = importlib.util.spec_from_file_location("moe_block_fp8", os.path.join(ROOT, "examples", "moe_block_fp8.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    E, h, m, topk = 4, 256, 128, 2
    layer = example.MoeBlockFp8(torch.randn(E, 2 * m, h, device="cuda").bfloat16(),
                                torch.randn(E, h, m, device="cuda").bfloat16())
    x, ids = torch.empty((0, h), dtype=BF16, device="cuda"), torch.empty((0, topk), dtype=torch.int64, device="cuda")
    w = torch.empty((0, topk), device="cuda")
    for train in (False, True):
        out, saved = layer.forward(x, ids, w, train)
        assert out.shape == (0, h)
    dx, dw, dw1, dw2 = layer.backward(out, saved)
    torch.cuda.synchronize()
    assert dx.shape == (0, h) and dw.shape == (0, topk)
    assert dw1.shape == (E, 2 * m, h) and torch.all(dw1 == 0)
    assert dw2.shape == (E, h, m) and torch.all(dw2 == 0)
