"""Helpers of the tests of 16-bit products, SwiGLU and low-rank adapters."""
import numpy as np
import torch

from tests import _block as H

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
#: Written around and into outputs before a call.
MARK = 776.0          # exact in every type


def marked(shape, dtype):
    """(whole, view): a view of this shape inside a tensor of marks."""
    numel = int(np.prod(shape))
    whole = torch.full((numel + 256,), MARK, dtype=dtype, device="cuda")
    return whole, whole[128:128 + numel].view(shape)


def untouched(whole, what):
    assert torch.all(whole[:128] == MARK) and torch.all(whole[-128:] == MARK), f"{what}: written around the output"


def product_bound(ref, mag, terms, dtype):
    """An FP32 sum of `terms` exact products: each step rounds or truncates a
    partial sum, which the sum of magnitudes bounds, by 2^-23 of it at most; then
    one rounding to the output type."""
    return (terms + 2) * 2.0 ** -23 * mag + H.UNIT[dtype] * np.abs(ref) + H.FLOOR[dtype]


def f64(t):
    return t.detach().cpu().double().numpy()


def halves(r, shape, dtype, sigma=1.0):
    """(device tensor, float64 values)"""
    t, _ = H.halves(r, shape, dtype, sigma)
    return t.to("cuda"), t.double().numpy()
