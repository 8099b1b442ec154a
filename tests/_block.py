"""Helpers of the block-128 FP8 and token-dispatch tests: inputs, transfers and
the error bounds (derived from the formats' precisions)."""
import zlib

import numpy as np
import torch

from oracle import block as B

#: Unit roundoff of each 16- and 32-bit type (half the spacing at 1).
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
#: Half the spacing of the type's smallest values.
FLOOR = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def rng(*key):
    """A generator of its own for each key (the same in every run)."""
    return np.random.default_rng(zlib.crc32(repr(key).encode()))


def halves(r, shape, dtype, sigma=1.0):
    """Normal values of a 16-bit type with a few large columns: (tensor, float32 array)."""
    x = (sigma * r.standard_normal(shape)).astype(np.float32)
    x[..., ::37] *= 8.0
    t = torch.from_numpy(x).to(dtype)
    return t, t.float().numpy()


def codes(r, m, k, two_d=False, sigma=1.0):
    """Quantised operand (codes, scales) of normal values."""
    return B.quant((sigma * r.standard_normal((m, k))).astype(np.float32), two_d)


def dev(x, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device)


def product_bound(ref, mag, k, dtype):
    """A block product's error: each K block's 128 products summed in FP32 (at
    most 128 roundings or truncations of 2^-23), its scale and its place in the
    sum over blocks (nkb + 4), relative to the sum of magnitudes; then the one
    rounding to the output type."""
    return (132 + -(-k // 128)) * 2.0 ** -23 * mag + UNIT[dtype] * np.abs(ref) + FLOOR[dtype]


def sum_bound(ref, mag, terms, dtype):
    """An FP32 sum of `terms` products, then one rounding to the output type."""
    return (terms + 2) * 2.0 ** -24 * mag + UNIT[dtype] * np.abs(ref) + FLOOR[dtype]


def check(out, ref, bound, what):
    out = out.detach().cpu().double().numpy() if isinstance(out, torch.Tensor) else np.asarray(out, np.float64)
    assert out.shape == ref.shape, what
    err = np.abs(out - ref)
    # the bound's own FP32 rounding of |ref|-sized terms is second order
    bad = ~(err <= bound * (1 + 2.0 ** -7))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bound, worst {np.nanmax(err / bound):.3g} of it"
