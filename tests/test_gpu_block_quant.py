"""Block-128 FP8 quantisation on the GPU against the oracle: codes and scales
bit-exact (a code is the nearest E4M3 value of one FP32 quotient)."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import block as B
from oracle import formats as F
from tests import _block as H
from tests import _gpu as U

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


def _same_codes(q, want, what):
    q = q.cpu().numpy()
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal((q & 0x7F) == 0x7F, nan), f"{what}: NaN codes"
    assert np.array_equal(q[~nan], want[~nan]), f"{what}: {(q[~nan] != want[~nan]).sum()} codes differ"


def _same_scales(sf, want, what):
    assert np.array_equal(sf.cpu().numpy(), want, equal_nan=True), f"{what}: scales"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("two_d,transpose", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("batch,m,k", [(1, 1, 32), (1, 5, 160), (3, 32, 96), (2, 160, 416), (1, 128, 128),
                                       (1, 257, 1056)])
def test_codes_and_scales(dtype, two_d, transpose, batch, m, k):
    if transpose:
        m = -(-m // 32) * 32
    what = f"quant {dtype} 2d={two_d} t={transpose} {batch}x{m}x{k}"
    U.banner(what)
    r = H.rng(what)
    t, x = H.halves(r, (batch, m, k), dtype)
    q, sf = hq.block_quantize(t.cuda(), two_d, transpose)
    torch.cuda.synchronize()
    for b in range(batch):
        wq, ws = B.quant(x[b].T if transpose else x[b], two_d)
        _same_codes(q[b], wq, what)
        _same_scales(sf[b], ws, what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("two_d,transpose", [(False, False), (True, False), (False, True), (True, True)])
def test_special_blocks(dtype, two_d, transpose):
    """Zero blocks of both signs, the smallest values, values at every scale of
    the type, infinities and NaN in a block, each beside ordinary blocks."""
    U.banner(f"special {dtype} 2d={two_d} t={transpose}")
    m, k = 256, 1024
    r = H.rng("special")
    x = r.standard_normal((m, k)).astype(np.float32)
    x[:128, :128] = 0.0
    x[:128:2, :128] = -0.0
    x[:128, 128:256] = 2.0 ** (-24 if dtype is torch.float16 else -133) * r.integers(0, 3, (128, 128))
    x[:128, 256:384] *= 2.0 ** (-14 if dtype is torch.float16 else -126)
    x[:128, 384:512] *= 2.0 ** (13 if dtype is torch.float16 else 124)
    x[3, 512] = np.inf
    x[5, 640] = -np.inf
    x[7, 768] = np.nan
    x[9, 896:900] = [np.nan, np.inf, -np.inf, 0.0]
    t = torch.from_numpy(x).to(dtype)
    x = t.float().numpy()
    q, sf = hq.block_quantize(t.cuda(), two_d, transpose)
    torch.cuda.synchronize()
    wq, ws = B.quant(x.T if transpose else x, two_d)
    _same_codes(q, wq, "special")
    _same_scales(sf, ws, "special")


@pytest.mark.parametrize("two_d", [False, True])
def test_every_bf16_value(two_d):
    """Every finite BF16 value in blocks that share its exponent range."""
    U.banner(f"all bf16 2d={two_d}")
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    v = F.bf16_decode(bits)
    bits = bits[np.isfinite(v)]
    bits = bits[np.argsort(np.abs(F.bf16_decode(bits)), kind="stable")]
    bits = np.resize(bits, 512 * 128).reshape(512, 128)
    if two_d:
        bits = np.ascontiguousarray(bits.reshape(4, 128, 128).swapaxes(0, 1).reshape(128, 512))
    t = U.dev_bf16(bits, "cuda")
    q, sf = hq.block_quantize(t, two_d)
    wq, ws = B.quant(t.float().cpu().numpy(), two_d)
    _same_codes(q, wq, "all bf16")
    _same_scales(sf, ws, "all bf16")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,h,last", [(1, 32, None), (37, 416, None), (64, 256, 41), (64, 256, 0), (64, 128, 99)])
def test_swiglu(dtype, rows, h, last):
    """y's FP32 form is off by at most |gate| 2^-23 (exp2 of a rounded product)
    plus a few roundings: below 2^-17 for |gate| < 40.  The scale is off by as
    much, and a code sits at most one step from the float64 one, rarely (the
    quotient has to lie within 2^-16 of a midpoint).  Rows past the last end
    keep their contents."""
    what = f"swiglu {dtype} {rows}x{h} last={last}"
    U.banner(what)
    t, x = H.halves(H.rng(what), (rows, 2 * h), dtype)
    q = torch.full((rows, h), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((rows, -(-h // 128)), -7.0, device="cuda")
    ends = None if last is None else torch.tensor([min(3, last), last], dtype=torch.int32, device="cuda")
    hq.hq_fused_swiglu_block_quant(t.cuda(), q, sf, ends)
    torch.cuda.synchronize()
    n = rows if last is None else min(rows, last)
    y = B.swiglu(x, h)[:n]
    wq, ws = B.quant(y.astype(np.float32)) if n else (np.empty((0, h), np.uint8), np.empty((0, sf.shape[1])))
    assert np.all(np.abs(sf[:n].cpu().numpy() - ws) <= 2.0 ** -17 * np.abs(ws)), what
    got, want = F.e4m3_decode(q[:n].cpu().numpy()), F.e4m3_decode(wq)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -6))) - 3)
    off = np.abs(got - want)
    assert np.all(off <= step * (1 + 1e-9)), what
    assert n == 0 or np.mean(off > 0) <= 1e-2, what
    assert torch.all(q[n:] == 0xA5) and torch.all(sf[n:] == -7.0), f"{what}: rows past the last end written"
