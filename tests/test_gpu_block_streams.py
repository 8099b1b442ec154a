"""Quantisation, SwiGLU with quantisation and the combination's gradient on the
GPU at sizes whose outputs are stored past the caches (more than 128 MB), with
partial tiles at the ends: samples against the oracle, and no other output
written."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import block as B
from oracle import formats as F
from tests import _block as H
from tests import _gpu as U

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
LIMIT = 128 << 20


def _halves(what, shape, dtype, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(int(H.rng(what).integers(0, 2 ** 62)))
    return (sigma * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def _marked(numel, dtype, value):
    whole = torch.full((numel + 256,), value, dtype=dtype, device="cuda")
    return whole, whole[128:128 + numel]


def _untouched(whole, value, what):
    assert torch.all(whole[:128] == value) and torch.all(whole[-128:] == value), f"{what}: written around the output"


@pytest.mark.parametrize("two_d,transpose,batch,m,k", [
    (False, False, 1, 32777, 4128), (True, False, 3, 10921, 4128), (False, True, 1, 32800, 4128),
    (True, True, 3, 10944, 4128)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_quant(two_d, transpose, batch, m, k, dtype):
    """Sampled strips of tiles at both ends and between, bit for bit; every code
    and scale written."""
    what = f"large quant 2d={two_d} t={transpose} {batch}x{m}x{k} {dtype}"
    U.banner(what)
    assert batch * m * k > LIMIT
    x = _halves(what, (batch, m, k), dtype)
    x[:, 5, 7] = 0.0
    rows, cols = (k, m) if transpose else (m, k)
    wq, q = _marked(batch * m * k, torch.uint8, 0x7F)          # a NaN code, which finite values never take
    q = q.view(batch, rows, cols)
    ws, sf = _marked(batch * (-(-rows // 128) if two_d else rows) * -(-cols // 128), torch.float32, -7.0)
    sf = sf.view(batch, -1, -(-cols // 128))
    hq.hq_block_quant(x, q, sf, two_d, transpose)
    torch.cuda.synchronize()
    assert not torch.any(q == 0x7F) and not torch.any(sf == -7.0), f"{what}: outputs missing"
    _untouched(wq, 0x7F, what)
    _untouched(ws, -7.0, what)
    for b in {0, batch - 1}:
        for t in (0, rows // 256, (rows - 1) // 128):
            r = slice(128 * t, min(128 * t + 128, rows))
            for c in (slice(0, 256), slice(cols // 256 * 128, cols // 256 * 128 + 256), slice((cols - 1) // 128 * 128, cols)):
                part = (x[b].t() if transpose else x[b])[r, c].float().cpu().numpy()
                want, scales = B.quant(part, two_d)
                at = slice(t, t + 1) if two_d else r
                blocks = slice(c.start // 128, c.start // 128 + scales.shape[1])
                assert np.array_equal(q[b, r, c].cpu().numpy(), want), f"{what}: codes of rows {r}"
                assert np.array_equal(sf[b, at, blocks].cpu().numpy(), scales), f"{what}: scales of rows {r}"


def test_swiglu():
    """As test_gpu_block_quant.test_swiglu bounds it, on sampled rows."""
    rows, h = 32777, 4128
    what = f"large swiglu {rows}x{h}"
    U.banner(what)
    x = _halves(what, (rows, 2 * h), BF16)
    wq, q = _marked(rows * h, torch.uint8, 0x7F)
    ws, sf = _marked(rows * -(-h // 128), torch.float32, -7.0)
    q, sf = q.view(rows, h), sf.view(rows, -1)
    hq.hq_fused_swiglu_block_quant(x, q, sf)
    torch.cuda.synchronize()
    assert not torch.any(q == 0x7F) and not torch.any(sf == -7.0)
    _untouched(wq, 0x7F, what)
    _untouched(ws, -7.0, what)
    at = torch.tensor([0, 1, 63, 4096, 16385, rows - 2, rows - 1], device="cuda")
    want, scales = B.quant(B.swiglu(x[at].float().cpu().numpy(), h).astype(np.float32))
    assert np.all(np.abs(sf[at].cpu().numpy() - scales) <= 2.0 ** -17 * np.abs(scales))
    got, want = F.e4m3_decode(q[at].cpu().numpy()), F.e4m3_decode(want)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -6))) - 3)
    off = np.abs(got - want)
    assert np.all(off <= step * (1 + 1e-9)) and np.mean(off > 0) <= 1e-2


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_combine_backward(dtype):
    """Whole gradients against float64 on the GPU, a few tokens against the oracle;
    padding rows are zeros, rows past the last end left alone."""
    T, topk, E, h = 4111, 4, 16, 4104
    what = f"large combine backward {T} top {topk} h={h} {dtype}"
    U.banner(what)
    r = H.rng(what)
    ids = H.dev(np.where(r.random((T, topk)) < 0.02, -1, r.integers(0, E, (T, topk))))
    row_map, row_pair, ends, counts = hq.moe_sort(ids, E, 128)
    rows = row_pair.numel()
    assert rows * h * 2 > LIMIT
    y, dout = _halves(what, (rows, h), dtype), _halves(what + " out", (T, h), dtype, 0.1)
    w = H.dev(r.random((T, topk)).astype(np.float32))
    whole, dy = _marked(rows * h, dtype, 9.0)
    dy = dy.view(rows, h)
    dw = torch.full((T, topk), 9.0, device="cuda")
    hq.hq_moe_combine_backward(dout, y, row_map, w, ends, counts, dy, dw)
    torch.cuda.synchronize()
    _untouched(whole, 9.0, what)
    last = int(ends[-1])
    assert torch.all(dy[last:] == 9.0)
    pair = row_pair[:last].long()
    on = pair >= 0
    ref = w.double().view(-1)[pair.clamp(min=0), None] * dout.double()[pair.clamp(min=0) // topk] * on[:, None]
    bound = 3 * 2.0 ** -24 * ref.abs() + H.UNIT[dtype] * ref.abs() + H.FLOOR[dtype]
    assert torch.all((dy[:last].double() - ref).abs() <= bound * (1 + 2.0 ** -7)), f"{what}: dy"
    assert torch.all(dw[row_map < 0] == 0)
    t = np.unique(np.concatenate([r.integers(0, T, 20), [0, T - 1]]))
    c = lambda v: v.cpu().numpy()  # noqa: E731
    m = c(row_map[H.dev(t)])
    _, rdw, mag = B.combine_backward(c(dout[H.dev(t)].float()), c(y.float()), m, c(w[H.dev(t)]))
    H.check(dw[H.dev(t)], rdw, H.sum_bound(rdw, mag, h, torch.float32), f"{what}: dweights")
