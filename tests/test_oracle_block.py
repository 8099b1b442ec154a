"""The block-128 and dispatch oracle pinned against definitions it does not
share: torch's E4M3 cast, exact rationals, hand-worked maps, sums by loop."""
from fractions import Fraction as Fr

import numpy as np
import torch

from oracle import block as B
from oracle import formats as F
from tests import _block as H
from tests import _exact as X


def test_quant_by_exact_rationals():
    r = np.random.default_rng(0)
    x = (r.standard_normal((3, 130)) * 2.0 ** r.integers(-6, 6, (3, 130))).astype(np.float32)
    q, sf = B.quant(x)
    for i in range(3):
        for j in range(2):
            blk = [Fr(float(v)) for v in x[i, j * 128:(j + 1) * 128]]
            s = X.fp32_round(max(abs(v) for v in blk) / 448)
            assert Fr(float(sf[i, j])) == s
            for c, v in zip(q[i, j * 128:(j + 1) * 128], blk):
                assert (c & 0x7F) == X.nearest_code(X.fp32_round(v / s), X.E4M3)
                assert bool(c & 0x80) == (v < 0)


def test_quant_by_torch_cast():
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((256, 384)).astype(np.float32))
    for two_d in (False, True):
        bm = 128 if two_d else 1
        v = x.reshape(256 // bm, bm, 3, 128)
        s = v.abs().amax((1, 3)) / 448
        q = (v / s[:, None, :, None]).to(torch.float8_e4m3fn).reshape(256, 384).view(torch.uint8)
        oq, os_ = B.quant(x.numpy(), two_d)
        assert np.array_equal(oq, q.numpy()) and np.array_equal(os_, s.numpy())


def test_quant_special_blocks():
    x = np.zeros((1, 512), np.float32)
    x[0, 1], x[0, 130], x[0, 131], x[0, 260], x[0, 384] = -0.0, np.inf, 5.0, np.nan, 2.0 ** -140
    q, sf = B.quant(x)
    assert sf[0, 0] == 2.0 ** -126 and q[0, 0] == 0 and q[0, 1] == 0x80
    assert np.isinf(sf[0, 1]) and q[0, 131] == 0 and (q[0, 130] & 0x7F) == 0x7F
    assert np.isnan(sf[0, 2]) and np.all((q[0, 256:384] & 0x7F) == 0x7F)
    assert sf[0, 3] == 2.0 ** -126 and q[0, 384] == 0


def test_product_by_loops():
    r = np.random.default_rng(2)
    a, sa = B.quant(r.standard_normal((3, 160)).astype(np.float32))
    b, sb = B.quant(r.standard_normal((136, 160)).astype(np.float32), True)
    ref, _ = B.gemm(a, sa, b, sb)
    for m in range(3):
        for n in (0, 127, 128, 135):
            want = sum(float(sa[m, kb]) * float(sb[n // 128, kb])
                       * sum(float(F.e4m3_decode(a[m, k])) * float(F.e4m3_decode(b[n, k]))
                             for k in range(kb * 128, min(160, kb * 128 + 128))) for kb in range(2))
            assert abs(ref[m, n] - want) <= 1e-12 * max(1.0, abs(want))


def test_sort_by_hand():
    ids = np.array([[2, 0], [0, -1], [2, 2], [7, 0]])
    row_map, row_pair, ends, counts = B.sort(ids, 3, 4, 10)
    assert counts.tolist() == [3, 0, 3] and ends.tolist() == [4, 4, 8]
    assert row_map.tolist() == [[4, 0], [1, -1], [5, 6], [-1, 2]]
    assert row_pair.tolist() == [1, 2, 7, -1, 0, 4, 5, -1, -1, -1]


def test_combine_gradient_by_autograd():
    r = np.random.default_rng(3)
    ids = r.integers(-1, 5, (12, 3))
    m, _, _, _ = B.sort(ids, 5, 1, 36)
    y = torch.from_numpy(r.standard_normal((36, 7))).requires_grad_()
    w = torch.from_numpy(r.random((12, 3))).requires_grad_()
    d = r.standard_normal((12, 7))
    on = torch.from_numpy(m >= 0)
    out = (y[torch.from_numpy(np.maximum(m, 0)).long()] * (w * on)[..., None]).sum(1)
    assert np.allclose(out.detach().numpy(), B.combine(y.detach().numpy(), m, w.detach().numpy())[0], atol=1e-12)
    out.backward(torch.from_numpy(d))
    dy, dw, _ = B.combine_backward(d, y.detach().numpy(), m, w.detach().numpy())
    assert np.allclose(dy, y.grad.numpy(), atol=1e-12) and np.allclose(dw, w.grad.numpy(), atol=1e-12)


def test_the_bounds_catch_a_wrong_element():
    """A planted mistake -- one K block's scale taken from its neighbour, one row
    from another token -- lies outside the bounds; rounding to the type does not."""
    r = np.random.default_rng(4)
    a, sa = B.quant(r.standard_normal((20, 512)).astype(np.float32))
    b, sb = B.quant(r.standard_normal((130, 512)).astype(np.float32), True)
    ref, mag = B.gemm(a, sa, b, sb)
    bound = H.product_bound(ref, mag, 512, torch.bfloat16)
    H.check(torch.from_numpy(ref).bfloat16(), ref, bound, "rounded")
    wrong = sa.copy()
    wrong[7, 1] = sa[7, 2] * np.float32(1.2)
    off = np.abs(B.gemm(a, wrong, b, sb)[0] - ref)
    assert (off[7] > bound[7]).any()
    y = r.standard_normal((6, 64))
    m = np.array([[0, 1], [2, 3]], np.int32)
    ref, mag = B.combine(y, m)
    off = np.abs(B.combine(y, np.array([[0, 4], [2, 3]], np.int32))[0] - ref)
    assert (off[0] > H.sum_bound(ref, mag, 2, torch.bfloat16)[0]).any()
