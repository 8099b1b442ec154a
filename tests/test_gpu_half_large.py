"""The 16-bit operators where elements lie past 2^31 and bytes past 2^32: the last
rows, groups and tokens against float64."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from tests import _block as H
from tests import _gpu as U
from tests import _half as F

pytestmark = pytest.mark.gpu

BF16, F32 = F.BF16, F.F32


def _randn(*shape):
    return torch.empty(shape, dtype=BF16, device="cuda").normal_()


def _rows(m):
    return torch.tensor([0, 1, m // 2, m - 300, m - 2, m - 1], device="cuda")


@pytest.mark.parametrize("transpose", [False, True])
def test_contiguous_rows(transpose):
    U.banner(f"large contiguous t={transpose}")
    rows, n, k = 140000, 16392, 16
    a, b = _randn(rows, k), _randn(2, k, n) if transpose else _randn(2, n, k)
    out = torch.empty(rows, n, dtype=BF16, device="cuda")
    ends = torch.tensor([70001, rows], dtype=torch.int32, device="cuda")
    hq.hq_half_group_contiguous_gemm(a, b, ends, out, transpose=transpose)
    for t in _rows(rows).tolist():
        w = F.f64(b[int(t >= 70001)])
        w = w if transpose else w.T
        ref, mag = F.f64(a[t]) @ w, np.abs(F.f64(a[t])) @ np.abs(w)
        H.check(out[t], ref, F.product_bound(ref, mag, k, BF16), f"row {t}")


def test_wide_operands():
    """a, and each group's weights, of more than 2^31 bytes together."""
    U.banner("large operands")
    rows, n, k = 20000, 4104, 120000
    a, b = _randn(rows, k), _randn(3, n, k)
    out = torch.empty(rows, n, device="cuda")
    ends = torch.tensor([9000, 9000, rows], dtype=torch.int32, device="cuda")
    hq.hq_half_group_contiguous_gemm(a, b, ends, out)
    for t in (0, 8999, 9000, rows - 1):
        for c in (0, n - 1):
            x, w = F.f64(a[t]), F.f64(b[2 if t >= 9000 else 0, c])
            ref, mag = np.array([x @ w]), np.array([np.abs(x) @ np.abs(w)])
            H.check(out[t, c:c + 1], ref, F.product_bound(ref, mag, k, F32), f"row {t} column {c}")


def test_group_k():
    U.banner("large group k")
    rows, m, n = 300000, 8200, 16
    a, b = _randn(rows, m), _randn(rows, n)
    ends = torch.tensor([100, 299901, rows], dtype=torch.int32, device="cuda")
    out = torch.empty(3, m, n, device="cuda")
    hq.hq_half_group_k_gemm(a, b, ends, out)
    for g, lo, hi in ((0, 0, 100), (2, 299901, rows)):
        x, y = F.f64(a[lo:hi]), F.f64(b[lo:hi])
        ref, mag = x.T @ y, np.abs(x).T @ np.abs(y)
        H.check(out[g], ref, F.product_bound(ref, mag, hi - lo, F32), f"group {g}")
    # results past 2^32 bytes
    groups, m = 70, 8200
    a, b = _randn(groups * 3, m), _randn(groups * 3, m)
    out = torch.empty(groups, m, m, dtype=BF16, device="cuda")
    hq.hq_half_group_k_gemm(a, b, torch.arange(3, 3 * groups + 1, 3, dtype=torch.int32, device="cuda"), out)
    for g in (0, groups - 1):
        x, y = F.f64(a[3 * g:3 * g + 3, -40:]), F.f64(b[3 * g:3 * g + 3])
        ref, mag = x.T @ y, np.abs(x).T @ np.abs(y)
        H.check(out[g, -40:], ref, F.product_bound(ref, mag, 3, BF16), f"group {g} of {groups}")


def test_swiglu():
    U.banner("large swiglu")
    rows, h = 140000, 8200
    x, dy = _randn(rows, 2 * h), _randn(rows, h)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    hq.hq_swiglu(x, y)
    hq.hq_swiglu_backward(dy, x, dx)
    at = _rows(rows)
    small, sy, sdx = x[at], torch.empty(len(at), h, dtype=BF16, device="cuda"), torch.empty(len(at), 2 * h, dtype=BF16,
                                                                                          device="cuda")
    hq.hq_swiglu(small, sy)
    hq.hq_swiglu_backward(dy[at], small, sdx)
    assert torch.equal(y[at], sy) and torch.equal(dx[at], sdx)         # the small call is held to float64 elsewhere


def test_adapters():
    U.banner("large adapters")
    m, L, n, k, r = 140000, 3, 16392, 16392, 8
    x, base = _randn(m, k), _randn(m, n)
    a, b = _randn(L, r, k) * k ** -0.5, _randn(L, n, r) * r ** -0.5
    ids = torch.randint(-1, L, (m,), device="cuda")
    ends, row_map, row_pair = hq.lora_plan(ids, L)
    size = max(hq.hq_lora_workspace_size(m, n, k, r, L), hq.hq_lora_backward_workspace_size(m, n, k, r, L))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    v = torch.zeros(m, r, device="cuda")
    out = torch.empty_like(base)
    kw = dict(row_map=row_map, row_pair=row_pair, workspace=ws)
    hq.hq_lora(x, a, b, None, ends, out, base=base, v=v, **kw)
    dx = torch.empty_like(x)
    da, db = torch.empty(L, r, k, device="cuda"), torch.empty(L, n, r, device="cuda")
    hq.hq_lora_backward(base, x, v, a, b, None, ends, da, db, dx=dx, **kw)           # base for dy
    for t in _rows(m).tolist():
        g = int(ids[t])
        if g < 0:
            assert torch.equal(out[t], base[t]) and torch.all(dx[t] == 0)
            continue
        xv, dyv, A, B = F.f64(x[t]), F.f64(base[t]), F.f64(a[g]), F.f64(b[g])
        for got, ref, mag, inner in (
                (out[t], dyv + (A @ xv) @ B.T, np.abs(dyv) + (np.abs(A) @ np.abs(xv)) @ np.abs(B).T, k),
                (dx[t], (dyv @ B) @ A, (np.abs(dyv) @ np.abs(B)) @ np.abs(A), n)):
            # both FP32 sums and the inner ones taken to 16 bits, then one rounding
            bound = ((inner + r + 32) * 2.0 ** -23 + 2.0 ** -16) * mag + H.UNIT[BF16] * np.abs(ref) + H.FLOOR[BF16]
            H.check(got, ref, bound, f"token {t}")
    # the gradient's sums over all tokens of an adapter: the last column
    at = torch.arange(m, device="cuda")[ids == 2]
    vv = v[row_map[at].long()].double().cpu().numpy()
    dcol = base[at, n - 1].double().cpu().numpy()
    ref, mag = dcol @ vv, np.abs(dcol) @ np.abs(vv)
    H.check(db[2, n - 1], ref, F.product_bound(ref, mag, len(dcol) + 32, F32), "db")
