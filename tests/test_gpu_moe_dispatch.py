"""Tokens sorted by expert and back on the GPU against the oracle: maps, counts,
copied rows, codes and scales exactly; sums within their derived bounds."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import block as B
from tests import _block as H
from tests import _gpu as U

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def _ids(r, T, topk, E, kind="mixed"):
    if kind == "none":
        return np.full((T, topk), -1, np.int64)
    if kind == "one":
        return np.full((T, topk), E - 1, np.int64)
    ids = r.integers(0, E, (T, topk))
    if kind == "mixed":                      # some unassigned, some far out of range
        ids = np.where(r.random((T, topk)) < 0.1, -1, ids)
        ids = np.where(r.random((T, topk)) < 0.02, E + 2 ** 40, ids)
    return ids.astype(np.int64)


def _sorted(ids, E, align, spare=0):
    T, topk = ids.shape
    rows = hq.moe_max_rows(T, topk, E, align) + spare
    row_map = torch.full((T, topk), -9, dtype=torch.int32, device="cuda")
    row_pair = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    ends = torch.full((E,), -9, dtype=torch.int32, device="cuda")
    counts = torch.full((E,), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((hq.HQ_SORT_WORKSPACE_BYTES,), 0xEE, dtype=torch.uint8, device="cuda")
    hq.hq_moe_sort(H.dev(ids), E, align, row_map, row_pair, ends, counts, ws)
    torch.cuda.synchronize()
    return row_map, row_pair, ends, counts


CASES = [(0, 2, 4, 1, "mixed"), (1, 1, 1, 1, "full"), (1, 8, 64, 128, "mixed"), (7, 3, 5, 1, "mixed"),
         (64, 8, 64, 1, "mixed"), (100, 4, 32, 128, "mixed"), (65, 64, 1024, 16, "mixed"), (300, 2, 3, 7, "one"),
         (50, 2, 8, 128, "none"), (2500, 4, 32, 128, "mixed"), (5000, 8, 1000, 1, "mixed"), (3001, 3, 1, 1024, "mixed")]


@pytest.mark.parametrize("T,topk,E,align,kind", CASES)
def test_sort(T, topk, E, align, kind):
    what = f"sort T={T} top{topk} E={E} align={align} {kind}"
    U.banner(what)
    ids = _ids(H.rng(what), T, topk, E, kind)
    got = _sorted(ids, E, align, 5)
    want = B.sort(ids, E, align, got[1].numel())
    for g, w, name in zip(got, want, ("row_map", "row_pair", "group_end", "counts")):
        assert np.array_equal(g.cpu().numpy(), w), f"{what}: {name}"


def test_sort_large_in_runs():
    """Several workgroups, two sizes of run; and the allocating helper."""
    for T, topk, E in ((16384, 4, 32), (40000, 64, 128)):
        U.banner(f"sort T={T} top{topk} E={E}")
        ids = H.rng(T).integers(-1, E, (T, topk))
        row_map, row_pair, ends, counts = [t.cpu().numpy() for t in hq.moe_sort(H.dev(ids), E, 128)]
        flat = ids.reshape(-1)
        want = np.bincount(flat[flat >= 0], minlength=E)
        assert np.array_equal(counts, want) and np.array_equal(ends, np.cumsum(-(-want // 128) * 128))
        order = np.argsort(np.where(flat < 0, E, flat), kind="stable")[:want.sum()]
        rows = np.concatenate([s + np.arange(c) for s, c in zip(np.concatenate([[0], ends[:-1]]), want)])
        assert np.array_equal(row_pair[rows], order) and np.array_equal(row_map.reshape(-1)[order], rows)
        assert np.all(row_map.reshape(-1)[flat < 0] == -1)
        rest = np.ones(row_pair.size, bool)
        rest[rows] = False
        assert np.all(row_pair[rest] == -1)


@pytest.mark.parametrize("T,topk,E,align,h,dtype", [
    (1, 1, 1, 1, 32, BF16), (5, 3, 4, 1, 416, F16), (33, 8, 64, 1, 1056, BF16), (70, 2, 3, 128, 2080, BF16),
    (0, 2, 4, 128, 64, BF16), (200, 4, 16, 128, 512, F16)])
def test_permute_and_its_quantised_form(T, topk, E, align, h, dtype):
    what = f"permute T={T} top{topk} E={E} align={align} h={h} {dtype}"
    U.banner(what)
    r = H.rng(what)
    ids = _ids(r, T, topk, E)
    row_map, _, ends, counts = _sorted(ids, E, align, 3)
    rows = hq.moe_max_rows(T, topk, E, align) + 3
    t, x = H.halves(r, (T, h), dtype)
    m = row_map.cpu().numpy()
    pads = np.zeros(rows, bool)
    for e, c, lo in zip(ends.cpu().numpy(), counts.cpu().numpy(), np.concatenate([[0], ends.cpu().numpy()[:-1]])):
        pads[lo + c:e] = True
    for pad in (True, False):
        g, c = (ends, counts) if pad else (None, None)
        out = torch.full((rows, h), 9.0, dtype=dtype, device="cuda")
        hq.hq_moe_permute(t.cuda(), row_map, g, c, out)
        start = np.full((rows, h), 9.0, np.float32)
        if pad:
            start[pads] = 0.0
        assert np.array_equal(out.float().cpu().numpy(), B.permute(x, m, start)), what
        q = torch.full((rows, h), 0x55, dtype=torch.uint8, device="cuda")
        sf = torch.full((rows, -(-h // 128)), 5.0, device="cuda")
        hq.hq_moe_permute_block_quant(t.cuda(), row_map, g, c, q, sf)
        xq, xs = B.quant(x) if T else (np.empty((0, h), np.uint8), np.empty((0, sf.shape[1]), np.float32))
        sq, ss = np.full((rows, h), 0x55, np.uint8), np.full(sf.shape, 5.0, np.float32)
        if pad:
            sq[pads], ss[pads] = 0, 2.0 ** -126
        assert np.array_equal(q.cpu().numpy(), B.permute(xq, m, sq)), f"{what}: codes"
        assert np.array_equal(sf.cpu().numpy(), B.permute(xs, m, ss)), f"{what}: scales"


@pytest.mark.parametrize("T,topk,E,align,h,dtype", [
    (1, 1, 1, 1, 8, BF16), (5, 3, 4, 1, 416, F16), (33, 8, 64, 1, 1064, BF16), (70, 2, 3, 128, 2048, BF16),
    (40, 64, 100, 1, 520, F16), (200, 5, 16, 128, 4104, BF16)])
def test_combine_and_its_gradient(T, topk, E, align, h, dtype):
    what = f"combine T={T} top{topk} E={E} align={align} h={h} {dtype}"
    U.banner(what)
    r = H.rng(what)
    ids = _ids(r, T, topk, E)
    if T > 2:
        ids[1] = -1                                     # a token without a row
    row_map, _, ends, counts = _sorted(ids, E, align)
    rows = hq.moe_max_rows(T, topk, E, align)
    ty, y = H.halves(r, (rows, h), dtype)
    m = row_map.cpu().numpy()
    used = np.zeros(rows, bool)
    used[m[m >= 0]] = True
    y[~used] = np.nan                                   # rows that no pair maps to are never read into a sum
    ty = torch.from_numpy(y).to(dtype).cuda()
    w = r.random((T, topk)).astype(np.float32)
    w[m < 0] = np.nan                                   # nor are the weights of unassigned pairs
    for weights in (w, None):
        out = torch.full((T, h), 9.0, dtype=dtype, device="cuda")
        hq.hq_moe_combine(ty, row_map, None if weights is None else H.dev(weights), out)
        ref, mag = B.combine(y, m, weights)
        H.check(out, ref, H.sum_bound(ref, mag, topk, dtype), what)
    td, d = H.halves(r, (T, h), dtype, 0.1)
    dy = torch.full((rows, h), 9.0, dtype=dtype, device="cuda")
    dw = torch.full((T, topk), 9.0, device="cuda")
    hq.hq_moe_combine_backward(td.cuda(), ty, row_map, H.dev(w), ends, counts, dy, dw)
    rdy, rdw, mag = B.combine_backward(d, y, m, w)
    last = int(ends[-1])
    assert torch.all(dy[last:] == 9.0), f"{what}: rows past the last end written"
    H.check(dy[:last], rdy[:last], H.sum_bound(rdy, np.abs(rdy), 1, dtype)[:last], f"{what}: dy")
    H.check(dw, rdw, H.sum_bound(rdw, mag, h, torch.float32), f"{what}: dweights")
    # the loss sum(dout * combine(y, w)) is linear in w and in y: central
    # differences are exact up to float64 rounding
    loss = lambda yy, ww: float(np.sum(d * B.combine(yy, m, ww)[0]))  # noqa: E731
    base = np.where(np.isnan(y), 0.0, y).astype(np.float64)
    bw = H.sum_bound(rdw, mag, h, torch.float32)
    by = H.sum_bound(rdy, np.abs(rdy), 1, dtype)
    for _ in range(6):
        t, j = int(r.integers(0, T)), int(r.integers(0, topk))
        if m[t, j] < 0:
            assert float(dw[t, j]) == 0.0
            continue
        e = np.zeros((T, topk))
        e[t, j] = 0.5
        w0 = np.where(np.isnan(w), 0.0, w).astype(np.float64)
        diff = loss(base, w0 + e) - loss(base, w0 - e)
        assert abs(float(dw[t, j]) - diff) <= bw[t, j] + 1e-9 * np.abs(d[t]) @ np.abs(base[m[t, j]]) + 1e-9
        c = int(r.integers(0, h))
        p = base.copy()
        p[m[t, j], c] += 0.5
        q = base.copy()
        q[m[t, j], c] -= 0.5
        assert abs(float(dy[m[t, j], c]) - (loss(p, w0) - loss(q, w0))) <= by[m[t, j], c] + 1e-8


def test_map_entries_out_of_range_are_skipped():
    """A row map is device data: entries past the rows are unassigned, not followed."""
    U.banner("map out of range")
    r = H.rng("range")
    T, topk, rows, h = 6, 2, 10, 64
    m = np.array([[0, 10], [-1, 3], [2 ** 31 - 1, 4], [-2 ** 31, 5], [6, 99], [7, 8]], np.int32)
    t, x = H.halves(r, (T, h), BF16)
    out = torch.full((rows, h), 9.0, dtype=BF16, device="cuda")
    hq.hq_moe_permute(t.cuda(), H.dev(m), None, None, out)
    assert np.array_equal(out.float().cpu().numpy(), B.permute(x, m, np.full((rows, h), 9.0, np.float32)))
    ty, y = H.halves(r, (rows, h), BF16)
    res = torch.empty((T, h), dtype=BF16, device="cuda")
    hq.hq_moe_combine(ty.cuda(), H.dev(m), None, res)
    ref, mag = B.combine(y, m)
    H.check(res, ref, H.sum_bound(ref, mag, topk, BF16), "combine")


def test_round_trip_is_the_sum_of_copies():
    """Permute, then combine without weights: each token times its row count."""
    U.banner("round trip")
    r = H.rng("trip")
    T, topk, E, h = 90, 4, 8, 256
    ids = _ids(r, T, topk, E)
    row_map, _, ends, counts = _sorted(ids, E, 128)
    t, x = H.halves(r, (T, h), BF16)
    rows = torch.empty((hq.moe_max_rows(T, topk, E, 128), h), dtype=BF16, device="cuda")
    hq.hq_moe_permute(t.cuda(), row_map, ends, counts, rows)
    out = torch.empty((T, h), dtype=BF16, device="cuda")
    hq.hq_moe_combine(rows, row_map, None, out)
    n = (row_map.cpu().numpy() >= 0).sum(1, keepdims=True)
    H.check(out, x.astype(np.float64) * n, H.sum_bound(x * n, np.abs(x) * n, topk, BF16), "round trip")
