"""Block-128 FP8 products on the GPU against the float64 oracle, in every form,
at sizes and group shapes where tiles, K blocks and groups end raggedly."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import block as B
from tests import _block as H
from tests import _gpu as U

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _workspace():
    return torch.full((hq.HQ_BLOCK_WORKSPACE_BYTES,), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("m,n,k", [
    (1, 8, 32), (1, 128, 128), (1, 264, 4128), (2, 24, 160), (15, 136, 416), (16, 512, 1024), (17, 520, 2080),
    (31, 256, 512), (33, 1032, 96), (64, 640, 1536), (77, 384, 4096), (100, 2056, 544), (129, 248, 640),
    (200, 1000, 256), (255, 256, 768), (257, 264, 1184), (300, 776, 2048), (513, 520, 416),
])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_dense(m, n, k, dtype):
    what = f"dense {m}x{n}x{k} {dtype}"
    U.banner(what)
    r = H.rng(m, n, k)
    (a, sa), (b, sb) = H.codes(r, m, k), H.codes(r, n, k, True, 0.05)
    ref, mag = B.gemm(a, sa, b, sb)
    bound = H.product_bound(ref, mag, k, dtype)
    args = [H.dev(v) for v in (a, sa, b, sb)]
    for ws in (None, _workspace()):
        out = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
        hq.hq_block_gemm(*args, out, workspace=ws)
        torch.cuda.synchronize()
        H.check(out, ref, bound, f"{what} workspace={ws is not None}")


@pytest.mark.parametrize("m,n,k", [(3, 64, 128), (40, 264, 1056), (300, 512, 512)])
def test_integers_are_exact(m, n, k):
    """Integer codes with power-of-two scales: every partial sum is an exact FP32
    number, so FP32 outputs are exact and 16-bit ones rounded once."""
    U.banner(f"exact {m}x{n}x{k}")
    r = H.rng("exact", m, n, k)
    grid = np.array([0x00, 0x38, 0xB8, 0x40, 0xC0, 0x44, 0xC4, 0x48], np.uint8)      # 0, +-1, +-2, +-3, 4
    a, b = grid[r.integers(0, 8, (m, k))], grid[r.integers(0, 8, (n, k))]
    sa = np.exp2(r.integers(-2, 3, (m, -(-k // 128)))).astype(np.float32)
    sb = np.exp2(r.integers(-2, 3, (-(-n // 128), -(-k // 128)))).astype(np.float32)
    ref, _ = B.gemm(a, sa, b, sb)
    args = [H.dev(v) for v in (a, sa, b, sb)]
    for ws in (None, _workspace()):
        out = torch.empty((m, n), device="cuda")
        hq.hq_block_gemm(*args, out, workspace=ws)
        assert np.array_equal(out.cpu().numpy().astype(np.float64), ref)
        base = torch.from_numpy(r.integers(-9, 9, (m, n)).astype(np.float32)).cuda()
        acc = base.clone()
        hq.hq_block_gemm(*args, acc, accumulate=True, workspace=ws)
        assert np.array_equal(acc.cpu().numpy().astype(np.float64), ref + base.cpu().numpy())
        half = torch.empty((m, n), dtype=BF16, device="cuda")
        hq.hq_block_gemm(*args, half, workspace=ws)
        assert torch.equal(half, out.bfloat16())


def test_scale_of_every_block_and_row():
    """One nonzero code pair per (row, K block), distinct scales: a scale read
    from the wrong row, column block or K block shows."""
    U.banner("scale probe")
    m, n, k = 300, 392, 1184
    kb, nb = -(-k // 128), -(-n // 128)
    a, b = np.zeros((m, k), np.uint8), np.zeros((n, k), np.uint8)
    for j in range(kb):
        a[:, j * 128 + (7 * j) % min(128, k - j * 128)] = 0x38
        b[:, j * 128 + (7 * j) % min(128, k - j * 128)] = 0x38
    sa = (1 + np.arange(m)[:, None] * 0.001 + np.arange(kb)[None] * 0.37).astype(np.float32)
    sb = (1 + np.arange(nb)[:, None] * 0.11 + np.arange(kb)[None] * 0.53).astype(np.float32)
    ref, mag = B.gemm(a, sa, b, sb)
    for ws in (None, _workspace()):
        out = torch.empty((m, n), device="cuda")
        hq.hq_block_gemm(*[H.dev(v) for v in (a, sa, b, sb)], out, workspace=ws)
        H.check(out, ref, H.product_bound(ref, mag, k, F32), "scale probe")


@pytest.mark.parametrize("batch,m,n,k", [(1, 5, 64, 160), (3, 7, 136, 544), (4, 256, 256, 256), (2, 70, 392, 1024)])
def test_batch(batch, m, n, k):
    U.banner(f"batch {batch}x{m}x{n}x{k}")
    r = H.rng("batch", m, n, k)
    A, Bo = [H.codes(r, m, k) for _ in range(batch)], [H.codes(r, n, k, True) for _ in range(batch)]
    out = torch.empty((batch, m, n), dtype=BF16, device="cuda")
    hq.hq_block_gemm(H.dev(np.stack([x[0] for x in A])), H.dev(np.stack([x[1] for x in A])),
                     H.dev(np.stack([x[0] for x in Bo])), H.dev(np.stack([x[1] for x in Bo])), out,
                     workspace=_workspace())
    for i in range(batch):
        ref, mag = B.gemm(*A[i], *Bo[i])
        H.check(out[i], ref, H.product_bound(ref, mag, k, BF16), f"batch item {i}")


GROUPS = [
    ([3, 0, 1, 40], 2, 264, 544), ([0, 0, 0], 5, 128, 256), ([300, 17, 0, 129, 256, 64], 0, 392, 416),
    ([1] * 40, 3, 136, 1056), ([1000], 9, 520, 128), ([128, 256, 0, 384], 128, 512, 640),
    ([5, 90, 33, 0, 65, 2, 31, 128], 1, 1032, 1184),
]


@pytest.mark.parametrize("counts,spare,n,k", GROUPS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_group_contiguous(counts, spare, n, k, dtype):
    what = f"contiguous {counts}+{spare} n={n} k={k} {dtype}"
    U.banner(what)
    r = H.rng(what)
    E, rows = len(counts), sum(counts) + spare
    ends = np.cumsum(counts)
    a, sa = H.codes(r, max(rows, 1), k)
    W = [H.codes(r, n, k, True) for _ in range(E)]
    b, sb = np.stack([w[0] for w in W]), np.stack([w[1] for w in W])
    out = torch.full((max(rows, 1), n), -77.0, dtype=dtype, device="cuda")
    hq.hq_block_group_contiguous_gemm(H.dev(a), H.dev(sa), H.dev(b), H.dev(sb), U.dev_i32(ends, "cuda"), out)
    torch.cuda.synchronize()
    for g in range(E):
        lo, hi = int(ends[g]) - counts[g], int(ends[g])
        if hi > lo:
            ref, mag = B.gemm(a[lo:hi], sa[lo:hi], b[g], sb[g])
            H.check(out[lo:hi], ref, H.product_bound(ref, mag, k, dtype), f"{what} group {g}")
    assert torch.all(out[int(ends[-1]):] == -77.0), f"{what}: rows past the last end written"


def test_group_contiguous_clamps_device_ends():
    """Ends below zero, decreasing or past the rows are clamped, not followed."""
    U.banner("contiguous clamped ends")
    r = H.rng("clamp")
    E, rows, n, k = 5, 70, 136, 256
    a, sa = H.codes(r, rows, k)
    W = [H.codes(r, n, k, True) for _ in range(E)]
    b, sb = np.stack([w[0] for w in W]), np.stack([w[1] for w in W])
    out = torch.full((rows, n), -77.0, dtype=F32, device="cuda")
    hq.hq_block_group_contiguous_gemm(H.dev(a), H.dev(sa), H.dev(b), H.dev(sb),
                                      U.dev_i32([-4, 20, 10, 2 ** 31 - 1, 30], "cuda"), out)
    for g, (lo, hi) in enumerate([(0, 0), (0, 20), (20, 20), (20, 70), (70, 70)]):
        if hi > lo:
            ref, mag = B.gemm(a[lo:hi], sa[lo:hi], b[g], sb[g])
            H.check(out[lo:hi], ref, H.product_bound(ref, mag, k, F32), f"group {g}")


def test_many_groups():
    U.banner("1024 groups")
    r = H.rng("many")
    E, n, k = 1024, 24, 96
    counts = r.integers(0, 4, E)
    ends = np.cumsum(counts)
    a, sa = H.codes(r, int(ends[-1]), k)
    b, sb = H.codes(r, n, k, True)
    bs, sbs = np.stack([b] * E), np.stack([sb * np.float32(1 + g) for g in range(E)])
    out = torch.empty((int(ends[-1]), n), device="cuda")
    hq.hq_block_group_contiguous_gemm(H.dev(a), H.dev(sa), H.dev(bs), H.dev(sbs), U.dev_i32(ends, "cuda"), out)
    f = np.repeat(np.arange(1, E + 1), counts)[:, None]
    ref, mag = B.gemm(a, sa, b, sb)
    H.check(out, ref * f, H.product_bound(ref * f, mag * f, k, F32), "1024 groups")


@pytest.mark.parametrize("counts,max_m,n,k", [([3, 0, 16, 9], 16, 264, 544), ([40, 64, 1, 63, 0], 64, 392, 416),
                                              ([256, 0, 129, 300, -5], 256, 512, 640), ([1, 2], 7, 1032, 1184)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_group_masked(counts, max_m, n, k, dtype):
    what = f"masked {counts}/{max_m} n={n} k={k} {dtype}"
    U.banner(what)
    r = H.rng(what)
    E = len(counts)
    a, sa = H.codes(r, E * max_m, k)
    for g, c in enumerate(counts):          # padding rows: NaN codes and scales
        c = min(max(c, 0), max_m)
        a[g * max_m + c:(g + 1) * max_m] = 0x7F
        sa[g * max_m + c:(g + 1) * max_m] = np.nan
    W = [H.codes(r, n, k, True, 0.05) for _ in range(E)]
    b, sb = np.stack([w[0] for w in W]), np.stack([w[1] for w in W])
    out = torch.full((E * max_m, n), -77.0, dtype=dtype, device="cuda")
    hq.hq_block_group_masked_gemm(H.dev(a), H.dev(sa), H.dev(b), H.dev(sb), U.dev_i32(counts, "cuda"), out, max_m)
    torch.cuda.synchronize()
    for g, c in enumerate(counts):
        c, lo = min(max(c, 0), max_m), g * max_m
        if c:
            ref, mag = B.gemm(a[lo:lo + c], sa[lo:lo + c], b[g], sb[g])
            H.check(out[lo:lo + c], ref, H.product_bound(ref, mag, k, dtype), f"{what} group {g}")
        assert torch.all(out[lo + c:lo + max_m] == -77.0), f"{what}: padding of group {g} written"


@pytest.mark.parametrize("blocks,spare,m,n", [([1, 0, 3], 0, 40, 72), ([0, 0], 2, 17, 8), ([2, 9, 0, 1, 5], 1, 300, 264),
                                              ([40], 0, 130, 520), ([1] * 12, 4, 5, 136)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_group_k(blocks, spare, m, n, dtype):
    what = f"group_k {blocks}+{spare} {m}x{n} {dtype}"
    U.banner(what)
    r = H.rng(what)
    E, K = len(blocks), 128 * (sum(blocks) + spare)
    ends = 128 * np.cumsum(blocks)
    a, sa = H.codes(r, m, K)
    b, sb = H.codes(r, n, K, True)
    a[:, int(ends[-1]):], sa[:, sum(blocks):] = 0x7F, np.nan        # past the last end: never read into a sum
    out = torch.full((E, m, n), float("nan"), dtype=dtype, device="cuda")
    args = (H.dev(a), H.dev(sa), H.dev(b), H.dev(sb), U.dev_i32(ends, "cuda"))
    hq.hq_block_group_k_gemm(*args, out)
    torch.cuda.synchronize()
    refs = []
    for g in range(E):
        lo, hi = int(ends[g]) - 128 * blocks[g], int(ends[g])
        ref, mag = B.gemm(a[:, lo:hi], sa[:, lo // 128:hi // 128], b[:, lo:hi], sb[:, lo // 128:hi // 128])
        H.check(out[g], ref, H.product_bound(ref, mag, max(hi - lo, 1), dtype), f"{what} group {g}")
        refs.append((ref, H.product_bound(ref, mag, max(hi - lo, 1), F32)))
    if dtype is F32:
        acc = torch.full((E, m, n), 3.0, device="cuda")
        hq.hq_block_group_k_gemm(*args, acc, accumulate=True)
        for g, (ref, bound) in enumerate(refs):
            H.check(acc[g], ref + 3.0, bound + 2.0 ** -23 * (np.abs(ref) + 3), f"{what} accumulated group {g}")


def test_gradients_of_a_product():
    """dX and dW of Y = X W^T from quantised operands: against the formula, and
    against differences of sum(dY * Y) for the dequantised X, W and dY."""
    U.banner("gradients")
    r = H.rng("grad")
    m, n, k = 160, 288, 224
    tx, _ = H.halves(r, (m, k), BF16)
    tw, _ = H.halves(r, (n, k), BF16, 0.05)
    ty, _ = H.halves(r, (m, n), BF16, 0.01)
    # dX = dY W: dY in rows, W^T in 128 x 128 blocks
    gy, sgy = hq.block_quantize(ty.cuda())
    wt, swt = hq.block_quantize(tw.cuda(), True, True)
    dx = torch.empty((m, k), device="cuda")
    hq.hq_block_gemm(gy, sgy, wt, swt, dx)
    # dW = dY^T X: dY^T in rows along m, X^T in 128 x 128 blocks
    gyt, sgyt = hq.block_quantize(ty.cuda(), False, True)
    xt, sxt = hq.block_quantize(tx.cuda(), True, True)
    dw = torch.empty((n, k), device="cuda")
    hq.hq_block_gemm(gyt, sgyt, xt, sxt, dw)
    c = lambda t: t.cpu().numpy()  # noqa: E731
    Gy, W = B.dequant(c(gy), c(sgy)), B.dequant(c(wt), c(swt), True).T
    Gyt, X = B.dequant(c(gyt), c(sgyt)).T, B.dequant(c(xt), c(sxt), True).T
    bx = H.product_bound(Gy @ W, np.abs(Gy) @ np.abs(W), n, F32)
    bw = H.product_bound(Gyt.T @ X, np.abs(Gyt).T @ np.abs(X), m, F32)
    H.check(dx, Gy @ W, bx, "dX")
    H.check(dw, Gyt.T @ X, bw, "dW")
    h = 2.0 ** -10          # the loss is linear in each operand: differences are exact up to float64 rounding
    for _ in range(20):
        i, j, l = r.integers(0, m), r.integers(0, n), r.integers(0, k)
        e = np.zeros((m, k))
        e[i, l] = h
        d = (np.sum(Gy * ((X + e) @ W.T)) - np.sum(Gy * ((X - e) @ W.T))) / (2 * h)
        assert abs(float(dx[i, l]) - d) <= bx[i, l] + 1e-8
        e = np.zeros((n, k))
        e[j, l] = h
        d = (np.sum(Gyt * (X @ (W + e).T)) - np.sum(Gyt * (X @ (W - e).T))) / (2 * h)
        assert abs(float(dw[j, l]) - d) <= bw[j, l] + 1e-8


def test_nan_stays_in_its_row_and_column():
    U.banner("nan")
    r = H.rng("nan")
    m, n, k = 70, 136, 512
    a, sa = H.codes(r, m, k)
    b, sb = H.codes(r, n, k, True)
    a[13, 200], sa[40, 2], b[77, 300] = 0x7F, np.inf, 0xFF
    out = torch.empty((m, n), dtype=BF16, device="cuda")
    hq.hq_block_gemm(*[H.dev(v) for v in (a, sa, b, sb)], out)
    bad = ~torch.isfinite(out).cpu().numpy()
    want = np.zeros((m, n), bool)
    want[[13, 40]], want[:, 77] = True, True
    assert np.array_equal(bad, want)


def test_repeats_are_bit_identical_and_run_on_another_stream():
    U.banner("repeat, stream")
    r = H.rng("repeat")
    m, n, k = 77, 512, 4096
    args = [H.dev(v) for v in (*H.codes(r, m, k), *H.codes(r, n, k, True))]
    ws, outs = _workspace(), []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        out = torch.empty((m, n), device="cuda")
        with torch.cuda.stream(s if i % 2 else torch.cuda.current_stream()):
            hq.hq_block_gemm(*args, out, workspace=ws)
        torch.cuda.synchronize()
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_tiles_of_one_step(dtype):
    """More tiles than compute units, each a single K block (some none): the loads
    run several tiles ahead of the sums."""
    what = f"one-step tiles {dtype}"
    U.banner(what)
    r = H.rng("one step")
    blocks = [1, 0, 1, 1, 0, 1] * 8
    E, m, n, K = len(blocks), 600, 1104, 128 * sum(blocks)
    ends = 128 * np.cumsum(blocks)
    (a, sa), (b, sb) = H.codes(r, m, K), H.codes(r, n, K, True)
    out = torch.full((E, m, n), float("nan"), dtype=dtype, device="cuda")
    hq.hq_block_group_k_gemm(H.dev(a), H.dev(sa), H.dev(b), H.dev(sb), U.dev_i32(ends, "cuda"), out)
    for g in range(E):
        lo, hi = int(ends[g]) - 128 * blocks[g], int(ends[g])
        ref, mag = B.gemm(a[:, lo:hi], sa[:, lo // 128:hi // 128], b[:, lo:hi], sb[:, lo // 128:hi // 128])
        # the FP8 matrix instructions' own bound on a sum of one block (BF16 results):
        # each group of eight products keeps 13 bits below its largest, so it
        # loses less than 8 x 2^-13 of that
        own = 2.0 ** -10 * mag if dtype is BF16 else 0.0
        H.check(out[g], ref, H.product_bound(ref, mag, 128, dtype) + own, f"{what} group {g}")
    # short rows through the dense and contiguous forms
    m, n, k = 1500, 2056, 96
    (a, sa), (b, sb) = H.codes(r, m, k), H.codes(r, n, k, True)
    ref, mag = B.gemm(a, sa, b, sb)
    for grouped in (False, True):
        out = torch.empty((m, n), dtype=dtype, device="cuda")
        if grouped:
            hq.hq_block_group_contiguous_gemm(H.dev(a), H.dev(sa), H.dev(b[None]), H.dev(sb[None]),
                                              U.dev_i32([m], "cuda"), out)
        else:
            hq.hq_block_gemm(H.dev(a), H.dev(sa), H.dev(b), H.dev(sb), out)
        H.check(out, ref, H.product_bound(ref, mag, k, dtype), f"{what} grouped={grouped}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_tiles_of_few_steps(dtype):
    """More tiles than compute units, of none to nine K blocks each and with
    partly filled rows and columns: a tile ends at every place of the stages and of
    the scales' groups of four."""
    what = f"short tiles {dtype}"
    U.banner(what)
    r = H.rng("few steps")
    blocks = [2, 3, 1, 5, 0, 4, 9, 1, 1, 7, 6, 2, 8, 3, 0, 4, 5, 1]
    E, m, n, K = len(blocks), 600, 1352, 128 * sum(blocks)
    ends = 128 * np.cumsum(blocks)
    (a, sa), (b, sb) = H.codes(r, m, K), H.codes(r, n, K, True)
    out = torch.full((E, m, n), float("nan"), dtype=dtype, device="cuda")
    hq.hq_block_group_k_gemm(H.dev(a), H.dev(sa), H.dev(b), H.dev(sb), U.dev_i32(ends, "cuda"), out)
    for g in range(E):
        lo, hi = int(ends[g]) - 128 * blocks[g], int(ends[g])
        ref, mag = B.gemm(a[:, lo:hi], sa[:, lo // 128:hi // 128], b[:, lo:hi], sb[:, lo // 128:hi // 128])
        # as above: a group of eight products loses less than 8 x 2^-13 of its largest
        own = 2.0 ** -10 * mag if dtype is BF16 else 0.0
        H.check(out[g], ref, H.product_bound(ref, mag, max(hi - lo, 128), dtype) + own, f"{what} group {g}")


def test_split_of_large_tiles():
    """Few large tiles over a long K: slices of it in a workspace, odd rows, and the
    same bits from run to run."""
    U.banner("K slices of 256 x 256 tiles")
    r = H.rng("large slices")
    m, n, k = 1000, 5120, 8192
    (a, sa), (b, sb) = H.codes(r, m, k), H.codes(r, n, k, True)
    da, dsa, db, dsb = H.dev(a), H.dev(sa), H.dev(b), H.dev(sb)
    ws = torch.empty(hq.hq_block_gemm_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    outs = []
    for _ in range(3):
        out = torch.full((m, n), float("nan"), dtype=BF16, device="cuda")
        hq.hq_block_gemm(da, dsa, db, dsb, out, workspace=ws)
        outs.append(out)
    rows = np.array([0, 1, 63, 64, 127, 128, 255, 256, 511, 700, 767, 768, 900, 999])
    ref, mag = B.gemm(a[rows], sa[rows], b, sb)
    H.check(outs[0][torch.from_numpy(rows).cuda()], ref, H.product_bound(ref, mag, k, BF16), "slices")
    assert all(torch.equal(outs[0], o) for o in outs[1:])
