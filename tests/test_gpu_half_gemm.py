"""16-bit products by expert on the GPU against float64: sums within their derived
bounds, rows of no group untouched, whatever they hold."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import half as R
from tests import _block as H
from tests import _gpu as U
from tests import _half as F

pytestmark = pytest.mark.gpu

BF16, F16, F32 = F.BF16, F.F16, F.F32


def _ends(sizes, first=0):
    return np.cumsum(sizes).astype(np.int32) + first


def _check_rows(what, whole, out, ref, mag, terms, before=None):
    """Rows of groups within the bound, the others (NaN in ref) as they were."""
    torch.cuda.synchronize()
    F.untouched(whole, what)
    got = F.f64(out)
    rest = np.isnan(ref).all(1)
    assert np.array_equal(got[rest], np.full_like(got[rest], F.MARK) if before is None else before[rest]), \
        f"{what}: rows of no group"
    ref = ref[~rest]
    if before is not None:
        ref = ref + before[~rest]
        mag = mag + 0 * mag
    bound = F.product_bound(ref, mag[~rest], terms, out.dtype) + (0 if before is None else 2.0 ** -23 * np.abs(before[~rest]))
    H.check(got[~rest], ref, bound, what)


# (sizes of the groups, rows past the last end, n, k)
CONTIG = [
    ([1], 0, 8, 8), ([5], 3, 16, 24), ([0, 7, 0, 1], 2, 40, 64), ([3, 0, 250, 9, 61], 5, 264, 136),
    ([64, 64], 0, 128, 72), ([300], 1, 520, 200), ([257, 1, 513, 0, 130], 70, 256, 320),
    ([17] * 40, 0, 96, 512), ([1] * 7 + [0] * 9, 1, 1536, 2048), ([700, 900], 0, 776, 1032), ([130, 600, 20], 9, 4096, 64),
    ([2600, 3100], 33, 520, 192), ([1200] * 4 + [5], 0, 384, 96),
    # results of more than 32 MB: many tiles a workgroup, of one step each and of some
    ([2100, 3, 2101], 7, 4104, 64), ([4300, 1200], 0, 4096, 200), ([20] * 200, 0, 2056, 40),
]


@pytest.mark.parametrize("sizes,spare,n,k", CONTIG)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F16), (BF16, F32)])
def test_contiguous(sizes, spare, n, k, transpose, dtype, out_dtype):
    what = f"contiguous {sizes[:6]} of {len(sizes)} +{spare} n={n} k={k} t={transpose} {dtype}->{out_dtype}"
    U.banner(what)
    r = H.rng(what)
    ends = _ends(sizes)
    rows, E = int(ends[-1]) + spare, len(sizes)
    a, av = F.halves(r, (rows, k), dtype)
    a[rows - spare:] = float("nan")                     # belongs to no group
    b, bv = F.halves(r, (E, k, n) if transpose else (E, n, k), dtype, 0.1)
    whole, out = F.marked((rows, n), out_dtype)
    hq.hq_half_group_contiguous_gemm(a, b, H.dev(ends), out, transpose=transpose)
    ref, mag = R.contiguous(av, bv, ends, transpose)
    _check_rows(what, whole, out, ref, mag, k)


@pytest.mark.parametrize("ends", [[-5, 40, 30, 90], [500, 3, 9, 9], [0, 0, 0, 0], [10, 2 ** 31 - 1, 0, 5]])
@pytest.mark.parametrize("transpose", [False, True])
def test_contiguous_clamps_ends(ends, transpose):
    what = f"contiguous ends {ends} t={transpose}"
    U.banner(what)
    r = H.rng(what)
    a, av = F.halves(r, (100, 64), BF16)
    b, bv = F.halves(r, (4, 64, 64), BF16)
    whole, out = F.marked((100, 64), BF16)
    hq.hq_half_group_contiguous_gemm(a, b, H.dev(np.array(ends, np.int32)), out, transpose=transpose)
    ref, mag = R.contiguous(av, bv, ends, transpose)
    _check_rows(what, whole, out, ref, mag, 64)


@pytest.mark.parametrize("sizes,n,k", [([5, 0, 90], 72, 104), ([700, 300], 264, 520), ([1, 2, 0, 1], 520, 264),
                                       ([2000, 2300], 2056, 72)])
@pytest.mark.parametrize("transpose", [False, True])
def test_contiguous_accumulates(sizes, n, k, transpose):
    what = f"contiguous accumulate {sizes} n={n} k={k} t={transpose}"
    U.banner(what)
    r = H.rng(what)
    ends = _ends(sizes)
    rows, E = int(ends[-1]) + 3, len(sizes)
    a, av = F.halves(r, (rows, k), F16)
    b, bv = F.halves(r, (E, k, n) if transpose else (E, n, k), F16, 0.1)
    whole, out = F.marked((rows, n), F32)
    out.copy_(torch.randn(rows, n, device="cuda"))
    before = F.f64(out)
    hq.hq_half_group_contiguous_gemm(a, b, H.dev(ends), out, transpose=transpose, accumulate=True)
    ref, mag = R.contiguous(av, bv, ends, transpose)
    _check_rows(what, whole, out, ref, mag, k, before)


def test_more_groups_than_rows():
    U.banner("contiguous 1024 groups")
    r = H.rng("1024 groups")
    sizes = (r.random(1024) < 0.3).astype(np.int64) * r.integers(0, 4, 1024)
    ends = _ends(sizes)
    a, av = F.halves(r, (int(ends[-1]), 64), BF16)
    b, bv = F.halves(r, (1024, 24, 64), BF16)
    whole, out = F.marked((int(ends[-1]), 24), BF16)
    hq.hq_half_group_contiguous_gemm(a, b, H.dev(ends), out)
    ref, mag = R.contiguous(av, bv, ends)
    _check_rows("1024 groups", whole, out, ref, mag, 64)


@pytest.mark.parametrize("counts,max_m,n,k", [
    ([1, 0, 3], 3, 64, 72), ([16, -4, 99, 7], 16, 136, 264), ([64, 0, 33, 1, 63], 64, 264, 520),
    ([130, 5, 0, 128], 130, 256, 128), ([300, 0, 1], 300, 520, 192), ([0, 0], 5, 16, 16), ([9] * 70, 20, 200, 64),
    ([64, 3, 50, 0] * 16, 64, 4104, 72), ([30, 31] * 40, 32, 2056, 136), ([8] * 64, 8, 4104, 1032)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F32)])
def test_masked(counts, max_m, n, k, transpose, dtype, out_dtype):
    what = f"masked {counts[:6]} of {len(counts)} slots of {max_m} n={n} k={k} t={transpose} {dtype}->{out_dtype}"
    U.banner(what)
    r = H.rng(what)
    E = len(counts)
    a, av = F.halves(r, (E * max_m, k), dtype)
    for e, c in enumerate(counts):                      # what lies past a slot's count is not read into a result
        a[e * max_m + min(max(c, 0), max_m):(e + 1) * max_m] = float("inf")
    b, bv = F.halves(r, (E, k, n) if transpose else (E, n, k), dtype, 0.1)
    whole, out = F.marked((E * max_m, n), out_dtype)
    hq.hq_half_group_masked_gemm(a, b, H.dev(np.array(counts, np.int32)), out, max_m, transpose=transpose)
    ref, mag = R.masked(av, bv, counts, max_m, transpose)
    _check_rows(what, whole, out, ref, mag, k)


# (sizes, rows past the last end, m, n)
KGROUP = [([1], 0, 8, 8), ([0, 5, 33, 0], 3, 16, 40), ([64, 1, 127, 31], 0, 72, 136), ([300, 0, 513], 9, 264, 256),
          ([2000], 0, 128, 520), ([7] * 20, 1, 256, 24), ([0, 0, 0], 4, 24, 32), ([90, 700], 0, 520, 776),
          ([65, 66, 0, 2], 0, 1032, 1536), ([3, 0, 70, 9] * 50, 2, 136, 264),       # more groups than are ordered
          ([10, 90, 0, 130] * 10, 0, 520, 520), ([64] * 128, 0, 264, 136)]


@pytest.mark.parametrize("sizes,spare,m,n", KGROUP)
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F16, F32), (BF16, BF16), (F16, F16)])
def test_group_k(sizes, spare, m, n, dtype, out_dtype):
    what = f"group k {sizes[:6]} of {len(sizes)} +{spare} m={m} n={n} {dtype}->{out_dtype}"
    U.banner(what)
    r = H.rng(what)
    ends = _ends(sizes)
    rows, E = int(ends[-1]) + spare, len(sizes)
    a, av = F.halves(r, (rows, m), dtype)
    b, bv = F.halves(r, (rows, n), dtype, 0.1)
    a[rows - spare:], b[rows - spare:] = float("nan"), float("inf")
    whole, out = F.marked((E, m, n), out_dtype)
    hq.hq_half_group_k_gemm(a, b, H.dev(ends), out)
    torch.cuda.synchronize()
    F.untouched(whole, what)
    ref, mag = R.group_k(av[:ends[-1]], bv[:ends[-1]], ends)
    H.check(out, ref, F.product_bound(ref, mag, max(sizes), out_dtype), what)


def test_group_k_accumulates_and_clamps():
    for ends in ([10, 10, 90, 200], [-3, 50, 20, 77]):
        what = f"group k accumulate {ends}"
        U.banner(what)
        r = H.rng(what)
        a, av = F.halves(r, (100, 72), BF16)
        b, bv = F.halves(r, (100, 200), BF16)
        out = torch.randn(4, 72, 200, device="cuda")
        before = F.f64(out)
        hq.hq_half_group_k_gemm(a, b, H.dev(np.array(ends, np.int32)), out, accumulate=True)
        ref, mag = R.group_k(av, bv, ends)
        for g in range(4):
            if not mag[g].any():
                assert np.array_equal(F.f64(out[g]), before[g])
        H.check(out, ref + before, F.product_bound(ref + before, mag, 100, F32) + 2.0 ** -23 * np.abs(before), what)


def test_no_rows():
    a, b = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(3, 64, 64, dtype=BF16, device="cuda")
    ends = torch.zeros(3, dtype=torch.int32, device="cuda")
    hq.hq_half_group_contiguous_gemm(a, b, ends, torch.empty(0, 64, dtype=BF16, device="cuda"))
    out = torch.full((3, 64, 64), F.MARK, device="cuda")
    hq.hq_half_group_k_gemm(a, torch.empty(0, 64, dtype=BF16, device="cuda"), ends, out)
    assert torch.all(out == 0)
    out.fill_(F.MARK)
    hq.hq_half_group_k_gemm(a, torch.empty(0, 64, dtype=BF16, device="cuda"), ends, out, accumulate=True)
    assert torch.all(out == F.MARK)


def test_infinities_and_nan_stay_in_their_rows():
    """A row's NaN or Inf reaches that row of out, a weight's that column of its
    expert; nothing else."""
    U.banner("non-finite values")
    r = H.rng("nonfinite")
    for transpose in (False, True):
        a, av = F.halves(r, (90, 72), BF16)
        b, bv = F.halves(r, (3, 72, 72), BF16)
        ends = _ends([40, 17, 33])
        a[3, 5], b[1, 9, 9] = float("nan"), float("inf")
        out = torch.empty(90, 72, dtype=BF16, device="cuda")
        hq.hq_half_group_contiguous_gemm(a, b, H.dev(ends), out, transpose=transpose)
        bad = ~torch.isfinite(out)
        want = torch.zeros_like(bad)
        want[3] = True
        want[40:57, 9] = True
        assert torch.equal(bad, want)


def test_streams_and_graphs():
    """A call on a side stream, and calls captured into a graph: replays with eager
    work between them give the eager bits, for new inputs too."""
    U.banner("half products graph")
    torch.manual_seed(5)
    a, dy = torch.randn(600, 256, device="cuda").bfloat16(), torch.randn(600, 392, device="cuda").bfloat16()
    b = torch.randn(5, 392, 256, device="cuda").bfloat16()
    ends = torch.tensor([100, 100, 350, 351, 590], dtype=torch.int32, device="cuda")
    counts = torch.tensor([0, 7, 120, 1, 60], dtype=torch.int32, device="cuda")

    def once():
        y = torch.zeros(600, 392, dtype=BF16, device="cuda")
        hq.hq_half_group_contiguous_gemm(a, b, ends, y)
        dx = torch.zeros(600, 256, device="cuda")
        hq.hq_half_group_contiguous_gemm(dy, b, ends, dx, transpose=True)
        dw = torch.empty(5, 392, 256, device="cuda")
        hq.hq_half_group_k_gemm(dy, a, ends, dw)
        z = torch.zeros(600, 392, dtype=BF16, device="cuda")
        hq.hq_half_group_masked_gemm(a, b, counts, z, 120)
        return y, dx, dw, z

    eager = [t.clone() for t in once()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = once()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(eager, got):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = once()
    for i in range(4):
        a.copy_(torch.randn(600, 256, device="cuda"))
        ends.copy_(torch.randint(0, 601, (5,), device="cuda").sort().values)
        want = [t.clone() for t in once()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(captured, want):
            assert torch.equal(x, y), f"replay {i}"
