"""What the block-128 products keep of an inner sum, with the operands that
strain it: in every aligned group of eight neighbouring codes one product of
the largest size, its sign turning from group to group so that those cancel, and
seven products just above or below 2^-13 of it, whose sum is the result."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import block as B
from oracle import formats as F
from tests import _block as H
from tests import _gpu as U

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

#: E4M3 codes from 2^-15 to 2^-11 of the largest one, 448 (0x7E), and zero.
SMALL = np.array([0x00] + [c for c in range(1, 0x7F) if 2.0 ** -15 <= F.e4m3_decode(np.uint8(c)) / 448 <= 2.0 ** -11],
                 np.uint8)


def _straining(r, m, n, k):
    """a [m, k] as above: row i has its large code at place i % 8 of each group,
    and the small codes of rows that differ by 8 differ.  b [n, k]: large codes of
    a sign and size of its own in each row."""
    a = SMALL[r.integers(0, SMALL.size, (m, k))]
    a[: m // 2] = SMALL[r.integers(1, SMALL.size, (m // 2, 1))]     # half of the rows: one small value throughout
    rows, groups = np.arange(m)[:, None], np.arange(k // 8)[None]
    a[rows, 8 * groups + rows % 8] = 0x7E | (groups % 2 << 7)
    b = np.broadcast_to(r.choice(np.array([0x7E, 0xFE, 0x7D, 0xF8], np.uint8), (n, 1)), (n, k)).copy()
    sa = np.exp2(r.integers(-9, -6, (m, -(-k // 128)))).astype(np.float32)
    sb = np.exp2(r.integers(-2, 2, (-(-n // 128), -(-k // 128)))).astype(np.float32)
    return a, sa, b, sb


@pytest.mark.parametrize("blocks,m,n", [([1] * 8, 24, 136), ([1, 2, 0, 5, 1], 300, 264), ([3, 1, 12], 72, 520)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_group_k_keeps_fp32_sums(blocks, m, n, dtype):
    """Ranges of a single block up, with every result type: an FP32 sum, rounded once."""
    what = f"group_k precision {blocks} {m}x{n} {dtype}"
    U.banner(what)
    E, K = len(blocks), 128 * sum(blocks)
    ends = 128 * np.cumsum(blocks)
    a, sa, b, sb = _straining(H.rng(what), m, n, K)
    out = torch.full((E, m, n), float("nan"), dtype=dtype, device="cuda")
    hq.hq_block_group_k_gemm(H.dev(a), H.dev(sa), H.dev(b), H.dev(sb), U.dev_i32(ends, "cuda"), out)
    for g in range(E):
        lo, hi = int(ends[g]) - 128 * blocks[g], int(ends[g])
        ref, mag = B.gemm(a[:, lo:hi], sa[:, lo // 128:hi // 128], b[:, lo:hi], sb[:, lo // 128:hi // 128])
        H.check(out[g], ref, H.product_bound(ref, mag, max(hi - lo, 1), dtype), f"{what} group {g}")


def _kept(ref, mag, k, dtype, fp8):
    """The documented bound: an FP32 sum rounded once, and where the FP8 matrix
    instructions make the inner sums less than 2^-10 of their magnitudes on top
    (eight products of which seven lose up to 2^-13 of the largest)."""
    return H.product_bound(ref, mag, k, dtype) + (2.0 ** -10 * mag if fp8 else 0.0)


@pytest.mark.parametrize("m,n,k", [(8, 136, 1024), (16, 264, 2080), (24, 136, 512), (40, 264, 1056), (300, 520, 768),
                                   (72, 392, 384), (520, 1032, 640)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_dense_keeps_what_is_documented(m, n, k, dtype):
    """Only BF16 results of more than 16 rows and k >= 512 may use the FP8
    instructions; the others keep FP32 sums.  With and without a K split."""
    what = f"dense precision {m}x{n}x{k} {dtype}"
    U.banner(what)
    a, sa, b, sb = _straining(H.rng(what), m, n, k)
    ref, mag = B.gemm(a, sa, b, sb)
    bound = _kept(ref, mag, k, dtype, dtype is BF16 and m > 16 and k >= 512)
    for ws in (None, torch.empty(hq.HQ_BLOCK_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")):
        out = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
        hq.hq_block_gemm(*[H.dev(v) for v in (a, sa, b, sb)], out, workspace=ws)
        H.check(out, ref, bound, what)


@pytest.mark.parametrize("per,k", [(24, 512), (100, 1056), (400, 640), (60, 384)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_groups_keep_what_is_documented(per, k, dtype):
    """Contiguous groups and masked slots of `per` rows: BF16 results of k >= 512
    may use the FP8 instructions."""
    what = f"group precision {per} rows k={k} {dtype}"
    U.banner(what)
    r = H.rng(what)
    E, n = 3, 264
    a, sa, _, _ = _straining(r, E * per, n, k)
    W = [_straining(r, 8, n, k)[2:] for _ in range(E)]
    args = (H.dev(a), H.dev(sa), H.dev(np.stack([w[0] for w in W])), H.dev(np.stack([w[1] for w in W])))
    outs = [torch.full((E * per, n), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    hq.hq_block_group_contiguous_gemm(*args, U.dev_i32(per * np.arange(1, E + 1), "cuda"), outs[0])
    hq.hq_block_group_masked_gemm(*args, U.dev_i32([per] * E, "cuda"), outs[1], per)
    for g in range(E):
        rows = slice(g * per, (g + 1) * per)
        ref, mag = B.gemm(a[rows], sa[rows], *W[g])
        for out in outs:
            H.check(out[rows], ref, _kept(ref, mag, k, dtype, dtype is BF16 and k >= 512), f"{what} group {g}")
