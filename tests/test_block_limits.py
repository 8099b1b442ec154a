"""The largest calls of the block-128 FP8 and dispatch functions: a launch holds
fewer than 2^32 work items, and the host refuses what would pass that (CPU: the
call that just fits gets as far as its missing pointers), or takes another path."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import block as B
from tests import _block as H
from tests import _gpu as U

NUL = None
A = ctypes.c_void_p(0x10000)
NULL, SHAPE = -1, -2


def _quant(lib, batch, m, k, flags):
    return lib.hq_block_quant(None, NUL, batch, m, k, NUL, NUL, flags)


@pytest.mark.parametrize("batch,m,k,flags,code", [
    # 32 blocks a workgroup of 256 threads, 2^24 - 1 workgroups
    (1, (1 << 29) - 32, 32, 0, NULL), (1, (1 << 29) - 31, 32, 0, SHAPE), (4, 1 << 27, 96, 2, SHAPE),
    (1, (1 << 22) - 1, 128 * 128, 0, NULL), (1, 1 << 22, 128 * 128, 0, SHAPE),
    # one tile a workgroup
    (1, (1 << 31) - 128, 32, 4, NULL), (65535, 128, 128 * 256, 4, NULL), (65535, 128, 128 * 257, 4, SHAPE),
    (65535, 256, 128 * 128, 8, NULL), (65535, 256, 128 * 129, 8, SHAPE), (65535, 256, 128 * 129, 12, SHAPE)])
def test_quant(batch, m, k, flags, code):
    assert _quant(hq.load(), batch, m, k, flags) == code


@pytest.mark.parametrize("rows,h,code", [((1 << 29) - 32, 128, NULL), (1 << 29, 128, SHAPE), (1 << 22, 1 << 14, SHAPE)])
def test_swiglu(rows, h, code):
    assert hq.load().hq_fused_swiglu_block_quant(None, NUL, rows, h, NUL, 0, NUL, NUL, 0) == code


# (tokens, pieces of a row, groups with padding rows, refused): four pieces a
# workgroup of 256 threads and eight workgroups a group
PIECES = [((1 << 26) - 4, 1, 0, NULL), ((1 << 26) - 3, 1, 0, SHAPE), ((1 << 20) - 1, 64, 0, NULL),
          (1 << 20, 64, 0, SHAPE), ((1 << 26) - 4, 1, 1, SHAPE), ((1 << 26) - 36, 1, 1, NULL),
          ((1 << 26) - 35, 1, 1, SHAPE)]


@pytest.mark.parametrize("T,pieces,groups,code", PIECES)
def test_permute_and_combine(T, pieces, groups, code):
    lib = hq.load()
    pads = (A, A, groups) if groups else (NUL, NUL, 0)
    assert lib.hq_moe_permute(None, NUL, T, 1024 * pieces, NUL, 1, *pads, 8, NUL) == code
    assert lib.hq_moe_permute_block_quant(None, NUL, T, 1024 * pieces, NUL, 1, *pads, 8, NUL, NUL, 0) == code
    if not groups:
        assert lib.hq_moe_combine(None, NUL, T, 512 * pieces, NUL, 1, NUL, 8, NUL, 0) == code


@pytest.mark.parametrize("T,topk,groups,code", [
    ((1 << 24) - 1, 1, 0, NULL), (1 << 24, 4, 0, SHAPE), ((1 << 23) - 1, 8, 0, NULL), (1 << 23, 8, 0, SHAPE),
    (1 << 23, 64, 0, SHAPE), ((1 << 23) - 8, 8, 1, SHAPE), ((1 << 23) - 9, 8, 1, NULL)])
def test_combine_backward(T, topk, groups, code):
    pads = (A, A, groups) if groups else (NUL, NUL, 0)
    assert hq.load().hq_moe_combine_backward(None, NUL, NUL, T, 64, NUL, topk, NUL, *pads, 8, NUL, NUL, 0) == code


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 9])
def test_few_rows_of_many_columns(m):
    """Columns past one launch of the few-row kernel (2^26): the product is still
    computed, and every column is written."""
    U.banner(f"product {m} x (2^26 + 136) x 32")
    n, k = (1 << 26) + 136, 32
    r = H.rng("columns", m)
    (a, sa), (b, sb) = H.codes(r, m, k), H.codes(r, 128 * 61, k, True)
    db = torch.from_numpy(np.resize(b, (1 << 20, k))).cuda().repeat(65, 1)[:n].contiguous()
    dsb = torch.from_numpy(np.resize(sb, (1 << 13, 1))).cuda().repeat(65, 1)[: -(-n // 128)].contiguous()
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    hq.hq_block_gemm(H.dev(a), H.dev(sa), db, dsb, out)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    for lo in (0, 1 << 24, (1 << 25) + 8, (1 << 26) - 2048, n - 3000):
        lo = lo // 128 * 128
        hi = min(lo + 4096, n)
        cb, cs = db[lo:hi].cpu().numpy(), dsb[lo // 128:-(-hi // 128)].cpu().numpy()
        ref, mag = B.gemm(a, sa, cb, cs)
        H.check(out[:, lo:hi], ref, H.product_bound(ref, mag, k, torch.bfloat16), f"columns from {lo}")
