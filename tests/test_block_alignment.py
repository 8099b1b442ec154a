"""CPU tests: the block-128 and dispatch calls refuse index tensors that are not
aligned to their elements.  Pointers passed here are never dereferenced."""
import ctypes

import pytest

import fp4_gemm_moe_amd as hq

A = ctypes.c_void_p(0x10000)
TWO = ctypes.c_void_p(0x10002)
FOUR = ctypes.c_void_p(0x10004)
NUL = None
ALIGN = -3


def _refused(status):
    assert status == ALIGN and "aligned" in hq.hq_last_error()


def test_groups_ends_and_counts():
    lib = hq.load()
    _refused(lib.hq_fused_swiglu_block_quant(None, A, 8, 64, TWO, 4, A, A, 0))
    _refused(lib.hq_block_group_contiguous_gemm(None, 0, A, A, A, A, TWO, 4, A, 64, 64, 64))
    _refused(lib.hq_block_group_masked_gemm(None, 0, A, A, A, A, TWO, 4, 64, A, 64, 64))
    _refused(lib.hq_block_group_k_gemm(None, 0, A, A, A, A, TWO, 4, A, 64, 64, 128))


@pytest.mark.parametrize("kw", [dict(ids=FOUR), dict(map=TWO), dict(pair=TWO), dict(ends=TWO), dict(counts=TWO)])
def test_sort(kw):
    a = dict(ids=A, map=A, pair=A, ends=A, counts=A)
    a.update(kw)
    _refused(hq.load().hq_moe_sort(None, a["ids"], 8, 4, 8, 1, 32, a["map"], a["pair"], a["ends"], a["counts"], A,
                                   1 << 20))


@pytest.mark.parametrize("kw", [dict(map=TWO), dict(ends=TWO), dict(counts=TWO)])
def test_calls_that_walk_a_map(kw):
    lib = hq.load()
    a = dict(map=A, ends=A, counts=A)
    a.update(kw)
    pads = (a["ends"], a["counts"], 4)
    _refused(lib.hq_moe_permute(None, A, 8, 64, a["map"], 4, *pads, 32, A))
    _refused(lib.hq_moe_permute_block_quant(None, A, 8, 64, a["map"], 4, *pads, 32, A, A, 0))
    _refused(lib.hq_moe_combine_backward(None, A, A, 8, 64, a["map"], 4, A, *pads, 32, A, A, 0))
    if a["map"] is TWO:
        _refused(lib.hq_moe_combine(None, A, 8, 64, TWO, 4, A, 32, A, 0))
