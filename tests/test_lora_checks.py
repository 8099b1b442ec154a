"""CPU tests of what the adapters' calls accept and refuse at the edges of their
plans and sizes.  Every call ends in a refusal before any device work (where the
plan is accepted, at a misaligned scale, which is looked at after it), so no
pointer is dereferenced."""
import ctypes
import os

import pytest

import fp4_gemm_moe_amd as hq

A = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10002)
NULL, SHAPE, ALIGN = -1, -2, -3
ACCEPTED = ALIGN               # the plan and the sizes, before the scale


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(hq.library_path()):
        from fp4_gemm_moe_amd import build
        build.build(verbose=False)
    return hq.load()


def forward(lib, m, rows, n=64, k=64, r=16, L=4, row_map=A, row_pair=A, v=A):
    return lib.hq_lora(None, 0, A, A, A, MIS, A, L, row_map, row_pair, rows, A, A, v, m, n, k, r, A, 1 << 60)


def backward(lib, m, rows, n=64, k=64, r=16, L=4, row_map=A, row_pair=A, v=A):
    return lib.hq_lora_backward(None, 0, A, A, v, A, A, MIS, A, L, row_map, row_pair, rows, A, A, A, A, m, n, k, r, A,
                                1 << 60)


@pytest.mark.parametrize("call", [forward, backward])
def test_plans_without_places(lib, call):
    assert call(lib, 70, 0) == ACCEPTED
    assert call(lib, 70, 0, row_pair=None, v=None) == ACCEPTED
    # no map: the tokens are the places
    assert call(lib, 70, 0, row_map=None, row_pair=None) == SHAPE
    assert call(lib, 70, 69, row_map=None, row_pair=None) == SHAPE
    assert call(lib, 70, 70, row_map=None, row_pair=None) == ACCEPTED
    # places, but not which token each holds
    assert call(lib, 70, 1, row_pair=None) == NULL
