"""CPU tests of what the adapters' calls accept and refuse at the edges of their
plans and sizes.  Every call ends in a refusal before any device work (where the
plan is accepted, at a misaligned scale, which is looked at after it), so no
pointer is dereferenced."""
import ctypes
import os

import pytest

import fp4_gemm_moe_amd as hq

A = ctypes.c_void_p(0x10000)
OUT = ctypes.c_void_p(0x20000)
MIS = ctypes.c_void_p(0x10002)
NULL, SHAPE, ALIGN = -1, -2, -3
ACCEPTED = ALIGN               # the plan and the sizes, before the scale


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(hq.library_path()):
        from fp4_gemm_moe_amd import build
        build.build(verbose=False)
    return hq.load()


def forward(lib, m, rows, n=64, k=64, r=16, L=4, row_map=A, row_pair=A, v=A, out=OUT):
    return lib.hq_lora(None, 0, A, A, A, MIS, A, L, row_map, row_pair, rows, A, out, v, m, n, k, r, A, 1 << 60)


def backward(lib, m, rows, n=64, k=64, r=16, L=4, row_map=A, row_pair=A, v=A):
    return lib.hq_lora_backward(None, 0, A, A, v, A, A, MIS, A, L, row_map, row_pair, rows, A, OUT, A, A, m, n, k, r,
                                A, 1 << 60)


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


def test_work_items_of_the_launches_that_are_made(lib):
    """Calls whose launches stay below 2^32 work items are taken, those of which one would
    pass it are refused; launches of the other direction, or of a path that the
    call does not take, do not count."""
    # 2^28 tokens in tiles of 64: 2^23 workgroups of 256
    assert forward(lib, 1 << 28, 1 << 28, n=8, k=8, r=8) == ACCEPTED
    # the sum of 1024 adapters' chunks would take 2^24 workgroups, but only of the gradients
    assert forward(lib, 64, 64, n=128256, k=4096, r=128, L=1024) == ACCEPTED
    assert backward(lib, 64, 64, n=128256, k=4096, r=128, L=1024) == SHAPE
    # 16 places among 2^30 tokens: a workgroup for 64 tokens without an adapter, beside 5 of dx and 8 of da and db
    assert backward(lib, (1 << 30) - 14 * 64, 16) == ACCEPTED
    assert backward(lib, (1 << 30) - 13 * 64, 16) == SHAPE
    assert backward(lib, (1 << 30) - 8 * 64, 16) == SHAPE
    # the same in one launch of 1024 threads a workgroup
    assert forward(lib, (1 << 28) - 6 * 64, 16) == ACCEPTED
    assert forward(lib, (1 << 28) - 5 * 64, 16) == SHAPE
    # in place there are no workgroups for them
    assert forward(lib, (1 << 30) - 1, 16, out=A) == ACCEPTED
