"""CPU tests of the block-128 FP8 and dispatch calls: what the host refuses
before any device work, and the binding's checks.  Pointers passed here are
never dereferenced."""
import ctypes
import os

import pytest
import torch

import fp4_gemm_moe_amd as hq

A = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10002)     # neither 16- nor 4-byte aligned
FOUR = ctypes.c_void_p(0x10004)
NUL = None
NULL, SHAPE, ALIGN, MODE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(hq.library_path()):
        from fp4_gemm_moe_amd import build
        build.build(verbose=False)
    return hq.load()


def _refused(status, code):
    assert status == code and hq.hq_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(k=48), SHAPE), (dict(k=0), SHAPE), (dict(m=-1), SHAPE), (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE),
    (dict(batch=4, m=1 << 29), SHAPE), (dict(m=40, flags=8), SHAPE), (dict(flags=1), MODE), (dict(flags=16), MODE),
    (dict(m=(1 << 31) - 1, k=1 << 20), SHAPE), (dict(x=NUL), NULL), (dict(q=NUL), NULL), (dict(sf=NUL), NULL),
    (dict(x=MIS), ALIGN), (dict(q=FOUR), ALIGN), (dict(sf=MIS), ALIGN)])
def test_quant_refuses(lib, kw, code):
    a = dict(x=A, batch=1, m=64, k=64, q=A, sf=A, flags=0)
    a.update(kw)
    _refused(lib.hq_block_quant(None, a["x"], a["batch"], a["m"], a["k"], a["q"], a["sf"], a["flags"]), code)


@pytest.mark.parametrize("kw,code", [
    (dict(h=48), SHAPE), (dict(rows=-1), SHAPE), (dict(ends=A, groups=0), SHAPE), (dict(ends=A, groups=1025), SHAPE),
    (dict(flags=4), MODE), (dict(x=NUL), NULL), (dict(sf=NUL), NULL), (dict(x=MIS), ALIGN), (dict(sf=MIS), ALIGN)])
def test_swiglu_refuses(lib, kw, code):
    a = dict(x=A, rows=8, h=64, ends=NUL, groups=0, q=A, sf=A, flags=0)
    a.update(kw)
    _refused(lib.hq_fused_swiglu_block_quant(None, *[a[k] for k in ("x", "rows", "h", "ends", "groups", "q", "sf",
                                                                   "flags")]), code)


PRODUCT = [
    (dict(k=48), SHAPE), (dict(k=0), SHAPE), (dict(n=12), SHAPE), (dict(n=-8), SHAPE), (dict(m=-1), SHAPE),
    (dict(k=1 << 23), SHAPE), (dict(m=1 << 30, n=1 << 20), SHAPE), (dict(flags=1), MODE), (dict(flags=0x300), MODE),
    (dict(flags=0x400), MODE), (dict(flags=0x500), MODE), (dict(a=NUL), NULL), (dict(sa=NUL), NULL),
    (dict(b=NUL), NULL), (dict(sb=NUL), NULL), (dict(out=NUL), NULL), (dict(a=MIS), ALIGN), (dict(b=FOUR), ALIGN),
    (dict(out=FOUR), ALIGN), (dict(sa=MIS), ALIGN), (dict(sb=MIS), ALIGN)]


@pytest.mark.parametrize("kw,code", PRODUCT + [
    (dict(batch=65536), SHAPE), (dict(wsb=16), NULL), (dict(ws=FOUR, wsb=16), ALIGN)])
def test_dense_refuses(lib, kw, code):
    a = dict(flags=0, a=A, sa=A, b=A, sb=A, out=A, batch=1, m=64, n=64, k=64, ws=NUL, wsb=0)
    a.update(kw)
    _refused(lib.hq_block_gemm(None, *[a[k] for k in ("flags", "a", "sa", "b", "sb", "out", "batch", "m", "n", "k",
                                                      "ws", "wsb")]), code)


@pytest.mark.parametrize("kw,code", PRODUCT + [(dict(G=0), SHAPE), (dict(G=1025), SHAPE), (dict(ends=NUL), NULL)])
def test_contiguous_refuses(lib, kw, code):
    a = dict(flags=0, a=A, sa=A, b=A, sb=A, ends=A, G=4, out=A, m=64, n=64, k=64)
    a.update(kw)
    _refused(lib.hq_block_group_contiguous_gemm(None, *[a[k] for k in ("flags", "a", "sa", "b", "sb", "ends", "G",
                                                                       "out", "m", "n", "k")]), code)


@pytest.mark.parametrize("kw,code", [c for c in PRODUCT if "m" not in c[0]] + [
    (dict(G=0), SHAPE), (dict(m=0), SHAPE), (dict(m=1 << 30), SHAPE), (dict(counts=NUL), NULL)])
def test_masked_refuses(lib, kw, code):
    a = dict(flags=0, a=A, sa=A, b=A, sb=A, counts=A, G=4, m=64, out=A, n=64, k=64)
    a.update(kw)
    _refused(lib.hq_block_group_masked_gemm(None, *[a[k] for k in ("flags", "a", "sa", "b", "sb", "counts", "G", "m",
                                                                   "out", "n", "k")]), code)


@pytest.mark.parametrize("kw,code", [c for c in PRODUCT if c[0].get("k") != 0] + [
    (dict(k=160), SHAPE), (dict(k=-128), SHAPE), (dict(G=0), SHAPE), (dict(m=1 << 30), SHAPE), (dict(ends=NUL), NULL)])
def test_group_k_refuses(lib, kw, code):
    a = dict(flags=0, a=A, sa=A, b=A, sb=A, ends=A, G=4, out=A, m=64, n=64, k=128)
    a.update(kw)
    _refused(lib.hq_block_group_k_gemm(None, *[a[k] for k in ("flags", "a", "sa", "b", "sb", "ends", "G", "out", "m",
                                                              "n", "k")]), code)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(topk=0), SHAPE), (dict(topk=65), SHAPE), (dict(T=1 << 30), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(align=0), SHAPE), (dict(align=1025), SHAPE), (dict(rows=31), SHAPE),
    (dict(align=128, rows=32), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(ids=NUL), NULL), (dict(map=NUL), NULL),
    (dict(pair=NUL), NULL), (dict(ends=NUL), NULL), (dict(counts=NUL), NULL),
    (dict(T=20000, rows=80000, ws=NUL, wsb=0), NULL), (dict(T=20000, rows=80000, wsb=4), SHAPE),
    (dict(T=20000, rows=80000, ws=MIS), ALIGN)])
def test_sort_refuses(lib, kw, code):
    a = dict(ids=A, T=8, topk=4, E=8, align=1, rows=32, map=A, pair=A, ends=A, counts=A, ws=A, wsb=1 << 20)
    a.update(kw)
    _refused(lib.hq_moe_sort(None, *[a[k] for k in ("ids", "T", "topk", "E", "align", "rows", "map", "pair", "ends",
                                                    "counts", "ws", "wsb")]), code)


MAP = [(dict(T=-1), SHAPE), (dict(topk=0), SHAPE), (dict(topk=65), SHAPE), (dict(rows=-1), SHAPE),
       (dict(rows=1 << 31), SHAPE), (dict(map=NUL), NULL), (dict(x=NUL), NULL), (dict(out=NUL), NULL),
       (dict(x=MIS), ALIGN), (dict(out=FOUR), ALIGN)]
PAD = [(dict(ends=A), NULL), (dict(counts=A), NULL), (dict(ends=A, counts=A, G=0), SHAPE),
       (dict(ends=A, counts=A, G=1025), SHAPE)]


@pytest.mark.parametrize("kw,code", MAP + PAD + [(dict(h=40), SHAPE), (dict(h=0), SHAPE)])
def test_permute_refuses(lib, kw, code):
    a = dict(x=A, T=8, h=64, map=A, topk=4, ends=NUL, counts=NUL, G=0, rows=32, out=A)
    a.update(kw)
    _refused(lib.hq_moe_permute(None, *[a[k] for k in ("x", "T", "h", "map", "topk", "ends", "counts", "G", "rows",
                                                       "out")]), code)


@pytest.mark.parametrize("kw,code", MAP + PAD + [(dict(h=48), SHAPE), (dict(sf=NUL), NULL), (dict(sf=MIS), ALIGN),
                                                 (dict(flags=4), MODE)])
def test_permute_quant_refuses(lib, kw, code):
    a = dict(x=A, T=8, h=64, map=A, topk=4, ends=NUL, counts=NUL, G=0, rows=32, out=A, sf=A, flags=0)
    a.update(kw)
    _refused(lib.hq_moe_permute_block_quant(None, *[a[k] for k in ("x", "T", "h", "map", "topk", "ends", "counts",
                                                                   "G", "rows", "out", "sf", "flags")]), code)


@pytest.mark.parametrize("kw,code", MAP + [(dict(h=12), SHAPE), (dict(w=MIS), ALIGN), (dict(flags=4), MODE)])
def test_combine_refuses(lib, kw, code):
    a = dict(x=A, T=8, h=64, map=A, topk=4, w=A, rows=32, out=A, flags=0)
    a.update(kw)
    _refused(lib.hq_moe_combine(None, *[a[k] for k in ("x", "T", "h", "map", "topk", "w", "rows", "out", "flags")]),
             code)


@pytest.mark.parametrize("kw,code", MAP + PAD + [(dict(h=12), SHAPE), (dict(w=NUL), NULL), (dict(dw=NUL), NULL),
                                                 (dict(y=NUL), NULL), (dict(dw=MIS), ALIGN), (dict(flags=8), MODE)])
def test_combine_backward_refuses(lib, kw, code):
    a = dict(x=A, y=A, T=8, h=64, map=A, topk=4, w=A, ends=NUL, counts=NUL, G=0, rows=32, out=A, dw=A, flags=0)
    a.update(kw)
    _refused(lib.hq_moe_combine_backward(None, *[a[k] for k in ("x", "y", "T", "h", "map", "topk", "w", "ends",
                                                                "counts", "G", "rows", "out", "dw", "flags")]), code)


def test_empty_problems_are_no_ops(lib):
    assert lib.hq_block_quant(None, NUL, 1, 0, 64, NUL, NUL, 0) == 0
    assert lib.hq_block_quant(None, NUL, 0, 8, 64, NUL, NUL, 0) == 0
    assert lib.hq_block_gemm(None, 0, NUL, NUL, NUL, NUL, NUL, 1, 0, 64, 64, NUL, 0) == 0
    assert lib.hq_block_gemm(None, 0, NUL, NUL, NUL, NUL, NUL, 1, 8, 0, 64, NUL, 0) == 0
    assert lib.hq_block_group_contiguous_gemm(None, 0, NUL, NUL, NUL, NUL, NUL, 4, NUL, 0, 64, 64) == 0
    assert lib.hq_moe_permute(None, NUL, 0, 64, NUL, 1, NUL, NUL, 0, 0, NUL) == 0
    assert lib.hq_moe_combine(None, NUL, 0, 64, NUL, 1, NUL, 0, NUL, 0) == 0
    assert lib.hq_moe_combine_backward(None, NUL, NUL, 0, 64, NUL, 1, NUL, NUL, NUL, 0, 0, NUL, NUL, 0) == 0
    assert hq.hq_last_error() == ""


def test_sort_workspace_stays_within_its_constant(lib):
    n = ctypes.c_uint64(0)
    for T, topk in ((1, 1), (2048, 8), (1 << 20, 8), (1 << 24, 64)):
        assert lib.hq_moe_sort_workspace_size(T, topk, 1024, ctypes.byref(n)) == 0
        assert n.value <= hq.HQ_SORT_WORKSPACE_BYTES


def test_max_rows_holds_every_routing():
    import itertools
    for T, E, align in ((3, 2, 4), (2, 3, 3), (4, 2, 1)):
        most = max(sum(-(-ids.count(e) // align) * align for e in range(E))
                   for ids in itertools.product(range(E), repeat=T))
        assert most <= hq.moe_max_rows(T, 1, E, align)


def test_binding_checks_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, sf = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1)
    m = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises((ValueError, TypeError)):
        hq.hq_block_quant(x, q, sf)                                        # CPU tensors
    with pytest.raises((ValueError, TypeError)):
        hq.hq_block_quant(x.float(), q, sf)                                # wrong type
    with pytest.raises(ValueError):
        hq.hq_block_gemm(q, sf, q, sf, torch.zeros(4, 4), accumulate=False)  # CPU tensors
    with pytest.raises(ValueError):
        hq.hq_block_gemm(q, sf, q, sf, torch.zeros(4, 4, dtype=torch.bfloat16), accumulate=True)
    with pytest.raises(ValueError):
        hq.hq_block_group_masked_gemm(q, sf, q.view(1, 4, 64), sf, m[:1, 0], x, 3)
    with pytest.raises(ValueError):
        hq.hq_moe_permute(x, m, None, torch.zeros(2, dtype=torch.int32), x)
    with pytest.raises(ValueError):
        hq.hq_moe_permute(x[:3], m, None, None, x)
