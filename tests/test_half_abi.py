"""CPU tests of the 16-bit products, SwiGLU and the low-rank adapters: what the host
refuses before any device work, and the binding's checks.  Pointers passed here
are never dereferenced."""
import ctypes
import os

import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import half as R

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


PRODUCT = [(dict(n=12), SHAPE), (dict(n=-8), SHAPE), (dict(n=1 << 21), SHAPE), (dict(G=0), SHAPE), (dict(G=1025), SHAPE),
           (dict(flags=1), MODE), (dict(flags=0x100), MODE), (dict(flags=0x400), MODE), (dict(flags=4), MODE),
           (dict(a=NUL), NULL), (dict(b=NUL), NULL), (dict(out=NUL), NULL), (dict(at=NUL), NULL), (dict(a=FOUR), ALIGN),
           (dict(b=MIS), ALIGN), (dict(out=FOUR), ALIGN), (dict(at=MIS), ALIGN)]


@pytest.mark.parametrize("kw,code", PRODUCT + [
    (dict(k=12), SHAPE), (dict(k=0), SHAPE), (dict(k=1 << 21), SHAPE), (dict(m=-1), SHAPE), (dict(m=1 << 31), SHAPE),
    (dict(m=(1 << 31) - 1, n=1 << 20), SHAPE)])
def test_contiguous_refuses(lib, kw, code):
    a = dict(flags=0, a=A, b=A, at=A, G=4, out=A, m=64, n=64, k=64)
    a.update(kw)
    _refused(lib.hq_half_group_contiguous_gemm(None, *[a[k] for k in ("flags", "a", "b", "at", "G", "out", "m", "n",
                                                                      "k")]), code)


@pytest.mark.parametrize("kw,code", PRODUCT + [
    (dict(k=12), SHAPE), (dict(k=0), SHAPE), (dict(m=0), SHAPE), (dict(m=1 << 30), SHAPE)])
def test_masked_refuses(lib, kw, code):
    a = dict(flags=0, a=A, b=A, at=A, G=4, m=64, out=A, n=64, k=64)
    a.update(kw)
    _refused(lib.hq_half_group_masked_gemm(None, *[a[k] for k in ("flags", "a", "b", "at", "G", "m", "out", "n",
                                                                  "k")]), code)


@pytest.mark.parametrize("kw,code", PRODUCT + [
    (dict(flags=8), MODE), (dict(m=12), SHAPE), (dict(m=-8), SHAPE), (dict(m=1 << 21), SHAPE), (dict(rows=-1), SHAPE),
    (dict(rows=1 << 31), SHAPE), (dict(m=1 << 20, n=1 << 20), SHAPE)])
def test_group_k_refuses(lib, kw, code):
    a = dict(flags=0, a=A, b=A, at=A, G=4, out=A, m=64, n=64, rows=64)
    a.update(kw)
    _refused(lib.hq_half_group_k_gemm(None, *[a[k] for k in ("flags", "a", "b", "at", "G", "out", "m", "n", "rows")]),
             code)


def test_nothing_to_do(lib):
    assert lib.hq_half_group_contiguous_gemm(None, 0, NUL, A, A, 4, NUL, 0, 64, 64) == 0
    assert lib.hq_half_group_contiguous_gemm(None, 0, A, NUL, A, 4, NUL, 64, 0, 64) == 0
    assert lib.hq_half_group_k_gemm(None, 0, NUL, NUL, A, 4, NUL, 0, 64, 64) == 0
    assert lib.hq_swiglu(None, NUL, 0, 64, 0, NUL, 0, NUL, NUL, 0) == 0
    assert lib.hq_swiglu_backward(None, NUL, NUL, 0, 64, 0, NUL, 0, NUL, NUL, NUL, 0) == 0


SWIGLU = [(dict(h=12), SHAPE), (dict(h=0), SHAPE), (dict(h=1 << 28), SHAPE), (dict(rows=-1), SHAPE),
          (dict(rows=1 << 31), SHAPE), (dict(rows=1 << 20, h=1 << 15), SHAPE), (dict(G=-1), SHAPE), (dict(G=1025, slot=4), SHAPE),
          (dict(G=4), SHAPE), (dict(ends=A), SHAPE), (dict(valid=A), SHAPE), (dict(flags=1), MODE), (dict(x=NUL), NULL),
          (dict(y=NUL), NULL), (dict(x=FOUR), ALIGN), (dict(y=MIS), ALIGN), (dict(G=4, ends=MIS), ALIGN),
          (dict(G=4, slot=2, valid=MIS), ALIGN)]


@pytest.mark.parametrize("kw,code", SWIGLU)
def test_swiglu_refuses(lib, kw, code):
    a = dict(x=A, rows=8, h=64, G=0, ends=NUL, slot=0, valid=NUL, y=A, flags=0)
    a.update(kw)
    _refused(lib.hq_swiglu(None, *[a[k] for k in ("x", "rows", "h", "G", "ends", "slot", "valid", "y", "flags")]), code)


@pytest.mark.parametrize("kw,code", [c for c in SWIGLU if c[0] != dict(y=NUL)] + [
    (dict(dy=NUL), NULL), (dict(dx=NUL), NULL), (dict(dy=FOUR), ALIGN), (dict(dx=FOUR), ALIGN)])
def test_swiglu_backward_refuses(lib, kw, code):
    a = dict(dy=A, x=A, rows=8, h=64, G=0, ends=NUL, slot=0, valid=NUL, dx=A, y=A, flags=0)
    a.update(kw)
    _refused(lib.hq_swiglu_backward(None, *[a[k] for k in ("dy", "x", "rows", "h", "G", "ends", "slot", "valid", "dx",
                                                           "y", "flags")]), code)


LORA = [(dict(n=12), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(k=1 << 21), SHAPE), (dict(r=0), SHAPE),
        (dict(r=12), SHAPE), (dict(r=520), SHAPE), (dict(L=0), SHAPE), (dict(L=1025), SHAPE), (dict(m=-1), SHAPE),
        (dict(rows=-1), SHAPE), (dict(rows=1 << 30), SHAPE), (dict(m=1 << 30), SHAPE),
        (dict(rows=(1 << 30) - 1, n=1 << 20, k=1 << 20), SHAPE),
        (dict(map=NUL, pair=NUL, rows=65), SHAPE), (dict(wsb=0), SHAPE), (dict(map=NUL), NULL), (dict(pair=NUL), NULL),
        (dict(ends=NUL), NULL), (dict(ws=NUL), NULL), (dict(x=NUL), NULL), (dict(a=NUL), NULL), (dict(b=NUL), NULL),
        (dict(x=FOUR), ALIGN), (dict(a=MIS), ALIGN), (dict(b=FOUR), ALIGN), (dict(base=FOUR), ALIGN),
        (dict(v=FOUR), ALIGN), (dict(ws=FOUR), ALIGN), (dict(map=MIS), ALIGN), (dict(pair=MIS), ALIGN),
        (dict(ends=MIS), ALIGN), (dict(scale=MIS), ALIGN), (dict(flags=4), MODE)]


def _lora(lib, kw):
    a = dict(flags=0, x=A, a=A, b=A, scale=A, ends=A, L=4, map=A, pair=A, rows=64, base=A, out=A, v=A, m=64, n=64, k=64,
             r=16, ws=A, wsb=1 << 30)
    a.update(kw)
    return lib.hq_lora(None, *[a[k] for k in ("flags", "x", "a", "b", "scale", "ends", "L", "map", "pair", "rows",
                                              "base", "out", "v", "m", "n", "k", "r", "ws", "wsb")])


def _lora_backward(lib, kw):
    a = dict(flags=0, dy=A, x=A, v=A, a=A, b=A, scale=A, ends=A, L=4, map=A, pair=A, rows=64, base=A, dx=A, da=A, db=A,
             m=64, n=64, k=64, r=16, ws=A, wsb=1 << 30)
    a.update(kw)
    return lib.hq_lora_backward(None, *[a[k] for k in ("flags", "dy", "x", "v", "a", "b", "scale", "ends", "L", "map",
                                                       "pair", "rows", "base", "dx", "da", "db", "m", "n", "k", "r",
                                                       "ws", "wsb")])


@pytest.mark.parametrize("kw,code", LORA + [(dict(out=NUL), NULL), (dict(out=FOUR), ALIGN), (dict(flags=0x400), MODE)])
def test_lora_refuses(lib, kw, code):
    _refused(_lora(lib, kw), code)


@pytest.mark.parametrize("kw,code", LORA + [
    (dict(v=NUL), NULL), (dict(dy=NUL), NULL), (dict(da=NUL), NULL), (dict(db=NUL), NULL), (dict(dx=NUL), NULL),
    (dict(dy=FOUR), ALIGN), (dict(dx=FOUR), ALIGN), (dict(da=FOUR), ALIGN), (dict(db=FOUR), ALIGN), (dict(flags=0x200), MODE)])
def test_lora_backward_refuses(lib, kw, code):
    _refused(_lora_backward(lib, kw), code)


def test_lora_no_tokens(lib):
    assert _lora(lib, dict(m=0, rows=0, x=NUL, out=NUL, base=NUL, map=NUL, pair=NUL, v=NUL)) == 0


def test_workspace_sizes_refuse(lib):
    out = ctypes.c_uint64(0)
    for fn in (lib.hq_lora_workspace_size, lib.hq_lora_backward_workspace_size):
        _refused(fn(64, 64, 64, 16, 4, None), NULL)
        for bad in ((-1, 64, 64, 16, 4), (64, 12, 64, 16, 4), (64, 64, 0, 16, 4), (64, 64, 64, 4, 4), (64, 64, 64, 16, 0)):
            _refused(fn(*bad, ctypes.byref(out)), SHAPE)
        assert fn(64, 64, 64, 16, 4, ctypes.byref(out)) == 0


def test_binding_refuses():
    """Wrong types, sizes and places, before the library is called."""
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        hq.hq_half_group_contiguous_gemm(cpu, cpu.view(1, 4, 64), torch.zeros(1, dtype=torch.int32), cpu)
    with pytest.raises(ValueError, match="device"):
        hq.hq_swiglu(cpu, cpu[:, :32])
    with pytest.raises(ValueError, match="device"):
        hq.hq_lora(cpu, cpu.view(1, 4, 64), cpu.view(1, 64, 4), None, torch.zeros(1, dtype=torch.int32), cpu)


# ------------------------------------------------------------------ the oracle itself
def test_oracle_forms_agree():
    g = np.random.default_rng(1)
    a, b = g.standard_normal((20, 6)), g.standard_normal((3, 5, 6))
    ends = [4, 4, 17]
    out, _ = R.contiguous(a, b, ends)
    for t in range(20):
        e = 0 if t < 4 else 2
        if t < 17:
            assert np.allclose(out[t], [sum(a[t, k] * b[e, n, k] for k in range(6)) for n in range(5)])
        else:
            assert np.isnan(out[t]).all()
    flipped, _ = R.contiguous(a, np.ascontiguousarray(b.transpose(0, 2, 1)), ends, True)
    assert np.allclose(out, flipped, equal_nan=True)
    # the gradient for the weights: <dout, out> moves by <dW, d>
    dout, d = g.standard_normal((20, 5)), g.standard_normal(b.shape)
    dw, _ = R.group_k(dout[:17], a[:17], ends)
    moved = (dout * np.nan_to_num(R.contiguous(a, b + d, ends)[0] - out)).sum()
    assert np.isclose((dw * d).sum(), moved)


def test_oracle_swiglu_gradient():
    g = np.random.default_rng(2)
    x, dy, d = g.standard_normal((7, 16)), g.standard_normal((7, 8)), 1e-6
    step = g.standard_normal(x.shape)
    moved = (dy * (R.swiglu(x + d * step) - R.swiglu(x - d * step))).sum() / (2 * d)
    assert np.isclose((np.concatenate(R.swiglu_backward(dy, x), 1) * step).sum(), moved, rtol=1e-6)


def test_oracle_lora_gradients():
    g = np.random.default_rng(3)
    x, a, b = g.standard_normal((9, 6)), g.standard_normal((2, 3, 6)), g.standard_normal((2, 4, 3))
    scale, owner, dy = np.array([0.5, 2.0]), np.array([0, 1, -1, 1, 0, 0, -1, 1, 1]), g.standard_normal((9, 4))
    one = R.lora(x, a, b, scale, owner, None)
    grad = R.lora_backward(dy, x, one["v"], a, b, scale, owner, None)
    for at, name in enumerate(("dx", "da", "db")):
        args = [x, a, b]
        d = g.standard_normal(args[at].shape)
        args[at] = args[at] + d
        moved = (dy * (R.lora(*args, scale, owner, None)["out"] - one["out"])).sum()
        assert np.isclose((grad[name] * d).sum(), moved)
    row_map, row_pair, ends = R.plan(owner, 2)
    assert ends.tolist() == [3, 7] and row_pair.tolist() == [0, 4, 5, 1, 3, 7, 8, -1, -1]
    assert row_map.tolist() == [0, 3, -1, 4, 1, 2, -1, 5, 6]
