"""16-bit products on the GPU in every plan of _half_plans.py: whole outputs against
float64 products, and nothing written around the output or in rows that have no
group.  Bounds: an FP32 sum of exact products, each step off by 2^-23 of the sum
of magnitudes at most, then one rounding to the result's type (or, accumulated,
one addition in FP32)."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from tests import _block as H
from tests import _gpu as U
from tests import _half as F
from tests import _half_plans as P

pytestmark = pytest.mark.gpu

TYPE = {"bf16": F.BF16, "fp16": F.F16, "f32": F.F32, "add": F.F32}


def _generator(what):
    U.banner(what)
    return torch.Generator(device="cuda").manual_seed(int(H.rng(what).integers(0, 2 ** 62)))


def _randn(g, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _out(g, shape, kind, t):
    """An output with marks around and in it (values to add to), and what it holds."""
    whole, out = F.marked(shape, TYPE[kind or t])
    if kind == "add":
        out.copy_(torch.randn(shape, generator=g, device="cuda"))
    return whole, out, out.clone()


def _hold(out, x, y, before, what):
    """out against x y (float64 factors), added to `before` where that is given."""
    ref, mag = x @ y, x.abs() @ y.abs()
    add = torch.zeros_like(ref) if before is None else before.double()
    bound = ((x.shape[1] + 2) * 2.0 ** -23 * mag + H.UNIT[out.dtype] * (ref + add).abs() + H.FLOOR[out.dtype]
             + 2.0 ** -23 * add.abs()) * (1 + 2.0 ** -7)
    err = (out.double() - (ref + add)).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, first at {bad.nonzero()[0].tolist()}, "
                           f"worst {float((err / bound).nan_to_num(9e9).max()):.3g} of it")


def _weights(g, groups, n, k, transpose, dtype):
    """The weights, and those of group e in float64 as [k, n]."""
    b = _randn(g, (groups, k, n) if transpose else (groups, n, k), dtype, 0.1)
    return b, lambda e: b[e].double() if transpose else b[e].double().t().contiguous()


@pytest.mark.parametrize("counts,spare,n,k,t,kind,transpose,plan", P.CONTIGUOUS)
def test_contiguous(counts, spare, n, k, t, kind, transpose, plan):
    what = f"contiguous {counts[:5]} of {len(counts)}+{spare} {n}x{k} {t}->{kind} t={transpose}: {plan}"
    g = _generator(what)
    rows, ends = sum(counts) + spare, np.cumsum(counts)
    a = _randn(g, (rows, k), TYPE[t])
    a[int(ends[-1]):] = float("nan")
    b, weights = _weights(g, len(counts), n, k, transpose, TYPE[t])
    whole, out, before = _out(g, (rows, n), kind, t)
    hq.hq_half_group_contiguous_gemm(a, b, U.dev_i32(ends, "cuda"), out, transpose=transpose, accumulate=kind == "add")
    torch.cuda.synchronize()
    for e, (c, end) in enumerate(zip(counts, ends)):
        r = slice(int(end) - c, int(end))
        if c:
            _hold(out[r], a[r].double(), weights(e), before[r] if kind == "add" else None, f"{what} group {e}")
    assert torch.equal(out[int(ends[-1]):], before[int(ends[-1]):]), f"{what}: rows past the last end"
    F.untouched(whole, what)


@pytest.mark.parametrize("counts,slot,n,k,t,kind,transpose,plan", P.MASKED)
def test_masked(counts, slot, n, k, t, kind, transpose, plan):
    what = f"masked {counts[:5]} of {len(counts)}/{slot} {n}x{k} {t}->{kind} t={transpose}: {plan}"
    g = _generator(what)
    E = len(counts)
    a = _randn(g, (E * slot, k), TYPE[t])
    for e, c in enumerate(counts):
        a[e * slot + c:(e + 1) * slot] = float("inf")
    b, weights = _weights(g, E, n, k, transpose, TYPE[t])
    whole, out, before = _out(g, (E * slot, n), kind, t)
    hq.hq_half_group_masked_gemm(a, b, U.dev_i32(counts, "cuda"), out, slot, transpose=transpose, accumulate=kind == "add")
    torch.cuda.synchronize()
    for e, c in enumerate(counts):
        r, rest = slice(e * slot, e * slot + c), slice(e * slot + c, (e + 1) * slot)
        if c:
            _hold(out[r], a[r].double(), weights(e), before[r] if kind == "add" else None, f"{what} group {e}")
        assert torch.equal(out[rest], before[rest]), f"{what}: padding of group {e}"
    F.untouched(whole, what)


@pytest.mark.parametrize("counts,spare,m,n,t,kind,plan", P.GROUP_K)
def test_group_k(counts, spare, m, n, t, kind, plan):
    what = f"group k {counts[:5]} of {len(counts)}+{spare} {m}x{n} {t}->{kind}: {plan}"
    g = _generator(what)
    rows, ends = sum(counts) + spare, np.cumsum(counts)
    a, b = _randn(g, (rows, m), TYPE[t]), _randn(g, (rows, n), TYPE[t], 0.1)
    a[int(ends[-1]):], b[int(ends[-1]):] = float("nan"), float("inf")
    whole, out, before = _out(g, (len(counts), m, n), kind, t)
    hq.hq_half_group_k_gemm(a, b, U.dev_i32(ends, "cuda"), out, accumulate=kind == "add")
    torch.cuda.synchronize()
    for e, (c, end) in enumerate(zip(counts, ends)):
        r = slice(int(end) - c, int(end))
        if c:
            _hold(out[e], a[r].double().t().contiguous(), b[r].double(), before[e] if kind == "add" else None,
                  f"{what} group {e}")
        else:
            assert torch.equal(out[e], before[e] if kind == "add" else torch.zeros_like(out[e])), f"{what} group {e}"
    F.untouched(whole, what)
