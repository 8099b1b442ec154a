"""SwiGLU in 16 bits and its gradient on the GPU against float64 and differences."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import half as R
from tests import _block as H
from tests import _gpu as U
from tests import _half as F

pytestmark = pytest.mark.gpu

BF16, F16 = F.BF16, F.F16


def _bounds(x, dy, dtype):
    """exp(-|gate|): its argument is off by 2^-23 |gate| (two roundings), the
    exponential, the reciprocal, two sums and five products by 2^-23 each; below
    2^-126 it may be zero.  Then one rounding."""
    h = x.shape[1] // 2
    gate, up = x[:, :h], x[:, h:]
    rel = (np.abs(gate) + 12) * 2.0 ** -23
    t = np.exp(-np.abs(gate))
    s, rest = np.where(gate >= 0, 1, t) / (1 + t), np.where(gate >= 0, t, 1) / (1 + t)
    tiny = 2.0 ** -125 * (1 + np.abs(gate))

    def done(ref, err):
        return err + H.UNIT[dtype] * np.abs(ref) + H.FLOOR[dtype]

    y = R.swiglu(x)
    out = {"y": (y, done(y, rel * np.abs(y) + tiny * np.abs(up)))}
    if dy is not None:
        dg, du = R.swiglu_backward(dy, x)
        eg = np.abs(dy * up) * (s * (1 + np.abs(gate) * rest) * rel + tiny)
        out["dx"] = (np.concatenate([dg, du], 1),
                     np.concatenate([done(dg, eg), done(du, rel * np.abs(du) + tiny * np.abs(dy))], 1))
    return out


def _inputs(r, rows, h, dtype, sigma=2.0):
    x, xv = F.halves(r, (rows, 2 * h), dtype, sigma)
    dy, dyv = F.halves(r, (rows, h), dtype, 0.5)
    return x, xv, dy, dyv


@pytest.mark.parametrize("rows,h", [(1, 8), (3, 40), (70, 256), (129, 1048), (512, 2048), (1, 17408), (0, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_all_rows(rows, h, dtype):
    what = f"swiglu {rows}x{h} {dtype}"
    U.banner(what)
    x, xv, dy, dyv = _inputs(H.rng(what), rows, h, dtype)
    want = _bounds(xv, dyv, dtype)
    whole, y = F.marked((rows, h), dtype)
    hq.hq_swiglu(x, y)
    wdx, dx = F.marked((rows, 2 * h), dtype)
    wy, y2 = F.marked((rows, h), dtype)
    hq.hq_swiglu_backward(dy, x, dx, y=y2)
    wdx2, dx2 = F.marked((rows, 2 * h), dtype)
    hq.hq_swiglu_backward(dy, x, dx2)
    torch.cuda.synchronize()
    for t in (whole, wdx, wy, wdx2):
        F.untouched(t, what)
    H.check(y, *want["y"], what)
    H.check(dx, *want["dx"], what)
    assert torch.equal(y, y2) and torch.equal(dx, dx2)
    # in place
    hq.hq_swiglu_backward(dy, x, x, y=dy)
    assert torch.equal(x, dx) and torch.equal(dy, y)


@pytest.mark.parametrize("form", ["ends", "ends valid", "slots", "slots valid", "bad ends"])
def test_selected_rows(form):
    """Rows of no group, and past a group's count, are neither read nor written."""
    what = f"swiglu {form}"
    U.banner(what)
    r = H.rng(what)
    rows, h, G = 200, 72, 4
    x, xv, dy, dyv = _inputs(r, rows, h, BF16)
    ends = [30, 30, 110, 170] if form != "bad ends" else [-4, 60, 20, 500]
    counts = [5, 9, 0, 100]
    kw = dict(num_groups=G)
    on = np.zeros(rows, bool)
    for g in range(G):
        if "ends" in form:
            cl = R.clamped(ends, rows)
            lo, hi = (cl[g - 1] if g else 0), cl[g]
        else:
            lo, hi = 40 * g, 40 * g + 40
        on[lo:min(hi, lo + counts[g]) if "valid" in form else hi] = True
    if "ends" in form:
        kw["group_end"] = H.dev(np.array(ends, np.int32))
    else:
        kw["slot_rows"] = 40
    if "valid" in form:
        kw["valid"] = H.dev(np.array(counts, np.int32))
    x[H.dev(~on)] = float("nan")
    want = _bounds(xv, dyv, BF16)
    whole, y = F.marked((rows, h), BF16)
    wdx, dx = F.marked((rows, 2 * h), BF16)
    hq.hq_swiglu(x, y, **kw)
    hq.hq_swiglu_backward(dy, x, dx, **kw)
    torch.cuda.synchronize()
    F.untouched(whole, what)
    F.untouched(wdx, what)
    for got, name in ((y, "y"), (dx, "dx")):
        ref, bound = want[name]
        H.check(F.f64(got)[on], ref[on], bound[on], f"{what} {name}")
        assert torch.all(got[H.dev(~on)] == F.MARK)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_every_gate(dtype):
    """Every finite gate of the type."""
    U.banner(f"swiglu gates {dtype}")
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    gate = bits.view(dtype)
    gate = gate[torch.isfinite(gate)]
    n = gate.numel() // 8 * 8
    gate = gate[:n].view(-1, 8)
    x = torch.cat([gate, torch.full_like(gate, -1.5)], 1).cuda()
    dy = torch.full_like(gate, 0.75).cuda()
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    hq.hq_swiglu(x, y)
    hq.hq_swiglu_backward(dy, x, dx)
    want = _bounds(F.f64(x), F.f64(dy), dtype)
    for got, name in ((y, "y"), (dx, "dx")):
        ref, bound = want[name]
        top = torch.finfo(dtype).max
        # past the type's largest value by less than half a step the result is that value, beyond it Inf
        over = np.abs(ref) * (1 - 2.0 ** -20) > top
        got = F.f64(got)
        assert np.all(np.isinf(got[over]) | (np.abs(got[over]) == top))
        H.check(got[~over], ref[~over], bound[~over], name)


def test_gradient_against_differences():
    """Central differences of the float64 definition at the FP16 inputs, against
    the kernel's gradient: the step 2^-10 leaves an error of its square times a third
    derivative below 1 per unit of dy up."""
    U.banner("swiglu differences")
    r = H.rng("swiglu differences")
    x, xv, dy, dyv = _inputs(r, 16, 64, F16, 1.0)
    dx = torch.empty_like(x)
    hq.hq_swiglu_backward(dy, x, dx)
    step = 2.0 ** -10
    for half in (0, 1):
        d = np.zeros_like(xv)
        d[:, half * 64:(half + 1) * 64] = step
        diff = (R.swiglu(xv + d) - R.swiglu(xv - d)) / (2 * step) * dyv
        got = F.f64(dx)[:, half * 64:(half + 1) * 64]
        up = np.abs(xv[:, 64:]) if half == 0 else 1.0
        bound = step ** 2 * np.abs(dyv) * up + (2.0 ** -11 + 2.0 ** -16) * np.abs(diff) + 2.0 ** -16 * np.abs(dyv) * up + 2.0 ** -24
        H.check(got, diff, bound, f"half {half}")


def test_binding_refuses():
    """Wrong types, sizes and selections of device tensors, before a launch."""
    x, y = torch.zeros(6, 32, dtype=BF16, device="cuda"), torch.full((6, 16), F.MARK, dtype=BF16, device="cuda")
    ends = torch.tensor([2, 6], dtype=torch.int32, device="cuda")
    for bad in (dict(group_end=ends[:0]), dict(valid=ends), dict(group_end=ends, num_groups=3), dict(group_end=ends.long()),
                dict(group_end=ends, valid=ends[:1]), dict(group_end=ends.cpu())):
        with pytest.raises(ValueError):
            hq.hq_swiglu(x, y, **bad)
    for bad in ((x, y.half()), (x, y[:5]), (x.float(), y), (x.t(), y), (x, y.t())):
        with pytest.raises(ValueError):
            hq.hq_swiglu(*bad)
    with pytest.raises(ValueError):
        hq.hq_swiglu_backward(y, x, x[:, :16])
    with pytest.raises(hq.HQError):
        hq.hq_swiglu(x, y, num_groups=2)              # neither ends nor slots
    torch.cuda.synchronize()
    assert torch.all(y == F.MARK)
