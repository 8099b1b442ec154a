"""Low-rank adapters on the GPU at the edges of their plans."""
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


def _workspace(size):
    return torch.full((size,), 0xEE, dtype=torch.uint8, device="cuda")          # its contents do not matter


# m, adapters, n, k, r: the inner sums' slices joined by a launch of their own (three), by the readers, one slice, few places
# in slices, one launch for all
@pytest.mark.parametrize("m,L,n,k,r", [(700, 2, 264, 4168, 16), (700, 2, 264, 4168, 64), (300, 3, 72, 2056, 128),
                                       (150, 4, 136, 264, 16), (900, 8, 72, 1032, 32), (40, 5, 264, 6152, 16),
                                       (20, 4, 72, 520, 16)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_past_the_last_end(m, L, n, k, r, dtype):
    """Tokens in the order of their adapters, without a map, and more behind them: v's
    rows of those are not written, and out's are base's."""
    what = f"lora past the last end m={m} L={L} n={n} k={k} r={r} {dtype}"
    U.banner(what)
    g = H.rng(what)
    ends = np.sort(g.integers(0, m - m // 4, L))
    ends[-1] = m - m // 4
    owner = np.searchsorted(ends, np.arange(m), side="right")
    owner[owner == L] = -1
    x, xv = F.halves(g, (m, k), dtype)
    a, av = F.halves(g, (L, r, k), dtype, k ** -0.5)
    b, bv = F.halves(g, (L, n, r), dtype, r ** -0.5)
    base, basev = F.halves(g, (m, n), dtype)
    ref = R.lora(xv, av, bv, np.ones(L), owner, basev)
    whole, v = F.marked((m, r), F32)
    out = torch.empty_like(base)
    hq.hq_lora(x, a, b, None, H.dev(ends.astype(np.int32)), out, base=base, v=v,
               workspace=_workspace(hq.hq_lora_workspace_size(m, n, k, r, L)))
    torch.cuda.synchronize()
    F.untouched(whole, what)
    last = int(ends[-1])
    assert torch.all(v[last:] == F.MARK), f"{what}: v of tokens without an adapter"
    H.check(v[:last], ref["v"][:last], F.product_bound(ref["v"][:last], ref["vmag"][:last], k, F32), f"{what}: v")
    # both FP32 sums, the inner ones taken to 16 bits, then one rounding
    bound = ((k + r + 32) * 2.0 ** -23 + 2.0 ** -16) * ref["mag"] + H.UNIT[dtype] * np.abs(ref["out"]) + H.FLOOR[dtype]
    H.check(out, ref["out"], bound, what)
    assert torch.equal(out[last:], base[last:])


@pytest.mark.parametrize("unused", [float("nan"), float("inf"), -2.0])
@pytest.mark.parametrize("m,align", [(40, 1), (40, 16), (3000, 1), (3000, 16)])
def test_an_unused_adapters_scale(unused, m, align):
    """da and db of an adapter without tokens are zeros whatever its scale, also
    where its places are there but hold no token; the others are as they were."""
    what = f"lora unused scale {unused} m={m} align={align}"
    U.banner(what)
    L, n, k, r = 5, 136, 264, 16
    g = H.rng(what)
    ids = g.choice([0, 2, 3], m).astype(np.int64)
    row_map, row_pair, ends, _ = hq.moe_sort(H.dev(ids).view(-1, 1), L, align)
    if align > 1:           # adapter 4 gets all the places that are left, without a token
        ends[4] = row_pair.numel()
    x, dy = F.halves(g, (m, k), BF16)[0], F.halves(g, (m, n), BF16)[0]
    a, b = F.halves(g, (L, r, k), BF16)[0], F.halves(g, (L, n, r), BF16)[0]
    v = torch.randn(row_pair.numel(), r, device="cuda")
    space = _workspace(hq.hq_lora_backward_workspace_size(m, n, k, r, L, row_pair.numel()))
    got = []
    for s in (1.5, unused):
        scale = torch.tensor([1.5, s, 1.5, 1.5, s], device="cuda")
        da, db = torch.empty(L, r, k, device="cuda"), torch.empty(L, n, r, device="cuda")
        hq.hq_lora_backward(dy, x, v, a, b, scale, ends, da, db, row_map=row_map, row_pair=row_pair, workspace=space)
        got.append((da, db))
    for before, after in zip(*got):
        assert torch.all(after[[1, 4]] == 0), f"{what}: gradients of an adapter without tokens"
        assert torch.equal(before[[0, 2, 3]], after[[0, 2, 3]])
    # one that has tokens does get its scale
    scale = torch.full((L,), unused, device="cuda")
    hq.hq_lora_backward(dy, x, v, a, b, scale, ends, da, db, row_map=row_map, row_pair=row_pair, workspace=space)
    if np.isfinite(unused):
        assert torch.equal(da, got[0][0] * (unused / 1.5)) or torch.allclose(da, got[0][0] * (unused / 1.5), rtol=1e-6)
    else:
        assert not torch.isfinite(da[[0, 2, 3]]).any() and not torch.isfinite(db[[0, 2, 3]]).any()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_no_places(dtype):
    """A map that holds no place: every token is without an adapter."""
    U.banner(f"lora no places {dtype}")
    m, L, n, k, r = 70, 3, 136, 72, 16
    g = H.rng("no places", str(dtype))
    x, base = F.halves(g, (m, k), dtype)[0], F.halves(g, (m, n), dtype)[0]
    a, b = F.halves(g, (L, r, k), dtype)[0], F.halves(g, (L, n, r), dtype)[0]
    ends = torch.zeros(L, dtype=torch.int32, device="cuda")
    kw = dict(row_map=torch.full((m,), -1, dtype=torch.int32, device="cuda"),
              row_pair=torch.empty(0, dtype=torch.int32, device="cuda"))
    v = torch.empty(0, r, device="cuda")
    out = torch.full((m, n), F.MARK, dtype=dtype, device="cuda")
    hq.hq_lora(x, a, b, None, ends, out, base=base, v=v, **kw)
    assert torch.equal(out, base)
    hq.hq_lora(x, a, b, None, ends, out, **kw)
    assert torch.all(out == 0)
    dx = torch.full((m, k), F.MARK, dtype=dtype, device="cuda")
    da, db = torch.full((L, r, k), F.MARK, device="cuda"), torch.full((L, n, r), F.MARK, device="cuda")
    hq.hq_lora_backward(base, x, v, a, b, None, ends, da, db, dx=dx, base=x, **kw)
    assert torch.equal(dx, x) and torch.all(da == 0) and torch.all(db == 0)
    hq.hq_lora_backward(base, x, v, a, b, None, ends, da.fill_(3), db.fill_(3), accumulate=True, **kw)
    assert torch.all(da == 3) and torch.all(db == 3)
