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
