"""Accumulating sums over the groups' rows on the GPU: a group without rows leaves
its result as it is, to the bit, and is not read or written at all."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import half as R
from tests import _block as H
from tests import _gpu as U
from tests import _half as F

pytestmark = pytest.mark.gpu

BF16, F32 = F.BF16, F.F32


# few tiles; more than a workgroup each, dealt longest first; more groups than are ordered, so that tiles of
# groups without rows come between the others
@pytest.mark.parametrize("sizes,m,n", [([0, 9, 0, 70, 0], 72, 136), ([0, 65, 0, 3] * 10, 520, 520),
                                       ([5, 0, 0, 66, 0] * 34, 264, 520)])
def test_results_of_empty_groups(sizes, m, n):
    what = f"group k, empty groups of {sizes[:5]} of {len(sizes)} {m}x{n}"
    U.banner(what)
    r = H.rng(what)
    ends = np.cumsum(sizes).astype(np.int32)
    a, av = F.halves(r, (int(ends[-1]), m), BF16)
    b, bv = F.halves(r, (int(ends[-1]), n), BF16, 0.1)
    out = torch.randn(len(sizes), m, n, device="cuda")
    empty = torch.from_numpy(np.array(sizes) == 0).cuda()
    out[empty] = -0.0                        # adding nothing would make it 0.0
    before = out.clone()
    hq.hq_half_group_k_gemm(a, b, H.dev(ends), out, accumulate=True)
    torch.cuda.synchronize()
    ref, mag = R.group_k(av, bv, ends)
    ref += F.f64(before)
    H.check(out, ref, F.product_bound(ref, mag, max(sizes), F32) + 2.0 ** -23 * np.abs(F.f64(before)), what)
    assert torch.equal(out.view(torch.int32)[empty], before.view(torch.int32)[empty]), f"{what}: changed"


def test_no_rows_at_all():
    U.banner("group k, no rows, accumulated")
    out = torch.full((3, 64, 64), -0.0, device="cuda")
    a = torch.empty(0, 64, dtype=BF16, device="cuda")
    hq.hq_half_group_k_gemm(a, a, torch.zeros(3, dtype=torch.int32, device="cuda"), out, accumulate=True)
    assert torch.signbit(out).all()
