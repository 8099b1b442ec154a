"""Low-rank adapters on the GPU near the limits of their launches: 2^28 tokens that
have adapters, and nearly 2^30 of which 16 have one."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from tests import _block as H
from tests import _gpu as U
from tests import _half as F

pytestmark = pytest.mark.gpu

BF16, F32 = F.BF16, F.F32
L, N, K, R = 3, 8, 8, 8


def _randn(*shape):
    return torch.empty(shape, dtype=BF16, device="cuda").normal_()


def _adapters():
    return _randn(L, R, K), _randn(L, N, R) * R ** -0.5


def _expected(x, base, w, v):
    """A token's row of base + (x w^T) v^T, and its bound (see test_gpu_lora.py)."""
    ref = F.f64(base) + (F.f64(w) @ F.f64(x)) @ F.f64(v).T
    mag = np.abs(F.f64(base)) + (np.abs(F.f64(w)) @ np.abs(F.f64(x))) @ np.abs(F.f64(v)).T
    return ref, ((16 + 32) * 2.0 ** -23 + 2.0 ** -16) * mag + H.UNIT[BF16] * np.abs(ref) + H.FLOOR[BF16]


def test_all_with_an_adapter():
    U.banner("lora of 2^28 tokens")
    m = 1 << 28
    x, base = _randn(m, K), _randn(m, N)
    a, b = _adapters()
    ends = torch.tensor([5, (1 << 27) + 77, m - 100], dtype=torch.int32, device="cuda")
    out = torch.empty_like(base)
    ws = torch.empty(hq.hq_lora_workspace_size(m, N, K, R, L), dtype=torch.uint8, device="cuda")
    hq.hq_lora(x, a, b, None, ends, out, base=base, workspace=ws)
    for t in (0, 4, 5, 1 << 20, (1 << 27) + 76, (1 << 27) + 77, m - 12345, m - 101):
        g = int((ends <= t).sum())
        ref, bound = _expected(x[t], base[t], a[g], b[g])
        H.check(out[t], ref, bound, f"token {t}")
    assert torch.equal(out[m - 100:], base[m - 100:])
    for lo in range(0, m, 1 << 25):             # nothing was left out: the share is not zero but by chance
        part = slice(lo, min(lo + (1 << 25), m - 100))
        assert bool((out[part] != base[part]).any(1).float().mean() > 0.99), f"tokens from {lo} on"


def test_few_with_an_adapter():
    U.banner("lora gradients of nearly 2^30 tokens")
    m, places = (1 << 30) - (1 << 16), 16
    x, dy = _randn(m, K), _randn(m, N)
    a, b = _adapters()
    who = torch.tensor([0, 63, 64, 1 << 20, (1 << 28) + 1, (1 << 29) - 1, 1 << 29, m - 1000, m - 65, m - 64, m - 2, m - 1],
                       dtype=torch.int32, device="cuda")
    ends = torch.tensor([3, 3, 12], dtype=torch.int32, device="cuda")
    row_pair = torch.full((places,), -1, dtype=torch.int32, device="cuda")
    row_pair[:12] = who
    row_map = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    row_map[who.long()] = torch.arange(12, dtype=torch.int32, device="cuda")
    v = torch.randn(places, R, device="cuda")
    dx = torch.empty_like(x)
    da, db = torch.empty(L, R, K, device="cuda"), torch.empty(L, N, R, device="cuda")
    ws = torch.empty(hq.hq_lora_backward_workspace_size(m, N, K, R, L, places), dtype=torch.uint8, device="cuda")
    hq.hq_lora_backward(dy, x, v, a, b, None, ends, da, db, dx=dx, base=x, row_map=row_map, row_pair=row_pair, workspace=ws)
    torch.cuda.synchronize()
    for i, t in enumerate(who.tolist()):
        g = 0 if i < 3 else 2
        ref, bound = _expected(dy[t], x[t], b[g].t().contiguous(), a[g].t().contiguous())
        H.check(dx[t], ref, bound, f"token {t}")
    dx[who.long()] = x[who.long()]
    for lo in range(0, m, 1 << 27):
        assert torch.equal(dx[lo:lo + (1 << 27)], x[lo:lo + (1 << 27)]), f"tokens from {lo} on"
    for g, at in ((0, who[:3]), (2, who[3:])):
        d, y = F.f64(dy[at.long()]), F.f64(x[at.long()])
        vv = F.f64(v[:3] if g == 0 else v[3:12])
        H.check(db[g], d.T @ vv, F.product_bound(d.T @ vv, np.abs(d).T @ np.abs(vv), 12 + 32, F32), f"db {g}")
        u, um = d @ F.f64(b[g]), np.abs(d) @ np.abs(F.f64(b[g]))
        H.check(da[g], u.T @ y, F.product_bound(u.T @ y, um.T @ np.abs(y), N + 12 + 32, F32), f"da {g}")
    assert torch.all(da[1] == 0) and torch.all(db[1] == 0)
