"""Block-128 products on the GPU in every plan of _block_plans.py: whole outputs
against float64 products of the decoded operands, samples of them against the
oracle, and nothing written around the output or in rows that have no group.

Codes are normal ones, scales spread over a factor of four; FP16 results a second
time with scales that keep them below an infinity.  The bound is the FP32
sum's (see _block.product_bound).  Where the FP8 matrix instructions make the
inner sums, each is off by 1.5e-5 of its norm, 1.7e-4 for unit values, and those
errors are independent: over nkb >= 4 blocks their sum is below a twentieth of the
bound, which grows with nkb and not with its root."""
import numpy as np
import pytest
import torch

import fp4_gemm_moe_amd as hq
from oracle import block as B
from oracle import formats as F
from tests import _block as H
from tests import _block_plans as P
from tests import _gpu as U

pytestmark = pytest.mark.gpu

MARK = -77.0


def _operand(g, rows, k, scale_rows):
    """Codes [rows, k] of normal values and their scales [scale_rows, ceil(k / 128)]."""
    q = torch.randn((rows, k), generator=g, device="cuda").mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), 0.5 + 1.5 * torch.rand((scale_rows, -(-k // 128)), generator=g, device="cuda")


def _values(q, sf, block_rows):
    table = torch.from_numpy(F.e4m3_decode(np.arange(256, dtype=np.uint8))).cuda()
    f = sf.double().repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(block_rows, 0)[:q.shape[0]]
    return table[q.int()] * f


def _hold(out, a, sa, b, sb, what, add=0.0):
    """out (float64 of the result) against a b^T + add, whole and by the oracle's sample."""
    k = a.shape[1]
    x, y = _values(a, sa, 1), _values(b, sb, 128)
    ref, mag = x @ y.t().contiguous(), x.abs() @ y.abs().t().contiguous()
    bound = (132 + -(-k // 128)) * 2.0 ** -23 * mag + H.UNIT[out.dtype] * (ref + add).abs() + H.FLOOR[out.dtype]
    if add:
        bound += 2.0 ** -23 * (ref.abs() + add)
    got, bound = out.double(), bound * (1 + 2.0 ** -7)
    err = (got - (ref + add)).abs()
    bad = ~(err <= bound)
    if out.dtype is P.F16:          # from 65520 on the nearest FP16 value is an infinity
        bad &= ~((got == torch.inf * ref.sign()) & (ref.abs() + bound >= 65520))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, first at "
                           f"{bad.nonzero()[0].tolist()}, worst {float((err / bound).nan_to_num(9e9).max()):.3g} of it")
    r = H.rng(what)
    rows = torch.from_numpy(np.unique(r.integers(0, a.shape[0], 3))).cuda()
    nb = int(r.integers(0, sb.shape[0]))
    cols = slice(128 * nb, min(128 * nb + 128, b.shape[0]))
    c = lambda t: t.cpu().numpy()  # noqa: E731
    want, m = B.gemm(c(a[rows]), c(sa[rows]), c(b[cols]), c(sb[nb:nb + 1]))
    assert np.allclose(c(ref[rows, cols]), want, rtol=0, atol=1e-9 * np.max(m)), f"{what}: float64 form"


def _out(rows, n, dtype, fill=float("nan")):
    """An output with marked values around it."""
    whole = torch.full((rows * n + 256,), MARK, dtype=dtype, device="cuda")
    out = whole[128:128 + rows * n].view(rows, n)
    out.fill_(fill)
    return whole, out


def _untouched(whole, what):
    assert torch.all(whole[:128] == MARK) and torch.all(whole[-128:] == MARK), f"{what}: written around the output"


def _generator(what):
    U.banner(what)
    return torch.Generator(device="cuda").manual_seed(int(H.rng(what).integers(0, 2 ** 62)))


@pytest.mark.parametrize("m,n,k,dtype,ws,plan", P.DENSE)
def test_dense(m, n, k, dtype, ws, plan):
    what = f"{m}x{n}x{k} {dtype}: {plan}"
    g = _generator(what)
    (a, sa), (b, sb) = _operand(g, m, k, m), _operand(g, n, k, -(-n // 128))
    need = hq.hq_block_gemm_workspace_size(m, n, k, out_dtype=dtype) if ws else 0
    assert (need > 0) == any(s != "s1" for s in plan.split() if s[0] == "s")
    space = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    for scale, add in [(1, 0.0)] + [(1, 3.0)] * (dtype is P.F32) + [(2.0 ** -12, 0.0)] * (dtype is P.F16):
        sa = sa * scale
        whole, out = _out(m, n, dtype, add if add else float("nan"))
        hq.hq_block_gemm(a, sa, b, sb, out, accumulate=add > 0, workspace=space[:need] if ws else None)
        torch.cuda.synchronize()
        _hold(out, a, sa, b, sb, what, add)
        _untouched(whole, what)
        assert torch.all(space[need:] == 0xFF), f"{what}: written past the workspace"


@pytest.mark.parametrize("batch,m,n,k,dtype,ws,plan", P.BATCH)
def test_batch(batch, m, n, k, dtype, ws, plan):
    what = f"{batch} x {m}x{n}x{k} {dtype}: {plan}"
    g = _generator(what)
    A, W = [_operand(g, m, k, m) for _ in range(batch)], [_operand(g, n, k, -(-n // 128)) for _ in range(batch)]
    args = [torch.stack([x[i] for x in s]) for s in (A, W) for i in (0, 1)]
    space = torch.empty(hq.hq_block_gemm_workspace_size(m, n, k, batch, dtype), dtype=torch.uint8, device="cuda")
    for scale in (1, 2.0 ** -12) if dtype is P.F16 else (1,):
        args[1] = args[1] * scale
        whole, out = _out(batch * m, n, dtype)
        hq.hq_block_gemm(*args, out.view(batch, m, n), workspace=space if ws else None)
        torch.cuda.synchronize()
        for i in range(batch):
            _hold(out[i * m:(i + 1) * m], A[i][0], args[1][i], *W[i], f"{what} item {i}")
        _untouched(whole, what)


@pytest.mark.parametrize("counts,spare,n,k,dtype,plan", P.CONTIGUOUS)
def test_contiguous(counts, spare, n, k, dtype, plan):
    what = f"contiguous {counts}+{spare} {n}x{k} {dtype}: {plan}"
    g = _generator(what)
    rows, ends = sum(counts) + spare, np.cumsum(counts)
    a, sa = _operand(g, rows, k, rows)
    W = [_operand(g, n, k, -(-n // 128)) for _ in counts]
    whole, out = _out(rows, n, dtype, MARK)
    hq.hq_block_group_contiguous_gemm(a, sa, torch.stack([w[0] for w in W]), torch.stack([w[1] for w in W]),
                                      U.dev_i32(ends, "cuda"), out)
    torch.cuda.synchronize()
    for e, (c, end) in enumerate(zip(counts, ends)):
        if c:
            r = slice(int(end) - c, int(end))
            _hold(out[r], a[r], sa[r], *W[e], f"{what} group {e}")
    assert torch.all(out[int(ends[-1]):] == MARK), f"{what}: rows past the last end written"
    _untouched(whole, what)


@pytest.mark.parametrize("counts,slot,n,k,dtype,plan", P.MASKED)
def test_masked(counts, slot, n, k, dtype, plan):
    what = f"masked {counts}/{slot} {n}x{k} {dtype}: {plan}"
    g = _generator(what)
    E = len(counts)
    a, sa = _operand(g, E * slot, k, E * slot)
    W = [_operand(g, n, k, -(-n // 128)) for _ in counts]
    for e, c in enumerate(counts):              # rows without a token hold anything
        a[e * slot + c:(e + 1) * slot] = 0x7F
        sa[e * slot + c:(e + 1) * slot] = float("nan")
    for scale in (1, 2.0 ** -12) if dtype is P.F16 else (1,):
        sa = sa * scale
        whole, out = _out(E * slot, n, dtype, MARK)
        hq.hq_block_group_masked_gemm(a, sa, torch.stack([w[0] for w in W]), torch.stack([w[1] for w in W]),
                                      U.dev_i32(counts, "cuda"), out, slot)
        torch.cuda.synchronize()
        for e, c in enumerate(counts):
            if c:
                r = slice(e * slot, e * slot + c)
                _hold(out[r], a[r], sa[r], *W[e], f"{what} group {e}")
            assert torch.all(out[e * slot + c:(e + 1) * slot] == MARK), f"{what}: padding of group {e} written"
        _untouched(whole, what)


@pytest.mark.parametrize("blocks,m,n,dtype,plan", P.GROUP_K)
def test_group_k(blocks, m, n, dtype, plan):
    what = f"group_k {blocks} {m}x{n} {dtype}: {plan}"
    g = _generator(what)
    k, ends = 128 * sum(blocks), np.cumsum(blocks)
    (a, sa), (b, sb) = _operand(g, m, k, m), _operand(g, n, k, -(-n // 128))
    whole, out = _out(len(blocks) * m, n, dtype)
    hq.hq_block_group_k_gemm(a, sa, b, sb, U.dev_i32(128 * ends, "cuda"), out.view(len(blocks), m, n))
    torch.cuda.synchronize()
    for e, (c, end) in enumerate(zip(blocks, ends)):
        part = out[e * m:(e + 1) * m]
        if c == 0:
            assert torch.all(part == 0)
            continue
        lo, hi = int(end) - c, int(end)
        _hold(part, a[:, 128 * lo:128 * hi], sa[:, lo:hi], b[:, 128 * lo:128 * hi], sb[:, lo:hi], f"{what} group {e}")
    _untouched(whole, what)
