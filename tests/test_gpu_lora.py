"""Low-rank adapters and their gradients on the GPU against float64."""
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

# m, adapters, n, k, r, who has which adapter
CASES = [
    (1, 1, 8, 8, 8, "all"), (1, 8, 512, 640, 16, "all"), (3, 2, 24, 136, 8, "mixed"), (64, 32, 520, 264, 16, "mixed"),
    (65, 5, 72, 1032, 24, "runs"), (130, 1, 264, 72, 64, "all"), (300, 3, 136, 520, 128, "runs"),
    (257, 700, 64, 64, 8, "mixed"), (50, 4, 128, 128, 16, "none"), (200, 6, 40, 48, 136, "mixed"),
    (33, 2, 1544, 16, 512, "runs"), (600, 2, 384, 1024, 32, "one"), (0, 3, 64, 64, 16, "all"),
    # both inner sums in many slices; few tokens an adapter; more columns than a workgroup has at once
    (700, 2, 4104, 4168, 16, "runs"), (40, 5, 264, 6152, 16, "mixed"), (20, 4, 6152, 520, 200, "mixed"),
    (30, 3, 1096, 520, 56, "all"), (1600, 100, 2056, 72, 32, "mixed"), (3000, 2, 6152, 40, 80, "mixed"),
    (1500, 1, 136, 2568, 24, "runs"),
]


def _owners(r, m, L, kind):
    if kind == "none":
        return np.full(m, -1, np.int64)
    if kind == "one":
        return np.full(m, L - 1, np.int64)
    if kind == "runs":                      # requests of consecutive tokens
        ids = np.repeat(r.integers(-1, L, m), r.integers(1, 70, m))[:m]
        return ids.astype(np.int64)
    ids = r.integers(0, L, m)
    return ids if kind == "all" else np.where(r.random(m) < 0.2, r.choice([-1, L, 2 ** 40], m), ids)


class Case:
    def __init__(self, what, m, L, n, k, r, kind, dtype, align=1):
        g = H.rng(what)
        self.what, self.m, self.L, self.n, self.k, self.r, self.dtype = what, m, L, n, k, r, dtype
        ids = _owners(g, m, L, kind)
        self.owner = np.where((ids >= 0) & (ids < L), ids, -1)
        if align == 1:
            self.ends, self.map, self.pair = hq.lora_plan(H.dev(ids), L)
        else:
            self.map, self.pair, self.ends, _ = hq.moe_sort(H.dev(ids).view(-1, 1), L, align)
        self.places = self.pair.numel()
        self.x, self.xv = F.halves(g, (m, k), dtype)
        self.dy, self.dyv = F.halves(g, (m, n), dtype, 0.1)
        self.a, self.av = F.halves(g, (L, r, k), dtype, k ** -0.5)
        self.b, self.bv = F.halves(g, (L, n, r), dtype, r ** -0.5)
        self.base, self.basev = F.halves(g, (m, n), dtype)
        self.dbase, self.dbasev = F.halves(g, (m, k), dtype, 0.1)
        self.scale = g.uniform(0.25, 2.0, L).astype(np.float32)
        self.sd = H.dev(self.scale)
        self.kw = dict(row_map=self.map, row_pair=self.pair)

    def ws(self, back=False):
        size = (hq.hq_lora_backward_workspace_size if back else hq.hq_lora_workspace_size)(
            self.m, self.n, self.k, self.r, self.L, self.places)
        return torch.full((size,), 0xEE, dtype=torch.uint8, device="cuda")          # its contents do not matter

    def by_place(self, v):
        """Token values [m, r] -> [places, r], zeros where there is no token."""
        out = np.zeros((self.places, v.shape[1]))
        pair = self.pair.cpu().numpy()
        out[pair >= 0] = v[pair[pair >= 0]]
        return out


def _share_bound(ref, mag, inner, r, dtype):
    """Both FP32 sums (inner and r terms, a split's parts among them), the inner
    sums taken to 16 bits, scale and base; then one rounding."""
    return ((inner + r + 32) * 2.0 ** -23 + 2.0 ** -16) * mag + H.UNIT[dtype] * np.abs(ref) + H.FLOOR[dtype]


@pytest.mark.parametrize("m,L,n,k,r,kind", CASES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_forward(m, L, n, k, r, kind, dtype):
    what = f"lora m={m} L={L} n={n} k={k} r={r} {kind} {dtype}"
    U.banner(what)
    c = Case(what, m, L, n, k, r, kind, dtype)
    ref = R.lora(c.xv, c.av, c.bv, c.scale, c.owner, c.basev)
    bound = _share_bound(ref["out"], ref["mag"], k, r, dtype)
    whole, out = F.marked((m, n), dtype)
    wv, v = F.marked((c.places, r), F32)
    hq.hq_lora(c.x, c.a, c.b, c.sd, c.ends, out, base=c.base, v=v, workspace=c.ws(), **c.kw)
    torch.cuda.synchronize()
    F.untouched(whole, what)
    F.untouched(wv, what)
    H.check(out, ref["out"], bound, what)
    none = H.dev(c.owner < 0)
    assert torch.equal(out[none], c.base[none])
    used = c.pair.cpu().numpy() >= 0
    assert torch.all(v[H.dev(~used)] == F.MARK), f"{what}: places without a token"
    want = c.by_place(ref["v"])[used]
    H.check(F.f64(v)[used], want, F.product_bound(want, c.by_place(ref["vmag"])[used], k, F32), f"{what}: v")
    # without v, in place
    out2 = c.base.clone()
    hq.hq_lora(c.x, c.a, c.b, c.sd, c.ends, out2, base=out2, workspace=c.ws(), **c.kw)
    assert torch.equal(out, out2)
    # without a base and a scale: the share alone
    ref = R.lora(c.xv, c.av, c.bv, np.ones(L), c.owner, None)
    hq.hq_lora(c.x, c.a, c.b, None, c.ends, out, workspace=c.ws(), **c.kw)
    H.check(out, ref["out"], _share_bound(ref["out"], ref["mag"], k, r, dtype), f"{what}: no base")
    assert torch.all(out[none] == 0)


@pytest.mark.parametrize("m,L,n,k,r,kind", CASES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_backward(m, L, n, k, r, kind, dtype):
    what = f"lora backward m={m} L={L} n={n} k={k} r={r} {kind} {dtype}"
    U.banner(what)
    c = Case(what, m, L, n, k, r, kind, dtype)
    vt = H.rng(what, "v").standard_normal((m, r)).astype(np.float32)
    vp = c.by_place(vt).astype(np.float32)
    vp[c.pair.cpu().numpy() < 0] = np.nan               # places without a token are not read into a sum
    ref = R.lora_backward(c.dyv, c.xv, vt, c.av, c.bv, c.scale, c.owner, c.dbasev)
    whole, dx = F.marked((m, k), dtype)
    wa, da = F.marked((L, r, k), F32)
    wb, db = F.marked((L, n, r), F32)
    args = (c.dy, c.x, H.dev(vp), c.a, c.b, c.sd, c.ends)
    hq.hq_lora_backward(*args, da, db, dx=dx, base=c.dbase, workspace=c.ws(True), **c.kw)
    torch.cuda.synchronize()
    for t in (whole, wa, wb):
        F.untouched(t, what)
    H.check(dx, ref["dx"], _share_bound(ref["dx"], ref["dxmag"], n, r, dtype), f"{what}: dx")
    none = H.dev(c.owner < 0)
    assert torch.equal(dx[none], c.dbase[none])
    most = int(np.bincount(c.owner[c.owner >= 0], minlength=1).max()) if m else 0
    H.check(da, ref["da"], F.product_bound(ref["da"], ref["damag"], n + most + 32, F32), f"{what}: da")
    H.check(db, ref["db"], F.product_bound(ref["db"], ref["dbmag"], most + 32, F32), f"{what}: db")
    # added to what is there, without dx, bit for bit the same sums again
    da2, db2 = torch.zeros_like(da), torch.zeros_like(db)
    hq.hq_lora_backward(*args, da2, db2, accumulate=True, workspace=c.ws(True), **c.kw)
    assert torch.equal(da, da2) and torch.equal(db, db2)
    hq.hq_lora_backward(*args, da2, db2, accumulate=True, workspace=c.ws(True), **c.kw)
    assert torch.equal(da + da, da2) and torch.equal(db + db, db2)
    # in place, and without a base
    dx2 = c.dbase.clone()
    hq.hq_lora_backward(*args, da, db, dx=dx2, base=dx2, workspace=c.ws(True), **c.kw)
    assert torch.equal(dx, dx2)
    hq.hq_lora_backward(*args, da, db, dx=dx2, workspace=c.ws(True), **c.kw)
    ref = R.lora_backward(c.dyv, c.xv, vt, c.av, c.bv, c.scale, c.owner, None)
    H.check(dx2, ref["dx"], _share_bound(ref["dx"], ref["dxmag"], n, r, dtype), f"{what}: dx alone")
    assert torch.all(dx2[none] == 0)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_padded_and_unsorted_plans(dtype):
    """Groups padded to whole blocks of 16 places, and tokens that lie in the order
    of their adapters, without a map: the same results."""
    what = f"lora plans {dtype}"
    U.banner(what)
    m, L, n, k, r = 150, 4, 136, 264, 16
    c = Case(what, m, L, n, k, r, "mixed", dtype, align=16)
    ref = R.lora(c.xv, c.av, c.bv, c.scale, c.owner, c.basev)
    out = torch.empty(m, n, dtype=dtype, device="cuda")
    v = torch.full((c.places, r), float("nan"), device="cuda")
    hq.hq_lora(c.x, c.a, c.b, c.sd, c.ends, out, base=c.base, v=v, workspace=c.ws(), **c.kw)
    H.check(out, ref["out"], _share_bound(ref["out"], ref["mag"], k, r, dtype), what)
    dx, da, db = torch.empty_like(c.x), torch.empty(L, r, k, device="cuda"), torch.empty(L, n, r, device="cuda")
    hq.hq_lora_backward(c.dy, c.x, v, c.a, c.b, c.sd, c.ends, da, db, dx=dx, base=c.dbase, workspace=c.ws(True), **c.kw)
    assert torch.isfinite(da).all() and torch.isfinite(db).all()
    # the same tokens in the order of their adapters
    order = np.argsort(np.where(c.owner < 0, L, c.owner), kind="stable")
    o = H.dev(order)
    ends = H.dev(np.cumsum(np.bincount(c.owner[c.owner >= 0], minlength=L)).astype(np.int32))
    out2, v2 = torch.empty_like(out), torch.zeros(m, r, device="cuda")
    ws = torch.empty(max(hq.hq_lora_workspace_size(m, n, k, r, L), hq.hq_lora_backward_workspace_size(m, n, k, r, L)),
                     dtype=torch.uint8, device="cuda")
    hq.hq_lora(c.x[o], c.a, c.b, c.sd, ends, out2, base=c.base[o], v=v2, workspace=ws)
    H.check(out2, ref["out"][order], _share_bound(ref["out"], ref["mag"], k, r, dtype)[order], what)
    dx2, da2, db2 = torch.empty_like(dx), torch.empty_like(da), torch.empty_like(db)
    hq.hq_lora_backward(c.dy[o], c.x[o], v2, c.a, c.b, c.sd, ends, da2, db2, dx=dx2, base=c.dbase[o], workspace=ws)
    rb = R.lora_backward(c.dyv, c.xv, ref["v"], c.av, c.bv, c.scale, c.owner, c.dbasev)
    # v itself is within k 2^-23 of its sum of magnitudes
    for got in ((dx, da, db), (dx2[torch.argsort(o)], da2, db2)):
        H.check(got[0], rb["dx"], _share_bound(rb["dx"], rb["dxmag"], n, r, dtype), f"{what}: dx")
        H.check(got[1], rb["da"], F.product_bound(rb["da"], rb["damag"], n + m + 32, F32), f"{what}: da")
        vm = R.lora_backward(c.dyv, c.xv, ref["vmag"], c.av, c.bv, c.scale, c.owner, None)["dbmag"]
        H.check(got[2], rb["db"], F.product_bound(rb["db"], vm, k + m + 64, F32), f"{what}: db")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_requests_stay_apart(dtype):
    """Infinities and NaN of a token, an adapter or the base reach that token's row
    and that adapter's gradients; those of tokens without an adapter reach none."""
    what = f"lora non-finite {dtype}"
    U.banner(what)
    m, L, n, k, r = 60, 4, 72, 136, 16
    c = Case(what, m, L, n, k, r, "mixed", dtype)
    own = c.owner
    t0, none = int(np.nonzero(own == 1)[0][0]), int(np.nonzero(own < 0)[0][0])
    c.x[t0, 3], c.x[none], c.dy[none] = float("nan"), float("inf"), float("nan")
    c.a[2, 1, 1] = float("inf")
    out, v = torch.empty(m, n, dtype=dtype, device="cuda"), torch.zeros(c.places, r, device="cuda")
    hq.hq_lora(c.x, c.a, c.b, c.sd, c.ends, out, base=c.base, v=v, workspace=c.ws(), **c.kw)
    bad = ~torch.isfinite(out)
    want = np.zeros((m, n), bool)
    want[t0], want[own == 2] = True, True
    assert not (bad.cpu().numpy() & ~want).any() and bad[t0].all()
    assert bad[H.dev(own == 2)].any(1).all()
    dx, da, db = torch.empty_like(c.x), torch.empty(L, r, k, device="cuda"), torch.empty(L, n, r, device="cuda")
    v = torch.randn(c.places, r, device="cuda")
    hq.hq_lora_backward(c.dy, c.x, v, c.a, c.b, c.sd, c.ends, da, db, dx=dx, workspace=c.ws(True), **c.kw)
    assert torch.isfinite(db).all()
    bad = ~torch.isfinite(da)
    want = np.zeros((L, r, k), bool)
    want[1, :, 3] = True
    assert np.array_equal(bad.cpu().numpy(), want)
    bad = ~torch.isfinite(dx).cpu().numpy()
    want = np.zeros((m, k), bool)
    want[own == 2, 1] = True
    assert np.array_equal(bad, want)


def test_values_of_every_size():
    """Inner sums from 1e-6 to 1e6 in one batch: each row of FP16 results keeps its
    precision, and nothing overflows on the way."""
    what = "lora magnitudes"
    U.banner(what)
    m, L, n, k, r = 48, 3, 64, 64, 16
    for dtype in (BF16, F16):
        c = Case(what + str(dtype), m, L, n, k, r, "all", dtype)
        size = 10.0 ** np.linspace(-4, 4, m)
        x = (c.xv * size[:, None] * 0.1)
        c.x = torch.from_numpy(x).to(dtype).cuda()
        c.a = (c.a.float() * 8).to(dtype)
        c.b = (c.b.float() * 2.0 ** -7).to(dtype)
        ref = R.lora(F.f64(c.x), F.f64(c.a), F.f64(c.b), c.scale, c.owner, None)
        out, v = torch.empty(m, n, dtype=dtype, device="cuda"), torch.empty(m, r, device="cuda")
        hq.hq_lora(c.x, c.a, c.b, c.sd, c.ends, out, v=v, workspace=c.ws(), **c.kw)
        H.check(out, ref["out"], _share_bound(ref["out"], ref["mag"], k, r, dtype), what)
        dy = (c.dyv * size[::-1, None] * 0.01)
        c.dy = torch.from_numpy(dy).to(dtype).cuda()
        dx, da, db = torch.empty_like(c.x), torch.empty(L, r, k, device="cuda"), torch.empty(L, n, r, device="cuda")
        hq.hq_lora_backward(c.dy, c.x, v, c.a, c.b, c.sd, c.ends, da, db, dx=dx, workspace=c.ws(True), **c.kw)
        vt = F.f64(v)[c.map.cpu().numpy()]
        rb = R.lora_backward(F.f64(c.dy), F.f64(c.x), vt, F.f64(c.a), F.f64(c.b), c.scale, c.owner, None)
        H.check(dx, rb["dx"], _share_bound(rb["dx"], rb["dxmag"], n, r, dtype), f"{what}: dx")
        H.check(da, rb["da"], F.product_bound(rb["da"], rb["damag"], n + m + 32, F32), f"{what}: da")
        H.check(db, rb["db"], F.product_bound(rb["db"], rb["dbmag"], m + 32, F32), f"{what}: db")


def test_gradients_against_differences():
    """The gradients as derivatives of the float64 forward: sum(dy * out) moves by
    <gradient, d> along a direction d (out is linear in x, A and B each, so the
    difference is exact up to the gradients' own errors)."""
    what = "lora differences"
    U.banner(what)
    m, L, n, k, r = 40, 3, 72, 56, 8
    c = Case(what, m, L, n, k, r, "mixed", F16)
    one = R.lora(c.xv, c.av, c.bv, c.scale, c.owner, None)
    v = H.dev(c.by_place(one["v"]).astype(np.float32))
    dx, da, db = torch.empty_like(c.x), torch.empty(L, r, k, device="cuda"), torch.empty(L, n, r, device="cuda")
    hq.hq_lora_backward(c.dy, c.x, v, c.a, c.b, c.sd, c.ends, da, db, dx=dx, workspace=c.ws(True), **c.kw)
    g = H.rng(what, "d")
    loss = (one["out"] * c.dyv).sum()
    for got, at, rel in ((dx, 0, 2.0 ** -11), (da, 1, 2.0 ** -20), (db, 2, 2.0 ** -20)):
        args = [c.xv, c.av, c.bv]
        d = g.standard_normal(args[at].shape)
        args[at] = args[at] + d
        moved = (R.lora(*args, c.scale, c.owner, None)["out"] * c.dyv).sum() - loss
        grad = F.f64(got)
        tol = (rel + 200 * 2.0 ** -23) * np.abs(grad * d).sum() * 4
        assert abs((grad * d).sum() - moved) <= tol


def test_streams_and_graphs():
    """On a side stream, and captured into two graphs with a workspace each: replays
    with eager work between them give the eager bits, for new inputs and plans."""
    U.banner("lora graph")
    what = "lora graph"
    m, L, n, k, r = 200, 6, 264, 520, 16
    c = Case(what, m, L, n, k, r, "mixed", BF16)

    def once(ws, wb):
        out, v = torch.empty(m, n, dtype=BF16, device="cuda"), torch.zeros(m, r, device="cuda")
        hq.hq_lora(c.x, c.a, c.b, c.sd, c.ends, out, base=c.base, v=v, workspace=ws, **c.kw)
        dx, da, db = torch.empty_like(c.x), torch.empty(L, r, k, device="cuda"), torch.empty(L, n, r, device="cuda")
        hq.hq_lora_backward(c.dy, c.x, v, c.a, c.b, c.sd, c.ends, da, db, dx=dx, base=c.dbase, workspace=wb, **c.kw)
        return out, dx, da, db

    eager = [t.clone() for t in once(c.ws(), c.ws(True))]
    side = torch.cuda.Stream()
    ws, wb = c.ws(), c.ws(True)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = once(ws, wb)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(eager, got):
        assert torch.equal(x, y)
    spaces = [(c.ws(), c.ws(True)) for _ in range(2)]
    graphs, outs = [], []
    for s in spaces:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(once(*s))
        graphs.append(graph)
    g = H.rng(what, "ids")
    for i in range(4):
        c.x.copy_(torch.randn(m, k, device="cuda"))
        for dst, src in zip((c.ends, c.map, c.pair), hq.lora_plan(H.dev(g.integers(-1, L, m)), L)):
            dst.copy_(src)
        want = [t.clone() for t in once(ws, wb)]
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            for x, y in zip(o, want):
                assert torch.equal(x, y), f"replay {i}"


def test_two_calls_at_once():
    """Two batches on two streams, a workspace each, give what they give alone."""
    what = "lora two streams"
    U.banner(what)
    cases = [Case(what + str(i), m, L, n, k, r, "mixed", BF16) for i, (m, L, n, k, r) in
             enumerate([(500, 3, 1544, 2056, 16), (90, 40, 2056, 4104, 32)])]

    def run(c, ws, wb):
        out, v = torch.empty(c.m, c.n, dtype=BF16, device="cuda"), torch.zeros(c.places, c.r, device="cuda")
        hq.hq_lora(c.x, c.a, c.b, c.sd, c.ends, out, base=c.base, v=v, workspace=ws, **c.kw)
        dx = torch.empty_like(c.x)
        da, db = torch.empty(c.L, c.r, c.k, device="cuda"), torch.empty(c.L, c.n, c.r, device="cuda")
        hq.hq_lora_backward(c.dy, c.x, v, c.a, c.b, c.sd, c.ends, da, db, dx=dx, base=c.dbase, workspace=wb, **c.kw)
        return out, dx, da, db

    spaces = [(c.ws(), c.ws(True)) for c in cases]
    alone = [run(c, *s) for c, s in zip(cases, spaces)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for c, s, stream in zip(cases, spaces, streams):
            with torch.cuda.stream(stream):
                got.append(run(c, *s))
        torch.cuda.synchronize()
        for want, have in zip(alone, got):
            for x, y in zip(want, have):
                assert torch.equal(x, y)
