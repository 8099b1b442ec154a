"""Cases for measuring the block-128 FP8 products and the token dispatch around them.

FP8 values are E4M3 codes with one FP32 scale for each block of 128: 1 x 128 along K for
activations and gradients, 128 x 128 for weights.  A block's scale is
s = max(amax / 448, 2^-126) and its codes are the E4M3 values nearest to x / s.

Kinds of cases:
  quant      BF16 rows or weight matrices (optionally transposed) -> codes and scales
  gemm       out[m, n] = sum over K blocks of sa[m, kb] sb[n / 128, kb] (a[m] . b[n])_kb
  contig     the same per expert over rows sorted by expert (cumulative ends)
  masked     the same per expert over padded slots with counts of valid rows
  kgroup     weight gradients: per expert a product that sums over the expert's rows
  dispatch   tokens sorted by expert, rows copied there and quantised
  combine    expert rows summed back into tokens with their routing weights
  combine_bwd  its gradient: for the expert rows and for the weights
"""
import math

import torch

own = False

BLK = 128
TINY = 2.0 ** -126
F8 = torch.float8_e4m3fn
#: Workspaces that a program keeps for the calls of one stream.
GEMM_WORKSPACE, SORT_WORKSPACE = 64 << 20, 1 << 20


def listed():
    return [
        # activations of a long prefill, before an expert or dense product
        {"name": "quant_rows_65536x4096", "kind": "quant", "batch": 1, "m": 65536, "k": 4096, "two_d": False,
         "transpose": False, "dtype": "bf16"},
        # expert weights for the gradient with respect to activations: 128 x 128 blocks, transposed
        {"name": "quant_weights_t_32x4096x1536", "kind": "quant", "batch": 32, "m": 4096, "k": 1536, "two_d": True,
         "transpose": True, "dtype": "bf16"},
        # one token of decoding through a dense layer
        {"name": "gemm_1x17408x5120", "kind": "gemm", "m": 1, "n": 17408, "k": 5120, "out": "bf16"},
        # a decoding batch, odd row count, long K, few output tiles
        {"name": "gemm_77x5120x17408", "kind": "gemm", "m": 77, "n": 5120, "k": 17408, "out": "bf16"},
        # a prefill chunk through a dense layer
        {"name": "gemm_4096x17408x5120", "kind": "gemm", "m": 4096, "n": 17408, "k": 5120, "out": "bf16"},
        # the gate|up product of a MoE layer over a long prefill: 16384 tokens, top 4 of 32 experts
        {"name": "contig_16384t4_e32_3072x4096", "kind": "contig", "tokens": 16384, "topk": 4, "experts": 32,
         "align": 128, "n": 3072, "k": 4096, "out": "bf16"},
        # decoding over padded expert slots, weights read once
        {"name": "masked_e64_256_4096x7168", "kind": "masked", "experts": 64, "max_m": 256, "n": 4096, "k": 7168,
         "out": "bf16"},
        # the weight gradient of the down projection over a training batch
        {"name": "kgroup_16384t4_e32_4096x1536", "kind": "kgroup", "tokens": 16384, "topk": 4, "experts": 32,
         "m": 4096, "n": 1536},
        # the dispatch of a small decoding batch, where latency counts
        {"name": "dispatch_64t8_e64_7168", "kind": "dispatch", "tokens": 64, "topk": 8, "experts": 64, "align": 1,
         "hidden": 7168, "dtype": "bf16"},
        # the dispatch of a long prefill or training batch, groups padded to whole blocks
        {"name": "dispatch_16384t4_e32_4096", "kind": "dispatch", "tokens": 16384, "topk": 4, "experts": 32,
         "align": 128, "hidden": 4096, "dtype": "bf16"},
        # expert outputs back into tokens
        {"name": "combine_1024t8_e16_2048", "kind": "combine", "tokens": 1024, "topk": 8, "experts": 16, "align": 1,
         "hidden": 2048, "dtype": "bf16"},
        # the gradient of the combination over a training batch
        {"name": "combine_bwd_16384t4_e32_4096", "kind": "combine_bwd", "tokens": 16384, "topk": 4, "experts": 32,
         "align": 128, "hidden": 4096, "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    kind = rng.choice(["quant", "gemm", "gemm", "contig", "masked", "kgroup", "dispatch", "combine", "combine_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    out = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    while True:
        if kind == "quant":
            t = rng.random() < 0.5
            c = {"kind": kind, "batch": log(1, 32), "m": log(32, 16384, 32) if t else log(1, 16384),
                 "k": log(256, 17408, 32), "two_d": rng.random() < 0.5, "transpose": t, "dtype": dtype}
            big = c["batch"] * c["m"] * c["k"] > 65536 * 4096
        elif kind == "gemm":
            c = {"kind": kind, "m": log(1, 4096), "n": log(128, 17408, 8), "k": log(256, 17408, 32), "out": out}
            big = c["m"] * c["n"] * c["k"] > 4096 * 17408 * 5120
        elif kind == "contig":
            c = {"kind": kind, "tokens": log(16, 16384), "topk": rng.randint(1, 8), "experts": log(8, 128),
                 "align": rng.choice([1, 128]), "n": log(512, 7168, 8), "k": log(512, 7168, 32), "out": out}
            big = (c["tokens"] * c["topk"] * c["n"] * c["k"] > 65536 * 4096 * 2048
                   or c["experts"] * c["n"] * c["k"] > 32 * 3072 * 4096)
        elif kind == "masked":
            c = {"kind": kind, "experts": log(8, 128), "max_m": log(16, 512), "n": log(512, 7168, 8),
                 "k": log(512, 7168, 32), "out": out}
            big = c["experts"] * c["n"] * c["k"] > 64 * 4096 * 7168 or c["experts"] * c["max_m"] > 32768
        elif kind == "kgroup":
            c = {"kind": kind, "tokens": log(128, 16384), "topk": rng.randint(1, 8), "experts": log(8, 64),
                 "m": log(512, 7168, 8), "n": log(512, 7168, 8)}
            big = (c["tokens"] * c["topk"] * c["m"] * c["n"] > 65536 * 4096 * 2048
                   or c["experts"] * c["m"] * c["n"] > 32 * 4096 * 1536)
        else:
            c = {"kind": kind, "tokens": log(1, 16384), "topk": rng.randint(1, 8), "experts": log(8, 256),
                 "align": rng.choice([1, 128]), "hidden": log(512, 7168, 32), "dtype": dtype}
            big = (c["tokens"] * c["topk"] + c["experts"] * c["align"]) * c["hidden"] > 67840 * 4096
        if not big:
            return c


# ------------------------------------------------------------------ inputs
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _values(g, shape, sigma, dtype=torch.bfloat16):
    """Normal values, every 97th column eight times larger (the outlier channels of activations)."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(sigma)
    x[..., ::97] *= 8.0
    return x.to(dtype)


def _routing(g, tokens, topk, experts):
    """Top-k experts of each token under uneven expert popularity, a few tokens dropped (-1), and
    normalised weights."""
    logits = torch.randn((tokens, experts), generator=g, device="cuda")
    logits += 0.7 * torch.randn((1, experts), generator=g, device="cuda")
    k = min(topk, experts)
    w, ids = logits.topk(k, dim=1)
    drop = torch.rand((tokens, k), generator=g, device="cuda") < 0.01
    return torch.where(drop, -1, ids).contiguous(), torch.softmax(w, 1).contiguous()


def _max_rows(tokens, topk, experts, align):
    pairs = tokens * topk
    return (pairs + min(experts, pairs) * (align - 1)) // align * align


def _codes(g, rows, k, batch=None):
    """Codes [.., rows, k] and the scales of their 1 x 128 blocks."""
    x = _values(g, (rows, k) if batch is None else (batch, rows, k), 1.0)
    return _quantise(x, False)


def _weights(g, batch, n, k):
    q, s = _quantise(torch.randn((batch, n, k), generator=g, device="cuda").mul_(0.02).bfloat16(), True)
    return q, s


def prepare(case, seed):
    g, c, kind = _gen(seed), case, case["kind"]
    dev = "cuda"
    s = {"c": c}
    if kind == "quant":
        shape = (c["batch"], c["m"], c["k"])
        sigma = 0.02 if c["two_d"] else 1.0
        s["x"] = _values(g, shape, sigma, DTYPES[c["dtype"]])
        rows, cols = (c["k"], c["m"]) if c["transpose"] else (c["m"], c["k"])
        s["q"] = torch.zeros((c["batch"], rows, cols), dtype=torch.uint8, device=dev)
        srows = -(-rows // BLK) if c["two_d"] else rows
        s["sf"] = torch.zeros((c["batch"], srows, -(-cols // BLK)), device=dev)
    elif kind == "gemm":
        s["a"], s["sa"] = _codes(g, c["m"], c["k"])
        b, sb = _weights(g, 1, c["n"], c["k"])
        s["b"], s["sb"] = b[0], sb[0]
        s["ws"] = torch.zeros(GEMM_WORKSPACE, dtype=torch.uint8, device=dev)
        s["out"] = torch.zeros((c["m"], c["n"]), dtype=DTYPES[c["out"]], device=dev)
    elif kind == "contig":
        ids, _ = _routing(g, c["tokens"], c["topk"], c["experts"])
        rows = _max_rows(c["tokens"], ids.shape[1], c["experts"], c["align"])
        _, _, s["ends"], _ = _plain_sort(ids, c["experts"], c["align"], rows)
        s["host_ends"] = s["ends"].tolist()
        s["a"], s["sa"] = _codes(g, rows, c["k"])
        s["b"], s["sb"] = _weights(g, c["experts"], c["n"], c["k"])
        s["out"] = torch.zeros((rows, c["n"]), dtype=DTYPES[c["out"]], device=dev)
    elif kind == "masked":
        E, M = c["experts"], c["max_m"]
        s["counts"] = torch.randint(0, M + 1, (E,), generator=g, device=dev, dtype=torch.int32)
        a, sa = _codes(g, M, c["k"], E)
        s["a"], s["sa"] = a.view(E * M, -1), sa.view(E * M, -1)
        s["b"], s["sb"] = _weights(g, E, c["n"], c["k"])
        s["out"] = torch.zeros((E * M, c["n"]), dtype=DTYPES[c["out"]], device=dev)
    elif kind == "kgroup":
        ids, _ = _routing(g, c["tokens"], c["topk"], c["experts"])
        rows = _max_rows(c["tokens"], ids.shape[1], c["experts"], BLK)
        _, _, s["ends"], _ = _plain_sort(ids, c["experts"], BLK, rows)
        s["host_ends"] = s["ends"].tolist()
        s["a"], s["sa"] = _quantise(_values(g, (c["m"], rows), 0.01), False)
        s["b"], s["sb"] = _quantise(_values(g, (c["n"], rows), 1.0), True)
        s["out"] = torch.zeros((c["experts"], c["m"], c["n"]), device=dev)
    else:
        E, h, dt = c["experts"], c["hidden"], DTYPES[c["dtype"]]
        s["ids"], s["w"] = _routing(g, c["tokens"], c["topk"], E)
        T, k = s["ids"].shape
        rows = _max_rows(T, k, E, c["align"])
        s["rows"] = rows
        if kind == "dispatch":
            s["x"] = _values(g, (T, h), 1.0, dt)
            s["row_map"] = torch.zeros((T, k), dtype=torch.int32, device=dev)
            s["row_pair"] = torch.zeros(rows, dtype=torch.int32, device=dev)
            s["ends"] = torch.zeros(E, dtype=torch.int32, device=dev)
            s["counts"] = torch.zeros(E, dtype=torch.int32, device=dev)
            s["q"] = torch.zeros((rows, h), dtype=torch.uint8, device=dev)
            s["sf"] = torch.zeros((rows, -(-h // BLK)), device=dev)
            s["ws"] = torch.zeros(SORT_WORKSPACE, dtype=torch.uint8, device=dev)
        else:
            s["row_map"], _, s["ends"], s["counts"] = _plain_sort(s["ids"], E, c["align"], rows)
            s["y"] = _values(g, (rows, h), 1.0, dt)
            if kind == "combine":
                s["out"] = torch.zeros((T, h), dtype=dt, device=dev)
            else:
                s["dout"] = _values(g, (T, h), 0.01, dt)
                s["dy"] = torch.zeros((rows, h), dtype=dt, device=dev)
                s["dw"] = torch.zeros((T, k), device=dev)
    return s


# ------------------------------------------------------------------ plain forms
def _quantise(x, two_d):
    """x [.., m, k] -> E4M3 codes (uint8, as x) and FP32 scales [.., m or m / 128, k / 128]."""
    lead, m, k = x.shape[:-2], x.shape[-2], x.shape[-1]
    bm = BLK if two_d else 1
    pm, pk = -m % bm, -k % BLK
    v = x.float()
    if pm or pk:
        v = torch.nn.functional.pad(v, (0, pk, 0, pm))
    v = v.reshape(lead + ((m + pm) // bm, bm, (k + pk) // BLK, BLK))
    s = (v.abs().amax((-3, -1)) / 448.0).clamp(min=TINY)
    q = (v / s[..., :, None, :, None]).clamp(-448.0, 448.0).to(F8)
    q = q.reshape(lead + (m + pm, k + pk))[..., :m, :k]
    return q.contiguous().view(torch.uint8), s


def _values_of(q, s, two_d):
    """Codes and scales -> FP32 values."""
    m, k = q.shape[-2], q.shape[-1]
    f = s.repeat_interleave(BLK, -1)[..., :k]
    if two_d:
        f = f.repeat_interleave(BLK, -2)[..., :m, :]
    return q.view(F8).float() * f


def _plain_sort(ids, experts, align, rows):
    flat = ids.reshape(-1)
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(experts, device=ids.device)).sum(0)
    padded = (counts + align - 1) // align * align
    ends = padded.cumsum(0)
    # sorted place -> row: the group's padded start plus the rank inside the group
    shift = (ends - padded) - (counts.cumsum(0) - counts)
    shift = torch.cat([shift, shift.new_zeros(1)])
    sorted_key = key[order]
    row = torch.arange(n, device=ids.device) + shift[sorted_key]
    row = torch.where(sorted_key < experts, row, rows)
    row_pair = torch.full((rows + 1,), -1, device=ids.device)
    row_pair[row] = order
    row_map = torch.empty(n, dtype=torch.int32, device=ids.device)
    row_map[order] = torch.where(row < rows, row, -1).int()
    return row_map.view(ids.shape), row_pair[:rows].int(), ends.int(), counts.int()


def _grouped(s, c, ends):
    """a's rows in runs that end at `ends`, each times its own matrix; rows past the last end stay zero."""
    a = _values_of(s["a"], s["sa"], False)
    b = _values_of(s["b"], s["sb"], True)
    sizes = [e - f for e, f in zip(ends, [0] + ends)]
    parts = [x @ w.t() for x, w in zip(a[:ends[-1]].split(sizes), b)]
    return torch.cat(parts + [a.new_zeros((a.shape[0] - ends[-1], c["n"]))]).to(DTYPES[c["out"]])


def run(state):
    return (_own if own else _plain)(state)


def _plain(s):
    c, kind = s["c"], s["c"]["kind"]
    if kind == "quant":
        q, sf = _quantise(s["x"].transpose(1, 2) if c["transpose"] else s["x"], c["two_d"])
        return {"q": q.view(F8), "sf": sf}
    if kind == "gemm":
        a, b = _values_of(s["a"], s["sa"], False), _values_of(s["b"], s["sb"], True)
        return {"out": (a @ b.t()).to(DTYPES[c["out"]])}
    if kind == "contig":
        return {"out": _grouped(s, c, s["host_ends"])}
    if kind == "masked":
        E, M = c["experts"], c["max_m"]
        a, b = _values_of(s["a"], s["sa"], False).view(E, M, -1), _values_of(s["b"], s["sb"], True)
        y = torch.bmm(a, b.transpose(1, 2).contiguous())
        y *= (torch.arange(M, device=y.device) < s["counts"][:, None])[..., None]
        return {"out": y.view(E * M, -1).to(DTYPES[c["out"]])}
    if kind == "kgroup":
        a, b, ends = _values_of(s["a"], s["sa"], False), _values_of(s["b"], s["sb"], True), s["host_ends"]
        return {"out": torch.stack([a[:, f:e] @ b[:, f:e].t() for f, e in zip([0] + ends, ends)])}
    if kind == "dispatch":
        row_map, row_pair, ends, counts = _plain_sort(s["ids"], c["experts"], c["align"], s["rows"])
        used = torch.arange(s["rows"], device=row_map.device) < ends[-1]
        x = s["x"].float()[(row_pair.long() // row_map.shape[1]).clamp(min=0)]
        q, sf = _quantise(x * (row_pair >= 0)[:, None], False)
        return {"row_map": row_map, "row_pair": row_pair, "ends": ends, "counts": counts,
                "q": q.view(F8), "sf": sf * used[:, None]}
    T, k = s["row_map"].shape
    here = (s["row_map"] >= 0)
    at = s["row_map"].long().clamp(min=0)
    if kind == "combine":
        rows = s["y"].float()[at.view(-1)].view(T, k, -1)
        return {"out": (rows * (s["w"] * here)[..., None]).sum(1).to(s["y"].dtype)}
    w = s["w"] * here
    dout = s["dout"].float()
    rows = s["y"].float()[at.view(-1)].view(T, k, -1)
    dw = (rows * dout[:, None]).sum(-1) * here
    dy = dout.new_zeros((s["rows"] + 1, dout.shape[1]))
    dy[torch.where(here, at, s["rows"]).view(-1)] = (dout[:, None] * w[..., None]).view(T * k, -1)
    return {"dy": dy[:-1].to(s["y"].dtype), "dw": dw}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import fp4_gemm_moe_amd as hq
    c, kind = s["c"], s["c"]["kind"]
    if kind == "quant":
        hq.hq_block_quant(s["x"], s["q"], s["sf"], block_2d=c["two_d"], transpose=c["transpose"])
        return {"q": s["q"].view(F8), "sf": s["sf"]}
    if kind == "gemm":
        hq.hq_block_gemm(s["a"], s["sa"], s["b"], s["sb"], s["out"], workspace=s["ws"])
        return {"out": s["out"]}
    if kind == "contig":
        hq.hq_block_group_contiguous_gemm(s["a"], s["sa"], s["b"], s["sb"], s["ends"], s["out"])
        return {"out": s["out"]}
    if kind == "masked":
        hq.hq_block_group_masked_gemm(s["a"], s["sa"], s["b"], s["sb"], s["counts"], s["out"], c["max_m"])
        return {"out": s["out"]}
    if kind == "kgroup":
        hq.hq_block_group_k_gemm(s["a"], s["sa"], s["b"], s["sb"], s["ends"], s["out"])
        return {"out": s["out"]}
    if kind == "dispatch":
        hq.hq_moe_sort(s["ids"], c["experts"], c["align"], s["row_map"], s["row_pair"], s["ends"], s["counts"],
                       workspace=s["ws"])
        hq.hq_moe_permute_block_quant(s["x"], s["row_map"], s["ends"], s["counts"], s["q"], s["sf"])
        return {"row_map": s["row_map"], "row_pair": s["row_pair"], "ends": s["ends"], "counts": s["counts"],
                "q": s["q"].view(F8), "sf": s["sf"]}
    if kind == "combine":
        hq.hq_moe_combine(s["y"], s["row_map"], s["w"], s["out"])
        return {"out": s["out"]}
    hq.hq_moe_combine_backward(s["dout"], s["y"], s["row_map"], s["w"], s["ends"], s["counts"], s["dy"], s["dw"])
    return {"dy": s["dy"], "dw": s["dw"]}


# ------------------------------------------------------------------ 64-bit definition
def _blocks64(x, bm):
    """x [m, k] float64: the block scales, and the values of x / s rounded to E4M3, both float64."""
    m, k = x.shape
    sf = torch.empty((-(-m // bm), -(-k // BLK)), dtype=torch.float64, device=x.device)
    q = torch.empty_like(x)
    for j in range(sf.shape[1]):
        col = x[:, j * BLK:(j + 1) * BLK]
        top = col.abs().amax(1)
        if bm > 1:
            top = torch.nn.functional.pad(top, (0, -m % bm)).view(-1, bm).amax(1)
        sf[:, j] = torch.clamp(top / 448.0, min=TINY)
        v = (col / sf[:, j].repeat_interleave(bm)[:m, None]).clamp(-448.0, 448.0)
        # the E4M3 grid: three bits below the leading one, and steps of 2^-9 below 2^-6
        e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(e - 3)
        q[:, j * BLK:(j + 1) * BLK] = torch.round(v / step) * step
    return q, sf


def _e4m3_table(device):
    v = []
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        mag = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v.append(-mag if code & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device=device)


def _product64(a, sa, b, sb):
    """a [m, k], b [n, k] codes with their scales (1 x 128, 128 x 128) -> [m, n] in 64 bits."""
    table = _e4m3_table(a.device)
    out = torch.zeros((a.shape[0], b.shape[0]), dtype=torch.float64, device=a.device)
    for j in range(sa.shape[1]):
        x = table[a[:, j * BLK:(j + 1) * BLK].long()] * sa[:, j, None].double()
        y = table[b[:, j * BLK:(j + 1) * BLK].long()]
        y = y * sb[:, j].double().repeat_interleave(BLK)[:b.shape[0], None]
        out.addmm_(x, y.t())
    return out


def exact(case, seed):
    s, c, kind = prepare(case, seed), case, case["kind"]
    if kind == "quant":
        qs, sfs = [], []
        for x in s["x"]:
            q, sf = _blocks64((x.t() if c["transpose"] else x).double(), BLK if c["two_d"] else 1)
            qs.append(q)
            sfs.append(sf)
        return {"q": torch.stack(qs), "sf": torch.stack(sfs)}
    if kind == "gemm":
        return {"out": _product64(s["a"], s["sa"], s["b"], s["sb"])}
    if kind in ("contig", "masked"):
        out = torch.zeros((s["a"].shape[0], c["n"]), dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            if kind == "contig":
                lo, hi = (s["host_ends"][e - 1] if e else 0), s["host_ends"][e]
            else:
                lo = e * c["max_m"]
                hi = lo + int(s["counts"][e])
            out[lo:hi] = _product64(s["a"][lo:hi], s["sa"][lo:hi], s["b"][e], s["sb"][e])
        return {"out": out}
    if kind == "kgroup":
        out = torch.zeros((c["experts"], c["m"], c["n"]), dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            lo, hi = (s["host_ends"][e - 1] if e else 0), s["host_ends"][e]
            if hi > lo:
                out[e] = _product64(s["a"][:, lo:hi], s["sa"][:, lo // BLK:hi // BLK],
                                    s["b"][:, lo:hi], s["sb"][:, lo // BLK:hi // BLK])
        return {"out": out}
    if kind == "dispatch":
        q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        sf = torch.zeros(s["sf"].shape, dtype=torch.float64, device="cuda")
        xq, xs = _blocks64(s["x"].double(), 1)
        ids, row = s["ids"].cpu(), 0
        for e in range(c["experts"]):
            tokens = (ids == e).nonzero()[:, 0].to("cuda")     # token order, then slot order
            n = tokens.numel()
            q[row:row + n], sf[row:row + n] = xq[tokens], xs[tokens]
            last = row + -(-n // c["align"]) * c["align"]
            sf[row + n:last] = TINY
            row = last
        return {"row_map": None, "row_pair": None, "ends": None, "counts": None, "q": q, "sf": sf}
    if kind == "combine":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for j in range(s["w"].shape[1]):
            t = (s["row_map"][:, j] >= 0).nonzero()[:, 0]
            out[t] += s["w"][t, j, None].double() * s["y"][s["row_map"][t, j].long()].double()
        return {"out": out}
    dy = torch.zeros(s["dy"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")
    for j in range(s["w"].shape[1]):
        t = (s["row_map"][:, j] >= 0).nonzero()[:, 0]
        r, d = s["row_map"][t, j].long(), s["dout"][t].double()
        dy[r] = s["w"][t, j, None].double() * d
        dw[t, j] = (d * s["y"][r].double()).sum(1)
    return {"dy": dy, "dw": dw}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, kind = case, case["kind"]
    wide = {"bf16": 2, "fp16": 2, "fp32": 4}
    if kind == "quant":
        n = c["batch"] * c["m"] * c["k"]
        return {"bytes": n * 3 + 4 * n / (BLK * BLK if c["two_d"] else BLK), "flops": 2 * n}
    if kind == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": m * k * (1 + 4 / BLK) + n * k * (1 + 4 / BLK ** 2) + m * n * wide[c["out"]],
                "flops": 2 * m * n * k}
    if kind == "contig":
        r, n, k, E = c["tokens"] * min(c["topk"], c["experts"]), c["n"], c["k"], c["experts"]
        return {"bytes": r * k * (1 + 4 / BLK) + min(E, r) * n * k + r * n * wide[c["out"]], "flops": 2 * r * n * k}
    if kind == "masked":
        r, n, k = c["experts"] * c["max_m"] / 2, c["n"], c["k"]
        return {"bytes": r * k * (1 + 4 / BLK) + c["experts"] * n * k + r * n * wide[c["out"]], "flops": 2 * r * n * k}
    if kind == "kgroup":
        r, m, n = c["tokens"] * min(c["topk"], c["experts"]), c["m"], c["n"]
        return {"bytes": r * (m + n) + 4 * r * m / BLK + c["experts"] * m * n * 4, "flops": 2 * r * m * n}
    T, k, h = c["tokens"], min(c["topk"], c["experts"]), c["hidden"]
    if kind == "dispatch":
        return {"bytes": T * h * 2 + T * k * (h * (1 + 4 / BLK) + 16), "flops": 2 * T * h}
    if kind == "combine":
        return {"bytes": T * k * (h * 2 + 8) + T * h * 2, "flops": 2 * T * k * h}
    return {"bytes": T * h * 2 + T * k * (h * 4 + 12), "flops": 3 * T * k * h}
