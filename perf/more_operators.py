"""Cases for measuring the 16-bit products grouped by expert, SwiGLU with its gradient, and
low-rank adapters beside a shared projection.

Kinds of cases:
  contig     out[r] = a[r] b[g]^T for the rows r of expert g, sorted by expert (cumulative ends);
             with "t" the weights are [k, n] (the gradient for the activations)
  masked     the same over padded expert slots with counts of valid rows
  kgroup     out[g] = sum over the rows r of expert g of a[r]^T b[r] (the gradient for the weights)
  swiglu     y = up * silu(gate) of rows [gate | up]
  swiglu_bwd the gradient for [gate | up], and y once more (the down product's operand)
  lora       out[t] = base[t] + scale[g] (x[t] A[g]^T) B[g]^T for the adapter g of token t
  lora_bwd   the gradients for x, A and B

Values are bfloat16 or float16.  The adapter A[g] is [r, k] and B[g] is [n, r]; a token's
adapter comes from its request, and tokens of requests without one keep the base projection.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one token of decoding through the gate half of its 8 experts, where latency counts
        {"name": "contig_1t8_e16_1536x2048", "kind": "contig", "tokens": 1, "topk": 8, "experts": 16, "n": 1536,
         "k": 2048, "t": False, "dtype": "fp16", "out": "half"},
        # the down projection of a MoE layer over a long prefill or training batch
        {"name": "contig_16384t4_e32_4096x1536", "kind": "contig", "tokens": 16384, "topk": 4, "experts": 32,
         "n": 4096, "k": 1536, "t": False, "dtype": "bf16", "out": "half"},
        # the gradient of that projection for its activations
        {"name": "contig_t_16384t4_e32_1536x4096", "kind": "contig", "tokens": 16384, "topk": 4, "experts": 32,
         "n": 1536, "k": 4096, "t": True, "dtype": "bf16", "out": "half"},
        # decoding over padded expert slots, weights read once
        {"name": "masked_e64_64_4096x2048", "kind": "masked", "experts": 64, "max_m": 64, "n": 4096, "k": 2048,
         "t": False, "dtype": "bf16", "out": "half"},
        # the gradient of the down projection for its weights, over a training batch
        {"name": "kgroup_16384t4_e32_4096x1536", "kind": "kgroup", "tokens": 16384, "topk": 4, "experts": 32,
         "m": 4096, "n": 1536, "dtype": "bf16", "out": "fp32"},
        # a decoding batch between the two products: 64 tokens, 8 experts each
        {"name": "swiglu_512x2048", "kind": "swiglu", "rows": 512, "h": 2048, "dtype": "fp16"},
        # a training batch's gradient, 16384 tokens and 4 experts each
        {"name": "swiglu_bwd_65536x1536", "kind": "swiglu_bwd", "rows": 65536, "h": 1536, "dtype": "bf16"},
        # one request's next token beside a square projection
        {"name": "lora_1x5120x5120_a8_r16", "kind": "lora", "m": 1, "n": 5120, "k": 5120, "adapters": 8, "r": 16,
         "requests": 1, "save": False, "dtype": "bf16"},
        # a decoding batch of 64 requests, 32 adapters, beside a feed-forward projection
        {"name": "lora_64x17408x5120_a32_r16", "kind": "lora", "m": 64, "n": 17408, "k": 5120, "adapters": 32,
         "r": 16, "requests": 64, "save": False, "dtype": "bf16"},
        # a prefill chunk of several requests beside the same projection, x A^T kept for a backward pass
        {"name": "lora_4096x17408x5120_a8_r64", "kind": "lora", "m": 4096, "n": 17408, "k": 5120, "adapters": 8,
         "r": 64, "requests": 11, "save": True, "dtype": "bf16"},
        # a small training step, odd row count, three adapters of rank 8
        {"name": "lora_bwd_1000x1536x2048_a3_r8", "kind": "lora_bwd", "m": 1000, "n": 1536, "k": 2048, "adapters": 3,
         "r": 8, "requests": 7, "dtype": "fp16"},
        # a training batch of several adapters at once
        {"name": "lora_bwd_16384x4096x4096_a8_r16", "kind": "lora_bwd", "m": 16384, "n": 4096, "k": 4096,
         "adapters": 8, "r": 16, "requests": 32, "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    kind = rng.choice(["contig", "contig", "masked", "kgroup", "swiglu", "swiglu_bwd", "lora", "lora", "lora_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    out = rng.choice(["half", "half", "fp32"])
    while True:
        if kind == "contig":
            c = {"kind": kind, "tokens": log(1, 16384), "topk": rng.randint(1, 8), "experts": log(8, 128),
                 "n": log(512, 7168, 8), "k": log(512, 7168, 8), "t": rng.random() < 0.5, "dtype": dtype, "out": out}
            big = (c["tokens"] * c["topk"] * c["n"] * c["k"] > 65536 * 4096 * 1536
                   or c["experts"] * c["n"] * c["k"] > 64 * 4096 * 2048)
        elif kind == "masked":
            c = {"kind": kind, "experts": log(8, 128), "max_m": log(1, 512), "n": log(512, 7168, 8),
                 "k": log(512, 7168, 8), "t": rng.random() < 0.5, "dtype": dtype, "out": out}
            big = (c["experts"] * c["n"] * c["k"] > 64 * 4096 * 2048
                   or c["experts"] * c["max_m"] * c["n"] * c["k"] > 65536 * 4096 * 1536)
        elif kind == "kgroup":
            c = {"kind": kind, "tokens": log(128, 16384), "topk": rng.randint(1, 8), "experts": log(8, 64),
                 "m": log(512, 7168, 8), "n": log(512, 7168, 8), "dtype": dtype, "out": out}
            big = (c["tokens"] * c["topk"] * c["m"] * c["n"] > 65536 * 4096 * 1536
                   or c["experts"] * c["m"] * c["n"] > 64 * 4096 * 2048)
        elif kind in ("swiglu", "swiglu_bwd"):
            c = {"kind": kind, "rows": log(1, 65536), "h": log(256, 17408, 8), "dtype": dtype}
            big = c["rows"] * c["h"] > 65536 * 1536
        else:
            fwd = kind == "lora"
            m = log(1, 16384) if fwd else log(64, 16384)
            c = {"kind": kind, "m": m, "n": log(512, 17408, 8), "k": log(512, 17408, 8),
                 "adapters": log(1, 64), "r": rng.choice([8, 16, 16, 24, 32, 64, 128]),
                 "requests": rng.randint(max(1, m // 2), m) if m <= 256 else rng.randint(1, 64), "dtype": dtype}
            if fwd:
                c["save"] = m > 256
            big = m * (c["n"] + c["k"]) > (4096 * 22528 if fwd else 16384 * 8192)
        if not big:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _values(g, shape, sigma, dtype):
    """Normal values, every 97th column eight times larger (the outlier channels of activations)."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(sigma)
    x[..., ::97] *= 8.0
    return x.to(dtype)


def _weights(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").mul_(0.02).to(dtype)


def _routed_ends(g, tokens, topk, experts):
    """Cumulative ends of the experts' rows under uneven popularity, a few pairs dropped."""
    logits = torch.randn((tokens, experts), generator=g, device="cuda")
    logits += 0.7 * torch.randn((1, experts), generator=g, device="cuda")
    k = min(topk, experts)
    ids = logits.topk(k, dim=1).indices
    ids = torch.where(torch.rand((tokens, k), generator=g, device="cuda") < 0.01, experts, ids)
    ends = (ids.reshape(-1, 1) == torch.arange(experts, device="cuda")).sum(0).cumsum(0).int()
    return tokens * k, ends


def _adapter_plan(g, m, adapters, requests):
    """Tokens of consecutive requests, each request with one adapter or (one in sixteen) none, sorted by
    adapter in their order: the token's place, the place's token, and the adapters' cumulative ends."""
    cut = torch.randperm(max(m - 1, 1), generator=g, device="cuda")[:requests - 1] + 1
    starts = torch.zeros(m + 1, dtype=torch.int64, device="cuda")
    starts[cut] = 1
    request = starts[:m].cumsum(0)
    adapter = torch.randint(0, adapters, (m,), generator=g, device="cuda")
    none = torch.rand(m, generator=g, device="cuda") < 1 / 16
    none[0] = False
    key = torch.where(none, adapters, adapter)[request]
    order = torch.sort(key, stable=True).indices
    ends = (key[:, None] == torch.arange(adapters, device="cuda")).sum(0).cumsum(0).int()
    last = int(ends[-1])
    row_pair = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    row_pair[:last] = order[:last].int()
    row_map = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    row_map[order[:last]] = torch.arange(last, dtype=torch.int32, device="cuda")
    return row_map, row_pair, ends


def prepare(case, seed):
    g, c, kind, dev = _gen(seed), case, case["kind"], "cuda"
    dt = DTYPES[c["dtype"]]
    s = {"c": c}
    if kind in ("contig", "masked"):
        out = torch.float32 if c["out"] == "fp32" else dt
        E, wide = c["experts"], (c["k"], c["n"]) if c["t"] else (c["n"], c["k"])
        if kind == "contig":
            rows, s["ends"] = _routed_ends(g, c["tokens"], c["topk"], E)
            s["host_ends"] = s["ends"].tolist()
        else:
            rows = E * c["max_m"]
            s["counts"] = torch.randint(0, c["max_m"] + 1, (E,), generator=g, device=dev, dtype=torch.int32)
        s["a"] = _values(g, (rows, c["k"]), 1.0, dt)
        s["b"] = _weights(g, (E,) + wide, dt)
        s["out"] = torch.zeros((rows, c["n"]), dtype=out, device=dev)
    elif kind == "kgroup":
        rows, s["ends"] = _routed_ends(g, c["tokens"], c["topk"], c["experts"])
        s["host_ends"] = s["ends"].tolist()
        s["a"] = _values(g, (rows, c["m"]), 0.01, dt)
        s["b"] = _values(g, (rows, c["n"]), 1.0, dt)
        s["out"] = torch.zeros((c["experts"], c["m"], c["n"]), device=dev,
                               dtype=torch.float32 if c["out"] == "fp32" else dt)
    elif kind in ("swiglu", "swiglu_bwd"):
        s["x"] = _values(g, (c["rows"], 2 * c["h"]), 1.0, dt)
        s["y"] = torch.zeros((c["rows"], c["h"]), dtype=dt, device=dev)
        if kind == "swiglu_bwd":
            s["dy"] = _values(g, (c["rows"], c["h"]), 0.01, dt)
            s["dx"] = torch.zeros((c["rows"], 2 * c["h"]), dtype=dt, device=dev)
    else:
        L, r = c["adapters"], c["r"]
        s["map"], s["pair"], s["ends"] = _adapter_plan(g, c["m"], L, min(c["requests"], c["m"]))
        s["host_ends"] = s["ends"].tolist()
        s["x"] = _values(g, (c["m"], c["k"]), 1.0, dt)
        s["a"] = torch.randn((L, r, c["k"]), generator=g, device=dev).mul_(c["k"] ** -0.5).to(dt)
        s["b"] = _weights(g, (L, c["n"], r), dt)
        s["scale"] = torch.rand(L, generator=g, device=dev) * 2 + 0.25
        if kind == "lora":
            s["base"] = _values(g, (c["m"], c["n"]), 1.0, dt)
            s["out"] = torch.zeros((c["m"], c["n"]), dtype=dt, device=dev)
            s["v"] = torch.zeros((c["m"], r), device=dev) if c["save"] else None
        else:
            s["dy"] = _values(g, (c["m"], c["n"]), 0.01, dt)
            s["base"] = _values(g, (c["m"], c["k"]), 0.01, dt)          # the projection's own gradient for x
            s["dx"] = torch.zeros((c["m"], c["k"]), dtype=dt, device=dev)
            s["v"] = torch.zeros((c["m"], r), device=dev)
            for e, at, rows in _adapter_rows(s):
                s["v"][at] = s["x"][rows].float() @ s["a"][e].float().t()
            s["da"] = torch.zeros((L, r, c["k"]), device=dev)
            s["db"] = torch.zeros((L, c["n"], r), device=dev)
        if own:
            import fp4_gemm_moe_amd as hq
            size = hq.hq_lora_workspace_size if kind == "lora" else hq.hq_lora_backward_workspace_size
            s["ws"] = torch.zeros(size(c["m"], c["n"], c["k"], r, L), dtype=torch.uint8, device=dev)
    return s


def _adapter_rows(s):
    """For each adapter in use: its number, its places and their tokens."""
    lo = 0
    for e, hi in enumerate(s["host_ends"]):
        if hi > lo:
            yield e, slice(lo, hi), s["pair"][lo:hi].long()
        lo = hi


# ------------------------------------------------------------------ plain forms
def run(state):
    return (_own if own else _plain)(state)


def _plain(s):
    c, kind = s["c"], s["c"]["kind"]
    if kind == "contig":
        a, ends = s["a"].float(), s["host_ends"]
        out = torch.zeros((a.shape[0], c["n"]), device=a.device)
        for e, (lo, hi) in enumerate(zip([0] + ends, ends)):
            if hi > lo:
                w = s["b"][e].float()
                out[lo:hi] = a[lo:hi] @ (w if c["t"] else w.t())
        return {"out": out.to(s["out"].dtype)}
    if kind == "masked":
        E, M = c["experts"], c["max_m"]
        b = s["b"].float()
        y = torch.bmm(s["a"].float().view(E, M, -1), b if c["t"] else b.transpose(1, 2).contiguous())
        y *= (torch.arange(M, device=y.device) < s["counts"][:, None])[..., None]
        return {"out": y.view(E * M, -1).to(s["out"].dtype)}
    if kind == "kgroup":
        a, b, ends = s["a"].float(), s["b"].float(), s["host_ends"]
        out = torch.stack([a[lo:hi].t() @ b[lo:hi] for lo, hi in zip([0] + ends, ends)])
        return {"out": out.to(s["out"].dtype)}
    if kind == "swiglu":
        gate, up = s["x"].float().split(c["h"], 1)
        return {"y": (up * gate * torch.sigmoid(gate)).to(s["y"].dtype)}
    if kind == "swiglu_bwd":
        gate, up = s["x"].float().split(c["h"], 1)
        dy, sig = s["dy"].float(), torch.sigmoid(gate)
        dgate = dy * up * sig * (1.0 + gate * (1.0 - sig))
        dx = torch.cat([dgate, dy * gate * sig], 1)
        return {"dx": dx.to(s["dx"].dtype), "y": (up * gate * sig).to(s["y"].dtype)}
    if kind == "lora":
        out = s["base"].float()
        v = torch.zeros((c["m"], c["r"]), device=out.device)
        for e, at, rows in _adapter_rows(s):
            v[at] = s["x"][rows].float() @ s["a"][e].float().t()
            out[rows] += s["scale"][e] * (v[at] @ s["b"][e].float().t())
        out = {"out": out.to(s["out"].dtype)}
        return {**out, "v": v} if c["save"] else out
    dx = s["base"].float()
    da, db = torch.zeros_like(s["da"]), torch.zeros_like(s["db"])
    for e, at, rows in _adapter_rows(s):
        dy, f = s["dy"][rows].float(), s["scale"][e]
        u = dy @ s["b"][e].float()
        dx[rows] += f * (u @ s["a"][e].float())
        da[e] = f * (u.t() @ s["x"][rows].float())
        db[e] = f * (dy.t() @ s["v"][at])
    return {"dx": dx.to(s["dx"].dtype), "da": da, "db": db}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import fp4_gemm_moe_amd as hq
    c, kind = s["c"], s["c"]["kind"]
    if kind == "contig":
        hq.hq_half_group_contiguous_gemm(s["a"], s["b"], s["ends"], s["out"], transpose=c["t"])
        return {"out": s["out"]}
    if kind == "masked":
        hq.hq_half_group_masked_gemm(s["a"], s["b"], s["counts"], s["out"], c["max_m"], transpose=c["t"])
        return {"out": s["out"]}
    if kind == "kgroup":
        hq.hq_half_group_k_gemm(s["a"], s["b"], s["ends"], s["out"])
        return {"out": s["out"]}
    if kind == "swiglu":
        hq.hq_swiglu(s["x"], s["y"])
        return {"y": s["y"]}
    if kind == "swiglu_bwd":
        hq.hq_swiglu_backward(s["dy"], s["x"], s["dx"], y=s["y"])
        return {"dx": s["dx"], "y": s["y"]}
    if kind == "lora":
        hq.hq_lora(s["x"], s["a"], s["b"], s["scale"], s["ends"], s["out"], base=s["base"], row_map=s["map"],
                   row_pair=s["pair"], v=s["v"], workspace=s["ws"])
        return {"out": s["out"], "v": s["v"]} if c["save"] else {"out": s["out"]}
    hq.hq_lora_backward(s["dy"], s["x"], s["v"], s["a"], s["b"], s["scale"], s["ends"], s["da"], s["db"], dx=s["dx"],
                        base=s["base"], row_map=s["map"], row_pair=s["pair"], workspace=s["ws"])
    return {"dx": s["dx"], "da": s["da"], "db": s["db"]}


# ------------------------------------------------------------------ 64-bit definition
def exact(case, seed):
    s, c, kind = prepare(case, seed), case, case["kind"]
    d = torch.float64
    if kind in ("contig", "masked"):
        out = torch.zeros(s["out"].shape, dtype=d, device="cuda")
        for e in range(c["experts"]):
            if kind == "contig":
                lo, hi = (s["host_ends"][e - 1] if e else 0), s["host_ends"][e]
            else:
                lo = e * c["max_m"]
                hi = lo + int(s["counts"][e])
            w = s["b"][e].double()
            out[lo:hi] = s["a"][lo:hi].double().mm(w if c["t"] else w.t())
        return {"out": out}
    if kind == "kgroup":
        out = torch.zeros(s["out"].shape, dtype=d, device="cuda")
        for e in range(c["experts"]):
            lo, hi = (s["host_ends"][e - 1] if e else 0), s["host_ends"][e]
            out[e].addmm_(s["a"][lo:hi].double().t(), s["b"][lo:hi].double())
        return {"out": out}
    if kind in ("swiglu", "swiglu_bwd"):
        h = c["h"]
        y = torch.empty((c["rows"], h), dtype=d, device="cuda")
        dx = torch.empty((c["rows"], 2 * h), dtype=d, device="cuda") if kind == "swiglu_bwd" else None
        for lo in range(0, c["rows"], 4096):
            x = s["x"][lo:lo + 4096].double()
            gate, up = x[:, :h], x[:, h:]
            e = torch.exp(-gate)
            y[lo:lo + 4096] = up * (gate / (1 + e))
            if dx is not None:
                dy = s["dy"][lo:lo + 4096].double()
                dx[lo:lo + 4096, :h] = dy * up * (1 + e + gate * e) / (1 + e) ** 2
                dx[lo:lo + 4096, h:] = dy * (gate / (1 + e))
        return {"y": y} if dx is None else {"dx": dx, "y": y}
    owner = torch.full((c["m"],), -1, dtype=torch.int64)
    for e in range(c["adapters"]):
        lo, hi = (s["host_ends"][e - 1] if e else 0), s["host_ends"][e]
        owner[s["pair"][lo:hi].long().cpu()] = e
    owner = owner.cuda()
    if kind == "lora":
        out = s["base"].double()
        v = torch.zeros((c["m"], c["r"]), dtype=d, device="cuda")
        for e in range(c["adapters"]):
            t = (owner == e).nonzero()[:, 0]
            p = s["x"][t].double().mm(s["a"][e].double().t())
            v[s["map"][t].long()] = p
            out[t] += p.mm(s["b"][e].double().t()) * s["scale"][e].double()
        return {"out": out, "v": v} if c["save"] else {"out": out}
    dx = s["base"].double()
    da = torch.zeros(s["da"].shape, dtype=d, device="cuda")
    db = torch.zeros(s["db"].shape, dtype=d, device="cuda")
    for e in range(c["adapters"]):
        t = (owner == e).nonzero()[:, 0]
        x, v, f = s["x"][t].double(), s["v"][s["map"][t].long()].double(), s["scale"][e].double()
        dy = s["dy"][t].double() * f
        u = dy.mm(s["b"][e].double())
        dx[t] += u.mm(s["a"][e].double())
        da[e] = u.t().mm(x)
        db[e] = dy.t().mm(v)
    return {"dx": dx, "da": da, "db": db}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, kind = case, case["kind"]
    if kind in ("contig", "masked"):
        E, n, k, wide = c["experts"], c["n"], c["k"], 4 if c["out"] == "fp32" else 2
        r = c["tokens"] * min(c["topk"], E) if kind == "contig" else E * c["max_m"] / 2
        return {"bytes": r * k * 2 + min(E, r) * n * k * 2 + r * n * wide, "flops": 2 * r * n * k}
    if kind == "kgroup":
        r, m, n = c["tokens"] * min(c["topk"], c["experts"]), c["m"], c["n"]
        return {"bytes": r * (m + n) * 2 + c["experts"] * m * n * (4 if c["out"] == "fp32" else 2),
                "flops": 2 * r * m * n}
    if kind in ("swiglu", "swiglu_bwd"):
        e = c["rows"] * c["h"]
        return {"bytes": 6 * e, "flops": 6 * e} if kind == "swiglu" else {"bytes": 12 * e, "flops": 16 * e}
    m, n, k, r = c["m"], c["n"], c["k"], c["r"]
    used = min(c["adapters"], c["requests"], m)
    if kind == "lora":
        return {"bytes": 2 * (m * k + 2 * m * n + used * r * (n + k)) + (4 * m * r if c["save"] else 0),
                "flops": 2 * m * r * (n + k) + m * n}
    return {"bytes": 2 * (m * n + 3 * m * k) + 4 * m * r + used * r * (n + k) * 2 + c["adapters"] * r * (n + k) * 4,
            "flops": 4 * m * r * (n + k) + m * k}
