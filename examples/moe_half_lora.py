"""A MoE feed-forward layer in 16 bits behind a frozen projection with low-rank
adapters, forward and backward.

    python examples/moe_half_lora.py [--tokens 4096] [--hidden 2048] [--inter 1536] [--experts 32] [--topk 4]
                                     [--adapters 8] [--rank 16]

AdaptedProjection: a weight in block-128 FP8 that stays as it is, and beside its
product each token's own adapter, out = x W^T + scale[g] (x A[g]^T) B[g]^T.
MoeHalf: tokens sorted by expert, gate|up product, SwiGLU, down product, summed
back with their routing weights, all in the type of the weights.  Backward:
the gradients of the adapters and of the experts' weights in FP32, those of the
tokens and routing weights.  Run as a script it compares both with a float32
network and times them; --tokens 1 is a decoding step.
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fp4_gemm_moe_amd as hq  # noqa: E402


def _bytes(n, like):
    return torch.empty(n, dtype=torch.uint8, device=like.device)


class AdaptedProjection:
    """w [n, k] quantised once in 128 x 128 blocks, a [L, r, k], b [L, n, r] and
    scale [L] (float32) of the adapters that train."""

    def __init__(self, w, a, b, scale):
        self.w, self.w_t = hq.block_quantize(w, block_2d=True), hq.block_quantize(w, block_2d=True, transpose=True)
        self.a, self.b, self.scale = a, b, scale
        (self.n, self.k), (self.adapters, self.rank) = w.shape, a.shape[:2]

    def forward(self, x, adapter_ids, train=True):
        """x [T, k], adapter_ids [T] int64 (-1: none) -> [T, n], and what the
        backward pass needs."""
        T = x.shape[0]
        ends, row_map, row_pair = plan = hq.lora_plan(adapter_ids, self.adapters)
        out = torch.empty((T, self.n), dtype=x.dtype, device=x.device)
        hq.hq_block_gemm(*hq.block_quantize(x), *self.w, out)
        v = torch.empty((T, self.rank), device=x.device) if train else None
        hq.hq_lora(x, self.a, self.b, self.scale, ends, out, base=out, row_map=row_map, row_pair=row_pair, v=v,
                   workspace=_bytes(hq.hq_lora_workspace_size(T, self.n, self.k, self.rank, self.adapters), x))
        return out, (x, v, plan)

    def backward(self, dout, saved):
        """The gradients (x, a, b) for out's gradient dout."""
        x, v, (ends, row_map, row_pair) = saved
        dx = torch.empty_like(x)
        hq.hq_block_gemm(*hq.block_quantize(dout), *self.w_t, dx)
        da, db = torch.empty(self.a.shape, device=x.device), torch.empty(self.b.shape, device=x.device)
        size = hq.hq_lora_backward_workspace_size(x.shape[0], self.n, self.k, self.rank, self.adapters)
        hq.hq_lora_backward(dout, x, v, self.a, self.b, self.scale, ends, da, db, dx=dx, base=dx, row_map=row_map,
                            row_pair=row_pair, workspace=_bytes(size, x))
        return dx, da, db


class MoeHalf:
    """w1 [E, 2 inter, hidden] (gate rows, then up rows) and w2 [E, hidden,
    inter], bfloat16 or float16."""

    def __init__(self, w1, w2):
        self.w1, self.w2 = w1, w2
        self.experts, n, self.hidden = w1.shape
        self.inter = n // 2

    def forward(self, x, ids, weights):
        """x [T, hidden], ids [T, topk] int64, weights [T, topk] float32 -> [T,
        hidden], and what the backward pass needs."""
        row_map, _, ends, counts = hq.moe_sort(ids, self.experts)
        rows = hq.moe_max_rows(*ids.shape, self.experts)
        xr, gu, a, y = (torch.empty((rows, w), dtype=x.dtype, device=x.device)
                        for w in (self.hidden, 2 * self.inter, self.inter, self.hidden))
        hq.hq_moe_permute(x, row_map, ends, counts, xr)
        hq.hq_half_group_contiguous_gemm(xr, self.w1, ends, gu)
        hq.hq_swiglu(gu, a, group_end=ends)
        hq.hq_half_group_contiguous_gemm(a, self.w2, ends, y)
        out = torch.empty_like(x)
        hq.hq_moe_combine(y, row_map, weights, out)
        return out, (xr, weights, row_map, ends, counts, gu, y)

    def backward(self, dout, saved):
        """The gradients (x, routing weights, w1, w2) for out's gradient dout."""
        xr, weights, row_map, ends, counts, gu, y = saved
        dy, dweights = torch.empty_like(y), torch.empty_like(weights)
        hq.hq_moe_combine_backward(dout, y, row_map, weights, ends, counts, dy, dweights)
        a = torch.empty((y.shape[0], self.inter), dtype=y.dtype, device=y.device)
        hq.hq_half_group_contiguous_gemm(dy, self.w2, ends, a, transpose=True)
        dgu = torch.empty_like(gu)
        hq.hq_swiglu_backward(a, gu, dgu, y=a, group_end=ends)       # a: its gradient, then its values again
        dxr = torch.empty_like(xr)
        hq.hq_half_group_contiguous_gemm(dgu, self.w1, ends, dxr, transpose=True)
        dx = torch.empty_like(dout)
        hq.hq_moe_combine(dxr, row_map, None, dx)
        dw1, dw2 = (torch.empty(w.shape, device=w.device) for w in (self.w1, self.w2))
        hq.hq_half_group_k_gemm(dgu, xr, ends, dw1)
        hq.hq_half_group_k_gemm(dy, a, ends, dw2)
        return dx, dweights, dw1, dw2


def reference(x, ids, weights, w1, w2):
    """The MoE layer expert by expert, in the precision of its arguments."""
    out = torch.zeros_like(x)
    m = w2.shape[2]
    for e in range(w1.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[t] @ w1[e].t()).split(m, 1)
        out = out.index_add(0, t, weights[t, j, None] * ((up * torch.nn.functional.silu(gate)) @ w2[e].t()))
    return out


def share(x, adapter_ids, scale, a, b):
    """The adapters' share, adapter by adapter."""
    out = x.new_zeros(x.shape[0], b.shape[1])
    for g in range(a.shape[0]):
        t = (adapter_ids == g).nonzero()[:, 0]
        out = out.index_add(0, t, scale[g] * ((x[t] @ a[g].t()) @ b[g].t()))
    return out


def network(tokens, hidden, inter, experts, topk, adapters, rank, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w = (rand(hidden, hidden) * hidden ** -0.5).to(dtype)
    a, b = (rand(adapters, rank, hidden) * hidden ** -0.5).to(dtype), (rand(adapters, hidden, rank) * rank ** -0.5).to(dtype)
    scale = torch.rand(adapters, generator=g, device="cuda") + 0.5
    w1 = (rand(experts, 2 * inter, hidden) * hidden ** -0.5).to(dtype)
    w2 = (rand(experts, hidden, inter) * inter ** -0.5).to(dtype)
    x = rand(tokens, hidden).to(dtype)
    who = torch.randint(-1, adapters, (tokens,), generator=g, device="cuda")
    top, ids = rand(tokens, experts).topk(topk, 1)
    return (AdaptedProjection(w, a, b, scale), MoeHalf(w1, w2)), (x, who, ids, torch.softmax(top, 1))


def step(layers, x, who, ids, weights, dout):
    """Forward and backward: the result and the gradients by name."""
    proj, moe = layers
    h, kept = proj.forward(x, who)
    out, saved = moe.forward(h, ids, weights)
    dh, dweights, dw1, dw2 = moe.backward(dout, saved)
    dx, da, db = proj.backward(dh, kept)
    return h, out, {"dh": dh, "dweights": dweights, "dw1": dw1, "dw2": dw2, "dx": dx, "da": da, "db": db}


def compare(tokens, hidden, inter, experts, topk, adapters, rank, dtype=torch.bfloat16):
    """Relative errors against float32 autograd.  Each layer's is taken from the
    inputs that it had: the MoE layer's from the projection's results, the
    projection's gradients from the MoE layer's."""
    layers, (x, who, ids, weights) = network(tokens, hidden, inter, experts, topk, adapters, rank, dtype)
    proj, moe = layers
    dout = (0.1 * torch.randn(tokens, hidden, device="cuda")).to(dtype)
    h, out, got = step(layers, x, who, ids, weights, dout)
    args = {n: v.float().requires_grad_() for n, v in
            (("h", h), ("weights", weights), ("w1", moe.w1), ("w2", moe.w2), ("x", x), ("a", proj.a), ("b", proj.b))}
    ref = reference(args["h"], ids, args["weights"], args["w1"], args["w2"])
    ref.backward(dout.float())
    (codes, sf), (n, k) = proj.w, (proj.n, proj.k)
    w = codes.view(torch.float8_e4m3fn).float() * sf.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    href = args["x"] @ w.t() + share(args["x"], who, proj.scale, args["a"], args["b"])
    href.backward(got["dh"].float())
    rel = lambda a, b: float((a.float() - b).norm() / b.norm().clamp(min=1e-30))  # noqa: E731
    err = {"h": rel(h, href.detach()), "out": rel(out, ref.detach())}
    err.update({n: rel(v, args[n[1:]].grad) for n, v in got.items()})
    return err, (layers, x, who, ids, weights, dout)


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inter", 1536), ("experts", 32), ("topk", 4), ("adapters", 8),
                        ("rank", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    err, (layers, x, who, ids, weights, dout) = compare(a.tokens, a.hidden, a.inter, a.experts, a.topk, a.adapters, a.rank)
    print("relative errors against float32: " + ", ".join(f"{k} {v:.4f}" for k, v in err.items()))
    proj, moe = layers
    for name, fn in (("forward", lambda: moe.forward(proj.forward(x, who, train=False)[0], ids, weights)),
                     ("forward and backward", lambda: step(layers, x, who, ids, weights, dout))):
        for _ in range(3):
            fn()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            fn()
        torch.cuda.synchronize()
        print(f"{name}: {(time.perf_counter() - t) / 20 * 1e6:.1f} us")


if __name__ == "__main__":
    main()
