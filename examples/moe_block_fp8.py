"""A MoE feed-forward layer in block-128 FP8, forward and backward.

    python examples/moe_block_fp8.py [--tokens 4096] [--hidden 2048] [--inter 1536] [--experts 32] [--topk 4]

Forward: tokens are sorted by expert, their rows quantised on the way into
expert order, multiplied by the gate|up weights, passed through SwiGLU with
re-quantisation, multiplied by the down weights and summed back into tokens
with their routing weights.  Backward: the gradients of the routing weights,
of the tokens and of both weight tensors (FP32, summed per expert over its
rows).  Run as a script it compares both with a float32 layer and times them;
with --tokens 1 the forward is a single token's decoding step.
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fp4_gemm_moe_amd as hq  # noqa: E402


class MoeBlockFp8:
    """w1 [E, 2 inter, hidden] (gate rows, then up rows) and w2 [E, hidden,
    inter], bfloat16.  Both are quantised once in 128 x 128 blocks, as they are
    and transposed (for the gradients with respect to activations)."""

    def __init__(self, w1, w2):
        self.experts, n, self.hidden = w1.shape
        self.inter = n // 2
        self.w1, self.w2 = hq.block_quantize(w1, block_2d=True), hq.block_quantize(w2, block_2d=True)
        self.w1_t = hq.block_quantize(w1, block_2d=True, transpose=True)
        self.w2_t = hq.block_quantize(w2, block_2d=True, transpose=True)

    def forward(self, x, ids, weights, train=True):
        """x [T, hidden] bfloat16, ids [T, topk] int64, weights [T, topk]
        float32 -> [T, hidden] bfloat16, and what the backward pass needs."""
        dev, h, m = x.device, self.hidden, self.inter
        # the weights' gradients sum over whole blocks of 128 rows; decoding packs the rows
        align = 128 if train else 1
        row_map, _, ends, counts = hq.moe_sort(ids, self.experts, align)
        rows = hq.moe_max_rows(*ids.shape, self.experts, align)
        xq = torch.empty((rows, h), dtype=torch.uint8, device=dev)
        xs = torch.empty((rows, -(-h // 128)), device=dev)
        hq.hq_moe_permute_block_quant(x, row_map, ends, counts, xq, xs)
        gu = torch.empty((rows, 2 * m), dtype=torch.bfloat16, device=dev)
        hq.hq_block_group_contiguous_gemm(xq, xs, *self.w1, ends, gu)
        aq = torch.empty((rows, m), dtype=torch.uint8, device=dev)
        asf = torch.empty((rows, -(-m // 128)), device=dev)
        hq.hq_fused_swiglu_block_quant(gu, aq, asf, ends)
        y = torch.empty((rows, h), dtype=torch.bfloat16, device=dev)
        hq.hq_block_group_contiguous_gemm(aq, asf, *self.w2, ends, y)
        out = torch.empty_like(x)
        hq.hq_moe_combine(y, row_map, weights, out)
        return out, (x, weights, row_map, ends, counts, gu, y)

    def backward(self, dout, saved):
        """The gradients (x, routing weights, w1, w2) for out's gradient dout."""
        x, weights, row_map, ends, counts, gu, y = saved
        dev, h, m, E = dout.device, self.hidden, self.inter, self.experts
        rows = y.shape[0]
        used = torch.arange(rows, device=dev)[:, None] < ends[-1]      # rows past the last group hold anything
        dy = torch.empty_like(y)
        dweights = torch.empty_like(weights)
        hq.hq_moe_combine_backward(dout, y, row_map, weights, ends, counts, dy, dweights)
        # through the down product
        da = torch.empty((rows, m), dtype=torch.bfloat16, device=dev)
        hq.hq_block_group_contiguous_gemm(*hq.block_quantize(dy), *self.w2_t, ends, da)
        # through SwiGLU, a = up * silu(gate)
        gate, up = torch.where(used, gu, 0).float().split(m, 1)
        s = torch.sigmoid(gate)
        a = (up * gate * s).bfloat16()
        g = torch.where(used, da, 0).float()
        dgu = torch.cat([g * up * s * (1 + gate * (1 - s)), g * gate * s], 1).bfloat16()
        # through the gate|up product, and back into tokens
        dxr = torch.empty((rows, h), dtype=torch.bfloat16, device=dev)
        hq.hq_block_group_contiguous_gemm(*hq.block_quantize(dgu), *self.w1_t, ends, dxr)
        dx = torch.empty_like(x)
        hq.hq_moe_combine(dxr, row_map, None, dx)
        # the weights: sums over each expert's rows
        xr = torch.empty((rows, h), dtype=torch.bfloat16, device=dev)
        hq.hq_moe_permute(x, row_map, ends, counts, xr)
        dw1 = torch.empty((E, 2 * m, h), device=dev)
        hq.hq_block_group_k_gemm(*hq.block_quantize(dgu, transpose=True), *hq.block_quantize(xr, True, True), ends, dw1)
        dw2 = torch.empty((E, h, m), device=dev)
        hq.hq_block_group_k_gemm(*hq.block_quantize(dy, transpose=True), *hq.block_quantize(a, True, True), ends, dw2)
        return dx, dweights, dw1, dw2


def reference(x, ids, weights, w1, w2):
    """The layer in float32, expert by expert."""
    out = torch.zeros_like(x)
    m = w2.shape[2]
    for e in range(w1.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[t] @ w1[e].t()).split(m, 1)
        out = out.index_add(0, t, weights[t, j, None] * ((up * torch.nn.functional.silu(gate)) @ w2[e].t()))
    return out


def compare(tokens, hidden, inter, experts, topk, seed=0):
    """Relative errors of the outputs and gradients against float32 autograd."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = rand(tokens, hidden).bfloat16()
    w1, w2 = (rand(experts, 2 * inter, hidden) * hidden ** -0.5).bfloat16(), (rand(experts, hidden, inter) * inter ** -0.5).bfloat16()
    top, ids = rand(tokens, experts).topk(topk, 1)
    weights, dout = torch.softmax(top, 1), (0.1 * rand(tokens, hidden)).bfloat16()
    layer = MoeBlockFp8(w1, w2)
    out, saved = layer.forward(x, ids, weights)
    grads = layer.backward(dout, saved)
    args = [v.float().requires_grad_() for v in (x, weights, w1, w2)]
    ref = reference(args[0], ids, args[1], args[2], args[3])
    ref.backward(dout.float())
    rel = lambda a, b: float((a.float() - b).norm() / b.norm())  # noqa: E731
    err = {"out": rel(out, ref.detach())}
    err.update({n: rel(a, b.grad) for n, a, b in zip(("dx", "dweights", "dw1", "dw2"), grads, args)})
    err["decode"] = rel(layer.forward(x[:1], ids[:1], weights[:1], train=False)[0], ref[:1].detach())
    return err, (layer, x, ids, weights, dout, saved)


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inter", 1536), ("experts", 32), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    err, (layer, x, ids, weights, dout, saved) = compare(a.tokens, a.hidden, a.inter, a.experts, a.topk)
    print("relative errors against float32: " + ", ".join(f"{k} {v:.3f}" for k, v in err.items()))
    for name, fn in (("forward", lambda: layer.forward(x, ids, weights, a.tokens > 1)),
                     ("backward", lambda: layer.backward(dout, saved))):
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
