"""Block-128 FP8 and the MoE token dispatch (oracle; test infrastructure only).

Plain NumPy definitions in float64.  A block (1 x 128 along a row, or 128 x
128) of values x has the FP32 scale s = max(amax / 448, 2^-126) and the E4M3
codes nearest to the FP32 quotient x / s; a product sums, over K blocks, the
two scales times the codes' dot product.  The dispatch sorts (token, slot)
pairs by expert, in order, into groups padded to a multiple of `align`.
"""

import numpy as np

from . import formats as F

TINY = np.float32(2.0 ** -126)


def _nblk(n):
    return -(-n // 128)


def quant(x, two_d=False):
    """x [m, k] (exact in float32) -> codes uint8 [m, k] and scales float32."""
    x = np.asarray(x, np.float32)
    m, k = x.shape
    bm = 128 if two_d else 1
    sf = np.empty((-(-m // bm), _nblk(k)), np.float32)
    q = np.empty((m, k), np.uint8)
    with np.errstate(all="ignore"):
        for i in range(sf.shape[0]):
            for j in range(sf.shape[1]):
                blk = x[i * bm:(i + 1) * bm, j * 128:(j + 1) * 128]
                s = np.max(np.abs(blk)) / np.float32(448.0)        # NaN propagates
                s = s if np.isnan(s) else max(s, TINY)
                sf[i, j] = s
                v = blk / np.float32(s)
                code = F.e4m3_encode(np.where(np.isnan(v), 0.0, v).astype(np.float64))
                q[i * bm:(i + 1) * bm, j * 128:(j + 1) * 128] = np.where(np.isnan(v), 0x7F, code)
    return q, sf


def scales_full(sf, m, k, two_d=False):
    """One scale per element, float64."""
    f = np.repeat(np.asarray(sf, np.float64), 128, axis=-1)[..., :k]
    return np.repeat(f, 128, axis=-2)[..., :m, :] if two_d else f


def dequant(q, sf, two_d=False):
    q = np.asarray(q)
    m, k = q.shape[-2:]
    return F.e4m3_decode(q) * scales_full(sf, m, k, two_d)


def gemm(a, sa, b, sb):
    """(a b^T in float64, |a| |b|^T) of dequantised operands."""
    x, y = dequant(a, sa), dequant(b, sb, True)
    return x @ y.T, np.abs(x) @ np.abs(y).T


def swiglu(x, h):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return x[:, h:] * x[:, :h] / (1.0 + np.exp(-x[:, :h]))


def sort(ids, experts, align, max_rows):
    """(row_map, row_pair, group_end, counts) by walking the pairs in order."""
    ids = np.asarray(ids)
    T, k = ids.shape
    counts = np.array([(ids == e).sum() for e in range(experts)], np.int64)
    ends = np.cumsum(-(-counts // align) * align)
    nxt = np.concatenate([[0], ends[:-1]])
    row_map = np.full((T, k), -1, np.int32)
    row_pair = np.full(max_rows, -1, np.int32)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < experts:
                row_map[t, j] = nxt[e]
                row_pair[nxt[e]] = t * k + j
                nxt[e] += 1
    return row_map, row_pair, ends.astype(np.int32), counts.astype(np.int32)


def permute(x, row_map, out):
    """A copy of `out` with out[row_map[t, j]] = x[t]."""
    out = np.array(out)
    T, k = row_map.shape
    for t in range(T):
        for j in range(k):
            if 0 <= row_map[t, j] < out.shape[0]:
                out[row_map[t, j]] = x[t]
    return out


def combine(y, row_map, weights=None):
    """(sum over slots of w y[row], sum of the magnitudes), float64."""
    y = np.asarray(y, np.float64)
    T, k = row_map.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            r = row_map[t, j]
            if 0 <= r < y.shape[0]:
                v = (1.0 if weights is None else float(weights[t, j])) * y[r]
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


def combine_backward(dout, y, row_map, weights):
    """(dy, dweights, sum |dout y|) in float64; rows that no pair maps to are zero."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    T, k = row_map.shape
    dy, dw, mag = np.zeros_like(y), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = row_map[t, j]
            if 0 <= r < y.shape[0]:
                dy[r] = float(weights[t, j]) * dout[t]
                dw[t, j] = dout[t] @ y[r]
                mag[t, j] = np.abs(dout[t]) @ np.abs(y[r])
    return dy, dw, mag
