"""16-bit products by expert, SwiGLU with its gradient and low-rank adapters
(oracle; test infrastructure only).

Plain NumPy definitions in float64, row by row and group by group, with the sums
of magnitudes that the tests' error bounds are made of.
"""

import numpy as np


def clamped(ends, rows):
    """Non-decreasing ends in [0, rows]."""
    return np.minimum(np.maximum.accumulate(np.maximum(np.asarray(ends, np.int64), 0)), rows)


def group_rows(ends, rows):
    lo = 0
    for g, hi in enumerate(clamped(ends, rows)):
        yield g, lo, int(hi)
        lo = int(hi)


def contiguous(a, b, ends, transpose=False):
    """(out, magnitudes), NaN in the rows of no group."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    n = b.shape[2] if transpose else b.shape[1]
    out = np.full((a.shape[0], n), np.nan)
    mag = np.zeros_like(out)
    for g, lo, hi in group_rows(ends, a.shape[0]):
        w = b[g] if transpose else b[g].T
        out[lo:hi] = a[lo:hi] @ w
        mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w)
    return out, mag


def masked(a, b, counts, max_m, transpose=False):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    n = b.shape[2] if transpose else b.shape[1]
    out = np.full((a.shape[0], n), np.nan)
    mag = np.zeros_like(out)
    for g in range(b.shape[0]):
        lo = g * max_m
        hi = lo + min(max(int(counts[g]), 0), max_m)
        w = b[g] if transpose else b[g].T
        out[lo:hi] = a[lo:hi] @ w
        mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w)
    return out, mag


def group_k(a, b, ends):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    out = np.zeros((len(ends), a.shape[1], b.shape[1]))
    mag = np.zeros_like(out)
    for g, lo, hi in group_rows(ends, a.shape[0]):
        out[g] = a[lo:hi].T @ b[lo:hi]
        mag[g] = np.abs(a[lo:hi]).T @ np.abs(b[lo:hi])
    return out, mag


def swiglu(x):
    x = np.asarray(x, np.float64)
    h = x.shape[1] // 2
    gate, up = x[:, :h], x[:, h:]
    with np.errstate(over="ignore"):
        return up * (gate / (1.0 + np.exp(-gate)))


def swiglu_backward(dy, x):
    """(dgate, dup)."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    h = x.shape[1] // 2
    gate, up = x[:, :h], x[:, h:]
    t = np.exp(-np.abs(gate))
    s, rest = np.where(gate >= 0, 1, t) / (1 + t), np.where(gate >= 0, t, 1) / (1 + t)
    return dy * up * s * (1 + gate * rest), dy * gate * s


def plan(ids, adapters):
    """(row_map, row_pair, ends) of the tokens sorted by adapter."""
    ids = np.asarray(ids, np.int64)
    key = np.where((ids >= 0) & (ids < adapters), ids, adapters)
    order = np.argsort(key, kind="stable")
    ends = np.cumsum(np.bincount(key, minlength=adapters + 1)[:adapters])
    last = int(ends[-1])
    row_pair = np.full(ids.size, -1, np.int32)
    row_pair[:last] = order[:last]
    row_map = np.full(ids.size, -1, np.int32)
    row_map[order[:last]] = np.arange(last)
    return row_map, row_pair, ends.astype(np.int32)


def lora(x, a, b, scale, owner, base):
    """owner [m]: each token's adapter, -1 for none.  {"v": by token, "out"} and
    the magnitudes of their sums."""
    x, a, b = (np.asarray(t, np.float64) for t in (x, a, b))
    m, n, r = x.shape[0], b.shape[1], a.shape[1]
    out = np.zeros((m, n)) if base is None else np.asarray(base, np.float64).copy()
    v, vmag, omag = np.zeros((m, r)), np.zeros((m, r)), np.abs(out)
    for t in range(m):
        g = owner[t]
        if g >= 0:
            v[t], vmag[t] = a[g] @ x[t], np.abs(a[g]) @ np.abs(x[t])
            out[t] += scale[g] * (b[g] @ v[t])
            omag[t] += abs(scale[g]) * (np.abs(b[g]) @ vmag[t])
    return {"v": v, "vmag": vmag, "out": out, "mag": omag}


def lora_backward(dy, x, v, a, b, scale, owner, base):
    """v [m, r] by token.  {"dx", "da", "db"} and the magnitudes of their sums."""
    dy, x, v, a, b = (np.asarray(t, np.float64) for t in (dy, x, v, a, b))
    dx = np.zeros(x.shape) if base is None else np.asarray(base, np.float64).copy()
    res = {"dx": dx, "dxmag": np.abs(dx), "da": np.zeros(a.shape), "damag": np.zeros(a.shape),
           "db": np.zeros(b.shape), "dbmag": np.zeros(b.shape)}
    for t in range(x.shape[0]):
        g = owner[t]
        if g < 0:
            continue
        u, umag, f = dy[t] @ b[g], np.abs(dy[t]) @ np.abs(b[g]), float(scale[g])
        dx[t] += f * (u @ a[g])
        res["dxmag"][t] += abs(f) * (umag @ np.abs(a[g]))
        res["da"][g] += f * np.outer(u, x[t])
        res["damag"][g] += abs(f) * np.outer(umag, np.abs(x[t]))
        res["db"][g] += f * np.outer(dy[t], v[t])
        res["dbmag"][g] += abs(f) * np.outer(np.abs(dy[t]), np.abs(v[t]))
    return res
