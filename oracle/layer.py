"""64-bit definitions of the expert layer's operators, in numpy, one row and
one expert at a time. Shares nothing with the GPU path."""
from __future__ import annotations

import numpy as np


def _sigmoid(v):
    v = np.asarray(v, dtype=np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1 / (1 + e), e / (1 + e))


def _row_scores(row, score):
    """p of one row of logits: -inf scores 0, +inf counts as the largest
    float32 in the softmax, a NaN poisons the softmax's denominator."""
    row = np.asarray(row, dtype=np.float64)
    if score == "sigmoid":
        return np.where(np.isneginf(row), 0.0, _sigmoid(row))
    live = ~np.isneginf(row)
    if not live.any():
        return np.zeros_like(row)
    r = np.minimum(row, np.finfo(np.float32).max)
    e = np.zeros_like(row)
    e[live] = np.exp(r[live] - np.nanmax(r[live], initial=-np.inf))
    return e / e.sum()


def gate(logits, k, score="softmax", bias=None, renorm=True, scale=1.0,
         rank=None):
    """(ids, weights). ``rank``: the ranking to use (default the logits, or
    p + bias), for callers that fix how it is rounded."""
    logits = np.asarray(logits)
    T, E = logits.shape
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        row = logits[t].astype(np.float64)
        p = _row_scores(row, score)
        if rank is not None:
            order = np.asarray(rank[t], dtype=np.float64)
        elif score == "softmax":
            order = row
        else:
            order = p + (0 if bias is None else np.asarray(bias, np.float64))
        can = [e for e in range(E) if not np.isneginf(row[e]) and
               not np.isnan(row[e]) and order[e] > -np.inf]
        can.sort(key=lambda e: (-order[e], e))
        got = can[:k]
        ids[t, :len(got)] = got
        if score == "softmax" and renorm and got:
            r = np.minimum(row[got], np.finfo(np.float32).max)
            e = np.exp(r - r.max())
            pw = e / e.sum()
        else:
            pw = p[got]
            if renorm:
                pw = pw / (pw.sum() + 1e-20)
        w[t, :len(got)] = scale * pw
        if np.isnan(row).any():
            w[t] = np.nan
    return ids, w


def gate_backward(logits, ids, dw, score="softmax", renorm=True, scale=1.0):
    """Gradient of the logits at a fixed choice, by the chain rule with the
    full Jacobian of each row."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        sel = [int(e) for e in ids[t] if 0 <= e < E]
        g = scale * np.asarray([dw[t][j] for j in range(len(ids[t]))
                                if 0 <= ids[t][j] < E], dtype=np.float64)
        p = _row_scores(logits[t], score)
        if renorm:
            n = p[sel].sum() + 1e-20
            # d w_i / d p_j = (delta_ij - w_i) / n
            jac = (np.eye(len(sel)) - (p[sel] / n)[:, None]) / n
            g = jac.T @ g
        dp = np.zeros(E)
        dp[sel] = g
        if score == "softmax":
            out[t] = (np.diag(p) - np.outer(p, p)) @ dp
        else:
            out[t] = dp * p * (1 - p)
    return out


def quantize(x):
    """(q, scale) of rows: the factor 127 / top is a float32, as stated."""
    x = np.asarray(x, dtype=np.float32)
    q = np.zeros(x.shape, dtype=np.int8)
    s = np.zeros(x.shape[0], dtype=np.float32)
    for m, row in enumerate(x):
        if not np.isfinite(row).all():
            s[m] = np.nan
            continue
        top = np.abs(row).max(initial=np.float32(0))
        if top == 0:
            continue
        with np.errstate(over="ignore"):
            f = np.float32(127) / top
        if np.isinf(f):
            continue
        q[m] = np.rint(row * f).astype(np.int8)
        s[m] = top / np.float32(127)
    return q, s


def silu(v):
    return v * _sigmoid(v)


def matmul_i8(a, a_scale, w, w_scale, offsets=None, expert_of=None, index=None,
              index_div=1, gated=False, fill=np.nan):
    """[M, N] in float64; rows no group holds are ``fill``."""
    a, w = np.asarray(a, np.int64), np.asarray(w, np.int64)
    if w.ndim == 2:
        w, w_scale = w[None], np.asarray(w_scale)[None]
    w_scale = np.asarray(w_scale, np.float64).reshape(w.shape[:2])
    M = len(index) if index is not None else a.shape[0]
    off = [0, M] if offsets is None else [min(max(int(o), 0), M) for o in offsets]
    N = w.shape[1] // (2 if gated else 1)
    out = np.full((M, N), fill, dtype=np.float64)
    for g in range(len(off) - 1):
        e = g if expert_of is None else int(expert_of[g])
        if not 0 <= e < w.shape[0]:
            continue
        for m in range(off[g], off[g + 1]):
            r = m if index is None else (
                -1 if index[m] < 0 else int(index[m]) // index_div)
            if not 0 <= r < a.shape[0]:
                out[m] = 0
                continue
            v = (w[e] @ a[r]) * (float(a_scale[r]) * w_scale[e])
            out[m] = silu(v[:N]) * v[N:] if gated else v
    return out


def moe(x, router, gate_up, down, k, score="softmax", bias=None, renorm=True,
        scale=1.0, choice=None):
    """(out, ids, weights); matrices in float64, already scaled. ``choice``:
    (ids, weights) to use instead of the router's own."""
    x = np.asarray(x, np.float64)
    logits = x @ np.asarray(router, np.float64).T
    ids, w = choice if choice is not None else gate(logits, k, score, bias,
                                                    renorm, scale)
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(k):
            if ids[t, j] < 0:
                out[t] += w[t, j] * 0.0
                continue
            gu = gate_up[ids[t, j]] @ x[t]
            I = gu.shape[0] // 2
            out[t] += w[t, j] * (down[ids[t, j]] @ (silu(gu[:I]) * gu[I:]))
    return out, ids, w
