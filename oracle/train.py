"""64-bit definitions of the expert layer's training step, in numpy. Shares
nothing with the GPU path."""
from __future__ import annotations

import math

import numpy as np

from oracle.layer import _row_scores, _sigmoid, silu

BLOCK = 32


def scores(row, score):
    """p of one token: the softmax, or the sigmoids over their sum + 1e-20."""
    p = _row_scores(row, score)
    return p if score == "softmax" else p / (p.sum() + 1e-20)


def _sequences(offsets, T):
    off = [0, T] if offsets is None else [min(max(int(o), 0), T) for o in offsets]
    return [(off[s], max(off[s], off[s + 1])) for s in range(len(off) - 1)]


def balance(logits, ids, offsets=None, score="softmax"):
    """(loss [n], counts [n, E], prob [n, E])."""
    logits, ids = np.asarray(logits, np.float64), np.asarray(ids)
    T, E = logits.shape
    k = ids.shape[1]
    seqs = _sequences(offsets, T)
    loss, counts = np.zeros(len(seqs)), np.zeros((len(seqs), E), np.int64)
    prob = np.zeros((len(seqs), E))
    for s, (a, b) in enumerate(seqs):
        for t in range(a, b):
            prob[s] += scores(logits[t], score)
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if b > a:
            prob[s] /= b - a
            loss[s] = E / (k * (b - a)) * float(counts[s] @ prob[s])
    return loss, counts, prob


def balance_backward(logits, counts, dloss, k, offsets=None, score="softmax"):
    """Gradient of the logits by the full Jacobian of each token's scores; and
    the size of its terms (for tolerances)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for s, (a, b) in enumerate(_sequences(offsets, T)):
        for t in range(a, b):
            n = b - a
            g = float(dloss[s]) * E / (k * n * n) * np.asarray(counts[s], np.float64)
            p = _row_scores(logits[t], score)
            if score == "softmax":
                jac = np.diag(p) - np.outer(p, p)
                out[t] = jac.T @ g
                size[t] = np.abs(p * g) + p * (np.abs(p * g).sum())
            else:
                total = p.sum() + 1e-20
                # d (p_i / total) / d p_j = (delta_ij - p_i / total) / total
                jac = (np.eye(E) - (p / total)[:, None]) / total
                slope = p * _sigmoid(-logits[t])
                slope = np.where(np.isneginf(logits[t]), 0.0, slope)
                out[t] = (jac.T @ g) * slope
                q = p / total
                size[t] = np.abs(q * g) + q * (np.abs(q * g).sum())
    return out, size


def pack(x):
    """(q int8 [M, K], scale uint8 [M, blocks]), block by block from the
    definition: the smallest e >= -126 with top <= 127 * 2^e, but 121 at most,
    whose 127-fold is the last that is a float; past that q is +-127."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    nb = -(-K // BLOCK)
    q, scale = np.zeros((M, K), np.int8), np.zeros((M, nb), np.uint8)
    for m in range(M):
        for c in range(nb):
            v = x[m, c * BLOCK:(c + 1) * BLOCK]
            if not np.isfinite(v).all():
                scale[m, c] = 255
                continue
            top = np.abs(v).max()
            e = -126
            if top > 0:
                e = max(-126, math.frexp(top)[1] - 8)
                while top > math.ldexp(127.0, e) and e < 121:
                    e += 1
                e = min(e, 121)
                while e > -126 and top <= math.ldexp(127.0, e - 1):
                    e -= 1
            scale[m, c] = e + 127
            q[m, c * BLOCK:(c + 1) * BLOCK] = np.clip(np.rint(v * math.ldexp(1.0, -e)), -127, 127)
    return q, scale


def unpack(q, scale):
    q, scale = np.asarray(q, np.float64), np.asarray(scale)
    step = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return q * np.repeat(step, BLOCK, axis=1)[:, :q.shape[1]]


def kept(gu):
    """(gate, up) as their packed rows stand for."""
    gu = np.asarray(gu)
    I = gu.shape[1] // 2
    return unpack(*pack(gu[:, :I])), unpack(*pack(gu[:, I:]))


def gated(gu):
    gu = np.asarray(gu, np.float64)
    I = gu.shape[1] // 2
    return silu(gu[:, :I]) * gu[:, I:]


def gated_backward(gate, up, dh):
    """(dgu, silu(gate) up) at given gate and up."""
    gate, up, dh = (np.asarray(v, np.float64) for v in (gate, up, dh))
    s = _sigmoid(gate)
    slope = s + gate * s * _sigmoid(-gate)
    return np.concatenate([dh * up * slope, dh * gate * s], 1), gate * s * up


def weight_grad(dy, x, offsets=None, index=None, index_div=1):
    """([groups, N, K], sums of the terms' magnitudes), row by row."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    M = dy.shape[0]
    groups = _sequences(offsets, M)
    out = np.zeros((len(groups), dy.shape[1], x.shape[1]))
    size = np.zeros_like(out)
    for g, (a, b) in enumerate(groups):
        for m in range(a, b):
            r = m if index is None else (-1 if index[m] < 0 else int(index[m]) // index_div)
            row = x[r] if 0 <= r < x.shape[0] else np.zeros(x.shape[1])
            out[g] += np.outer(dy[m], row)
            size[g] += np.outer(np.abs(dy[m]), np.abs(row))
    return out, size


def combine(y, inv, weights=None, add=None):
    """(out, sum of the terms' magnitudes)."""
    y, inv = np.asarray(y, np.float64), np.asarray(inv)
    T, k = inv.shape
    w = np.ones((T, k)) if weights is None else np.asarray(weights, np.float64)
    out = np.zeros((T, y.shape[1])) if add is None else np.array(add, np.float64)
    size = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= inv[t, j] < y.shape[0]:
                out[t] += w[t, j] * y[inv[t, j]]
                size[t] += np.abs(w[t, j] * y[inv[t, j]])
    return out, size


def combine_backward(dout, y, inv, weights=None):
    """(dy, dweights, size of dweights' terms); rows of dy nobody names are
    NaN."""
    dout, y, inv = np.asarray(dout, np.float64), np.asarray(y, np.float64), np.asarray(inv)
    T, k = inv.shape
    w = np.ones((T, k)) if weights is None else np.asarray(weights, np.float64)
    dy, dw, size = np.full(y.shape, np.nan), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= inv[t, j] < y.shape[0]:
                dy[inv[t, j]] = w[t, j] * dout[t]
                dw[t, j] = dout[t] @ y[inv[t, j]]
                size[t, j] = np.abs(dout[t]) @ np.abs(y[inv[t, j]])
    return dy, dw, size
