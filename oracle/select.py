"""Oracle of the operators whose products select their weights per row (test infrastructure only).

float64 restatements, in plain numpy loops, of top-k routing, the
mixture-of-experts layer and the per-row low-rank adapters, with the gradients
of the first and the last.  Inputs arrive widened exactly to float64 and
results are unrounded.  Each ``*_bound`` function gives, per element, what an
fp32 evaluation with roundings of relative size ``u`` at the stated places may
be off by.
"""

import numpy as np
from math import erf

EPS32 = 2.0 ** -24     # unit roundoff of fp32


def route_topk(logits, k, normalize=1):
    """(indices int32 [T, k], weights float64 [T, k]): the k largest logits of each row, ties to the lowest index."""
    T, G = logits.shape
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        p, order = _softmax_row(logits[t])
        for r, i in enumerate(order[:k]):
            idx[t, r], w[t, r] = i, p[i]
        if normalize and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return idx, w


def _softmax_row(row):
    """(p, indices that can be picked, best first); NaN and -inf have p = 0 and cannot be picked."""
    can = [i for i in range(len(row)) if row[i] > -np.inf]
    p = np.zeros(len(row))
    if not can:
        return p, []
    top = max(row[i] for i in can)
    for i in can:
        p[i] = 1.0 if row[i] == top else np.exp(row[i] - top)
    p /= p.sum()
    return p, sorted(can, key=lambda i: (-row[i], i))


def route_topk_grad(logits, indices, grad_weights, normalize=1):
    """Gradient of the picks' weights, given their gradient, with respect to the logits."""
    T, G = logits.shape
    out = np.zeros((T, G))
    for t in range(T):
        q, _ = _softmax_row(logits[t])
        d, picked = np.zeros(G), np.zeros(G, bool)
        for r, i in enumerate(indices[t]):
            if 0 <= i < G:
                d[i] += grad_weights[t, r]
                picked[i] = True
        if normalize:
            q = np.where(picked, q, 0.0)
            q = q / q.sum() if q.sum() > 0 else q
        out[t] = q * (d - (q * d).sum())
    return out


_ERF = np.vectorize(erf, otypes=[float])


def activate(g, activation):
    if activation == "silu":
        return g / (1.0 + np.exp(-g))
    if activation == "gelu":
        return 0.5 * g * (1.0 + _ERF(g / np.sqrt(2.0)))
    return np.maximum(g, 0.0)


def moe_layer(x, w_gate, w_up, w_down, indices, weights, activation="silu"):
    """out[t] = sum_s weights[t, s] * (act(x[t] Wg[e]) * (x[t] Wu[e])) Wd[e], e = indices[t, s], skipped when < 0."""
    out = np.zeros((x.shape[0], w_down.shape[2]))
    for t, s in np.ndindex(*indices.shape):
        e = indices[t, s]
        if 0 <= e < w_gate.shape[0]:
            h = activate(x[t] @ w_gate[e], activation)
            if w_up is not None:
                h = h * (x[t] @ w_up[e])
            out[t] += (1.0 if weights is None else weights[t, s]) * (h @ w_down[e])
    return out


def moe_layer_bound(x, w_gate, w_up, w_down, indices, weights, activation="silu", u=0.0):
    """u for h's rounding, u for the output's, and fp32 sums of K and F terms; |act'| <= 1.13 for every activation."""
    K, F = w_gate.shape[1:]
    out = np.zeros((x.shape[0], w_down.shape[2]))
    for t, s in np.ndindex(*indices.shape):
        e = indices[t, s]
        if 0 <= e < w_gate.shape[0]:
            ax = np.abs(x[t])
            g, ga = x[t] @ w_gate[e], ax @ np.abs(w_gate[e])
            a = np.abs(activate(g, activation))
            da = 1.13 * K * EPS32 * ga + 8 * EPS32 * (a + np.abs(g))
            if w_up is not None:
                up, ua = np.abs(x[t] @ w_up[e]), ax @ np.abs(w_up[e])
            else:
                up, ua = np.ones(F), np.zeros(F)
            h = a * up
            dh = da * up + a * K * EPS32 * ua
            w = 1.0 if weights is None else abs(weights[t, s])
            out[t] += w * (((2 * u + F * EPS32) * h + 1.01 * dh + 2.0 ** -24) @ np.abs(w_down[e]))
    return out


def _rows_by_adapter(indices, G):
    return {g: np.nonzero(indices == g)[0] for g in range(G) if (indices == g).any()}


def lowrank_matmul(X, W, A, B, indices, scales=None):
    """X W plus, for the rows of adapter g, scales[g] (X A[g]) B[g]."""
    Y = X @ W
    for g, m in _rows_by_adapter(indices, A.shape[0]).items():
        Y[m] += (1.0 if scales is None else scales[g]) * ((X[m] @ A[g]) @ B[g])
    return Y


def lowrank_matmul_bound(X, W, A, B, indices, scales=None, u=0.0):
    """u each for the factor's, the low-rank part's and the output's rounding, and fp32 sums."""
    K, R = A.shape[1:]
    aX = np.abs(X)
    base = aX @ np.abs(W)
    low = np.zeros_like(base)
    for g, m in _rows_by_adapter(indices, A.shape[0]).items():
        low[m] = (1.0 if scales is None else abs(scales[g])) * ((aX[m] @ np.abs(A[g])) @ np.abs(B[g]))
    return (u + K * EPS32) * base + (3 * u + (2 * K + R) * EPS32) * low + 2.0 ** -24


def lowrank_matmul_grad(dY, X, W, A, B, indices, scales=None):
    """(dX, dA, dB) of lowrank_matmul for a frozen W."""
    dX = dY @ W.T
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for g, m in _rows_by_adapter(indices, A.shape[0]).items():
        s = 1.0 if scales is None else scales[g]
        V, U = s * (dY[m] @ B[g].T), s * (X[m] @ A[g])
        dX[m] += V @ A[g].T
        dA[g] = X[m].T @ V
        dB[g] = U.T @ dY[m]
    return dX, dA, dB


def lowrank_matmul_grad_bound(dY, X, W, A, B, indices, scales=None, u=0.0):
    K, R = A.shape[1:]
    M, N = dY.shape
    aX, aD = np.abs(X), np.abs(dY)
    low = np.zeros(X.shape)
    bA, bB = np.zeros(A.shape), np.zeros(B.shape)
    for g, m in _rows_by_adapter(indices, A.shape[0]).items():
        s = 1.0 if scales is None else abs(scales[g])
        V, U = s * (aD[m] @ np.abs(B[g]).T), s * (aX[m] @ np.abs(A[g]))
        low[m] = V @ np.abs(A[g]).T
        bA[g] = (2 * u + (2 * N + M) * EPS32) * (aX[m].T @ V)
        bB[g] = (2 * u + (2 * K + M) * EPS32) * (U.T @ aD[m])
    return ((u + N * EPS32) * (aD @ np.abs(W).T) + (3 * u + (2 * N + R) * EPS32) * low + 2.0 ** -24, bA + 2.0 ** -24,
            bB + 2.0 ** -24)
