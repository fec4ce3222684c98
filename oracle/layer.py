"""Oracle of the 8-bit product, the router's balance loss and the orthogonalised update (test infrastructure only).

float64 restatements in numpy.  Inputs arrive widened exactly to float64 (int8 as it is) and results are unrounded,
except for the quantisation of rows, whose definition is a sequence of fp32 operations.
"""

import numpy as np

from .select import EPS32, _softmax_row


def quantize_rows(x):
    """(q int8 [M, K], scales fp32 [M]): s = amax / 127 and q = rint(x / s), each one rounded fp32 operation."""
    x = np.asarray(x, np.float32)
    q, s = np.zeros(x.shape, np.int8), np.zeros(x.shape[0], np.float32)
    for m, row in enumerate(x):
        if not np.isfinite(row).all():
            s[m] = np.nan
            continue
        s[m] = (np.abs(row).max() if row.size else np.float32(0)) / np.float32(127)
        if s[m] > 0:
            q[m] = np.clip(np.rint(row / s[m]), -127, 127).astype(np.int8)
    return q, s


def int8_matmul(A, B, a_scale, b_scale, bias=None):
    acc = A.astype(np.float64) @ B.astype(np.float64)          # exact below 2^53
    y = acc * a_scale[:, None] * b_scale[None, :]
    return y if bias is None else y + bias


def int8_matmul_bound(A, B, a_scale, b_scale, bias=None, u=EPS32):
    """Three fp32 steps and one rounding of size u; and, where the sum of the magnitudes passes 2^24, an fp32 sum of
    16 products at a time, each off by at most 2^-23 of the magnitudes so far."""
    K = A.shape[1]
    mag = np.abs(A.astype(np.float64)) @ np.abs(B.astype(np.float64))
    scale = np.abs(a_scale[:, None] * b_scale[None, :])
    off = np.where(mag < 2.0 ** 24, EPS32 * np.abs(A.astype(np.float64) @ B.astype(np.float64)),
                   (K / 16 + 1) * 2.0 ** -23 * mag) * scale
    y = np.abs(int8_matmul(A, B, a_scale, b_scale, bias))
    part = np.abs(int8_matmul(A, B, a_scale, b_scale))
    return off * 1.01 + 4 * EPS32 * part + (u * 1.01 + EPS32) * y + 1e-37


def route_balance(logits, indices):
    """(loss, counts int32 [G + 1], mean_probs [G]); the last place of counts holds the rows that take part."""
    T, G = logits.shape
    counts, mean = np.zeros(G + 1, np.int32), np.zeros(G)
    for t in range(T):
        p, can = _softmax_row(logits[t])
        mean += p
        counts[G] += len(can) > 0
        for i in indices[t]:
            if 0 <= i < G:
                counts[i] += 1
    mean /= max(1, counts[G])
    share = counts[:G] / max(1, counts[:G].sum())
    return G * (share * mean).sum(), counts, mean


def route_balance_grad(logits, counts, grad_loss, base=None):
    T, G = logits.shape
    out = np.zeros((T, G)) if base is None else np.array(base, np.float64)
    C, rows = counts[:G].sum(), counts[G]
    if C == 0 or rows == 0:
        return out
    share = counts[:G] / C
    for t in range(T):
        p, _ = _softmax_row(logits[t])
        out[t] += grad_loss * (G / rows) * p * (share - (share * p).sum())
    return out


def orthogonalize(X, coefficients, eps, scale=1.0):
    """scale * X_steps of each matrix of X [..., M, N]; ``coefficients`` one (a, b, c) a step."""
    X = X / (np.sqrt((X * X).sum(axis=(-2, -1), keepdims=True)) + eps)
    for a, b, c in coefficients:
        T = np.swapaxes(X, -2, -1)
        if X.shape[-2] <= X.shape[-1]:
            A = X @ T
            X = a * X + (b * A + c * A @ A) @ X
        else:
            A = T @ X
            X = a * X + X @ (b * A + c * A @ A)
    return scale * X


def orthogonalize_bound(X, coefficients, eps, scale=1.0, operand=EPS32, output=EPS32):
    """Frobenius norm that the result of one matrix may be off by, for products whose operands are rounded by
    ``operand`` relative (fp32 sums on top) and a state rounded to fp32 in every step.

    An error E of a step's input reaches its output as at most max |p'| |E| over the singular values' range (p(s) = a s
    + b s^3 + c s^5: the derivative of an odd matrix polynomial is bounded by p's divided differences); to that come the
    step's own roundings."""
    X = np.asarray(X, np.float64)
    X = X if X.shape[0] <= X.shape[1] else X.T
    X = X / (np.linalg.norm(X) + eps)
    m, n = X.shape
    err = 2 * EPS32 * np.linalg.norm(X)
    for a, b, c in coefficients:
        s = np.linalg.svd(X, compute_uv=False)
        top, A = s[0], X @ X.T
        grid = np.linspace(0, top * 1.01 + 1e-12, 2000)
        slope = np.abs(a + 3 * b * grid ** 2 + 5 * c * grid ** 4).max()
        nx, na = np.linalg.norm(s), np.linalg.norm(s ** 2)
        dA = 2 * operand * top * nx + n * EPS32 * nx * nx + operand * na
        B = b * A + c * A @ A
        dB = abs(b) * dA + abs(c) * (2 * top ** 2 * (dA + operand * na) + m * EPS32 * na * na) + (operand + 4 * EPS32) * (
            abs(b) * na + abs(c) * np.linalg.norm(s ** 4))
        nb = np.linalg.norm(B, 2)
        local = dB * top + nb * operand * nx + m * EPS32 * np.linalg.norm(B) * nx
        X = a * X + B @ X
        err = slope * err + 1.1 * local + 4 * EPS32 * (abs(a) * nx + np.linalg.norm(X))
    return abs(scale) * (err * (1 + output) + (output + EPS32) * np.linalg.norm(X)) * 1.01 + 1e-30


def _bits(x, bits):
    """x rounded to `bits` significant bits, ties to even, no limit of range."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def _truncated(x):
    """x cut towards zero to 24 significant bits."""
    return (x.view(np.int64) & ~((1 << 29) - 1)).view(np.float64)


def _truncated_product(pairs, group, segment):
    """The sum of A @ B over ``pairs`` as the tensor cores add it: exact products of `group` terms of each in turn, every
    addition cut towards zero to 24 significant bits; after every `segment` terms the sum goes to an fp32 total."""
    K = pairs[0][0].shape[1]
    total = np.zeros((pairs[0][0].shape[0], pairs[0][1].shape[1]))
    for s in range(0, K, segment):
        acc = np.zeros_like(total)
        for k in range(s, min(s + segment, K), group):
            for A, B in pairs:
                acc = _truncated(acc + A[:, k:min(k + group, s + segment)] @ B[k:min(k + group, s + segment)])
        total = _bits(total + acc, 24)
    return total


def orthogonalize_emulated(X, coefficients, eps, scale=1.0, form="pairs"):
    """The chain of orthogonalize with the roundings of the products on the tensor cores, before the rounding of the output:
      pairs   operands of two values of 11 bits, the products of a value and a rest beside the others' sum, which goes
              to an fp32 total after 64 terms, 16 at a time
      single  operands of 11 bits, sums of 16 products at a time
      matmul  operands of two values of 11 bits, three products into one sum, 8 terms at a time (f32 MatMul's)
    and a state of 24 bits.  Its distance from orthogonalize says how far roundings take a matrix, which the bound
    above only limits from far away."""
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = _bits(X / (np.sqrt((X * X).sum()) + eps), 24)

    def product(A, B):
        ah, bh = _bits(A, 11), _bits(B, 11)
        if form == "single":
            return _truncated_product([(ah, bh)], 16, A.shape[1])
        al, bl = _bits(A - ah, 11), _bits(B - bh, 11)
        if form == "matmul":
            return _truncated_product([(al, bh), (ah, bl), (ah, bh)], 8, A.shape[1])
        return _truncated_product([(ah, bh)], 16, 64) + ah @ bl + al @ bh

    held = {"pairs": 22, "single": 11, "matmul": 24}[form]
    for a, b, c in coefficients:
        A = _bits(product(X, X.T), held)
        B = _bits(b * A + c * product(A, A), held)
        X = _bits(a * X + product(B, X), 24)
    return scale * (X.T if tall else X)


def half_steps(x, u):
    """Half a step of a type with unit roundoff u at each value of x: the most that rounding x can change it."""
    return u * np.ldexp(1.0, np.frexp(x)[1] - 1) * (x != 0)
