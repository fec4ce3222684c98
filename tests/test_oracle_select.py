"""Pins of oracle/select.py: values worked out by hand, and gradients against differences of the forward forms."""

import numpy as np
import pytest

from oracle import select


def test_route_by_hand():
    l = np.array([[0.0, np.log(2.0), np.log(5.0), np.log(2.0)],
                  [-np.inf, 1.0, np.nan, -np.inf],
                  [-np.inf] * 4,
                  [np.inf, 0.0, np.inf, 0.0],
                  [-0.0, 0.0, -1.0, 0.0]])
    idx, w = select.route_topk(l, 2, 0)
    assert idx.tolist() == [[2, 1], [1, -1], [-1, -1], [0, 2], [0, 1]]
    np.testing.assert_allclose(w[0], [0.5, 0.2], rtol=1e-15)
    np.testing.assert_allclose(w[1:4], [[1, 0], [0, 0], [0.5, 0.5]])
    idx, w = select.route_topk(l, 3, 1)
    assert idx[0].tolist() == [2, 1, 3]
    np.testing.assert_allclose(w[0], np.array([5, 2, 2]) / 9, rtol=1e-15)


@pytest.mark.parametrize("normalize", [0, 1])
def test_route_gradient_is_the_difference_of_the_weights(normalize):
    rng = np.random.default_rng(3)
    l, dw = rng.normal(size=(4, 7)), rng.normal(size=(4, 3))
    idx, _ = select.route_topk(l, 3, normalize)
    got = select.route_topk_grad(l, idx, dw, normalize)
    for i in range(7):
        e = np.zeros(7)
        e[i] = 1e-6
        hi, lo = select.route_topk(l + e, 3, normalize), select.route_topk(l - e, 3, normalize)
        assert (hi[0] == idx).all() and (lo[0] == idx).all()
        np.testing.assert_allclose(got[:, i], ((hi[1] - lo[1]) * dw).sum(axis=1) / 2e-6, atol=1e-8)


def test_moe_by_hand():
    x = np.array([[1.0, 2.0], [3.0, -1.0], [5.0, 5.0]])
    wg = np.array([[[1.0], [0.0]], [[0.0], [1.0]]])      # expert 0 takes x[0], expert 1 takes x[1]
    wu = np.array([[[0.0], [1.0]], [[2.0], [0.0]]])
    wd = np.array([[[1.0, -1.0]], [[10.0, 0.0]]])
    idx = np.array([[0, 1], [1, -1], [-1, -1]])
    w = np.array([[0.5, 0.25], [2.0, 9.0], [1.0, 1.0]])
    got = select.moe_layer(x, wg, wu, wd, idx, w, "relu")
    # token 0: 0.5 * (1 * 2) * [1, -1] + 0.25 * (2 * 2) * [10, 0]; token 1: relu(-1) = 0
    assert got.tolist() == [[1.0 + 10.0, -1.0], [0.0, 0.0], [0.0, 0.0]]
    assert select.activate(np.array([0.0]), "silu")[0] == 0.0
    np.testing.assert_allclose(select.activate(np.array([1.0, -1.0]), "gelu"), [0.8413447460685429, -0.15865525393145707])


def test_lowrank_by_hand_and_gradients_by_differences():
    X = np.array([[1.0, 2.0], [3.0, 4.0]])
    W = np.eye(2)
    A, B = np.array([[[1.0], [1.0]]]), np.array([[[1.0, -1.0]]])
    assert select.lowrank_matmul(X, W, A, B, np.array([0, -1]), np.array([2.0])).tolist() == [[7.0, -4.0], [3.0, 4.0]]
    rng = np.random.default_rng(4)
    M, K, N, R, G = 6, 4, 5, 2, 3
    X, W, A, B = (rng.normal(size=s) for s in ((M, K), (K, N), (G, K, R), (G, R, N)))
    dY, sc, idx = rng.normal(size=(M, N)), rng.uniform(0.5, 2, G), np.array([2, 0, -1, 2, 0, 0])
    grads = select.lowrank_matmul_grad(dY, X, W, A, B, idx, sc)
    assert not grads[1][1].any() and not grads[2][1].any()     # adapter 1 has no rows
    for theta, g in zip((X, A, B), grads):
        for _ in range(4):
            d = rng.normal(size=theta.shape)
            keep = theta.copy()
            theta += 1e-6 * d
            hi = (select.lowrank_matmul(X, W, A, B, idx, sc) * dY).sum()
            theta[...] = keep - 1e-6 * d
            lo = (select.lowrank_matmul(X, W, A, B, idx, sc) * dY).sum()
            theta[...] = keep
            np.testing.assert_allclose((g * d).sum(), (hi - lo) / 2e-6, rtol=1e-6, atol=1e-7)
