"""Pins of oracle/layer.py: values worked out by hand, gradients against differences, the iteration against singular values."""

import numpy as np

from oracle import layer

MUON = (3.4445, -4.7750, 2.0315)


def test_quantize_by_hand():
    x = np.array([[127.0, -63.5, 0.5, 1.5, 2.5, -0.5], [0.0] * 6, [1.0, np.inf, 0, 0, 0, 0], [np.nan, 1, 0, 0, 0, 0],
                  [-254.0, 254.0, 3.0, 1.0, 5.0, 0.0], [1e-45, 0, 0, 0, 0, 0]])
    q, s = layer.quantize_rows(x)
    assert s[0] == 1 and s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3]) and s[4] == 2 and s[5] == 0
    assert q.tolist() == [[127, -64, 0, 2, 2, 0], [0] * 6, [0] * 6, [0] * 6, [-127, 127, 2, 0, 2, 0], [0] * 6]


def test_int8_by_hand():
    A, B = np.array([[1, -2], [100, 127]], np.int8), np.array([[3, -128], [5, 127]], np.int8)
    y = layer.int8_matmul(A, B, np.array([2.0, 0.5]), np.array([1.0, 0.25]), np.array([10.0, -1.0]))
    np.testing.assert_array_equal(y, [[(3 - 10) * 2 + 10, (-128 - 254) * 2 * 0.25 - 1],
                                      [(300 + 635) * 0.5 + 10, (-12800 + 127 * 127) * 0.125 - 1]])


def test_balance_by_hand():
    l = np.log(np.array([[1.0, 1, 2], [1, 3, 0], [0, 0, 0]]) + 1e-300)
    l[1, 2] = -np.inf
    l[2] = -np.inf
    idx = np.array([[2, 0], [1, -1], [-1, -1]])
    loss, counts, mean = layer.route_balance(l, idx)
    assert counts.tolist() == [1, 1, 1, 2]
    np.testing.assert_allclose(mean, [(0.25 + 0.25) / 2, (0.25 + 0.75) / 2, 0.5 / 2])
    np.testing.assert_allclose(loss, 1.0)
    loss, counts, _ = layer.route_balance(l, np.array([[1, -1], [1, 5], [1, -1]]))
    assert counts.tolist() == [0, 3, 0, 2]
    np.testing.assert_allclose(loss, 3 * 0.5)
    assert layer.route_balance(l[2:], idx[2:])[0] == 0 and layer.route_balance(l, np.full((3, 1), -1))[0] == 0


def test_balance_gradient_is_the_difference_of_the_loss():
    rng = np.random.default_rng(1)
    l, idx = rng.normal(size=(5, 6)), rng.integers(0, 6, size=(5, 2))
    l[3, 2:4] = -np.inf
    l[4] = -np.inf
    _, counts, _ = layer.route_balance(l, idx)
    got = layer.route_balance_grad(l, counts, 1.5)
    for t in range(5):
        for j in range(6):
            d = np.zeros_like(l)
            d[t, j] = 1e-6
            diff = layer.route_balance(l + d, idx)[0] - layer.route_balance(l - d, idx)[0]
            np.testing.assert_allclose(got[t, j], 1.5 * diff / 2e-6, atol=1e-9)
    assert (got[4] == 0).all() and (got[3, 2:4] == 0).all()
    base = rng.normal(size=l.shape)
    np.testing.assert_allclose(layer.route_balance_grad(l, counts, 1.5, base), got + base)


def test_orthogonalize_acts_on_the_singular_values():
    rng = np.random.default_rng(2)
    for shape in ((4, 7), (7, 4), (1, 3), (5, 5)):
        X = rng.normal(size=(2,) + shape)
        got = layer.orthogonalize(X, [MUON] * 3 + [(1.5, -0.5, 0.0)], 1e-7, 0.5)
        for x, y in zip(X, got):
            u, s, v = np.linalg.svd(x, full_matrices=False)
            s = s / (np.linalg.norm(x) + 1e-7)
            for a, b, c in [MUON] * 3 + [(1.5, -0.5, 0.0)]:
                s = a * s + b * s ** 3 + c * s ** 5
            np.testing.assert_allclose(y, 0.5 * (u * s) @ v, atol=1e-12)
    assert (layer.orthogonalize(np.zeros((2, 3)), [MUON], 1e-7) == 0).all()


def test_orthogonalize_bound_holds_for_a_rounded_chain():
    rng = np.random.default_rng(3)
    for shape in ((16, 24), (40, 12)):
        X = rng.normal(size=shape)
        h = lambda t: (np.asarray(t) * 4096).astype(np.float16).astype(np.float64) / 4096        # noqa: E731
        W = X if shape[0] <= shape[1] else X.T
        S = W / np.linalg.norm(W)
        for a, b, c in [MUON] * 5:
            A = h(h(S) @ h(S).T)
            S = a * S + h(b * A + c * A @ A) @ h(S)
        want = layer.orthogonalize(W, [MUON] * 5, 0.0)
        assert np.linalg.norm(S - want) < layer.orthogonalize_bound(X, [MUON] * 5, 0.0, operand=2.0 ** -11)
        assert layer.orthogonalize_bound(X, [MUON] * 5, 0.0) < 2e-2 * np.linalg.norm(want)
