"""Pins of the emulated roundings of oracle/layer.py's orthogonalised update."""

import numpy as np
import pytest

from oracle import layer

MUON = (3.4445, -4.7750, 2.0315)


def test_bits_round_to_even():
    x = np.array([1.0, 1.0 + 2.0 ** -10, 1.0 + 2.0 ** -11, 1.0 + 3 * 2.0 ** -11, -5.0, 0.0, 2.0 ** -60 * 1.0004])
    np.testing.assert_array_equal(layer._bits(x, 11), [1.0, 1.0 + 2.0 ** -10, 1.0, 1.0 + 2.0 ** -9, -5.0, 0.0, 2.0 ** -60])


def test_truncated_sums_are_cut_towards_zero():
    one = np.ones((1, 2))
    small = np.array([[1.0], [2.0 ** -23 * 1.5]])
    assert layer._truncated_product([(one, small)], 1, 2)[0, 0] == 1.0 + 2.0 ** -23
    assert layer._truncated_product([(one, -small)], 1, 2)[0, 0] == -1.0 - 2.0 ** -23
    assert layer._truncated_product([(one, small * 2.0 ** -1)], 2, 2)[0, 0] == 0.5 + 2.0 ** -24
    # a second segment's sum is added with rounding
    assert layer._truncated_product([(one, small)], 1, 1)[0, 0] == 1.0 + 2.0 ** -22


@pytest.mark.parametrize("shape", [(40, 70), (70, 40), (33, 33)])
def test_emulated_roundings_are_of_the_stated_size(shape):
    X = np.random.default_rng(7).normal(size=shape)
    want = layer.orthogonalize(X, [MUON] * 3, 1e-7, 0.5)
    n = np.linalg.norm(want)
    off = {f: np.linalg.norm(layer.orthogonalize_emulated(X, [MUON] * 3, 1e-7, 0.5, f) - want) / n
           for f in ("pairs", "single", "matmul")}
    assert off["single"] < 2.0 ** -9 and off["pairs"] < 2.0 ** -19 and off["matmul"] < 2.0 ** -18
    assert off["single"] > 20 * off["pairs"]


def test_half_steps():
    x = np.array([1.0, 1.5, -2.0, 0.75, 0.0])
    np.testing.assert_array_equal(layer.half_steps(x, 2.0 ** -8), [2.0 ** -8, 2.0 ** -8, 2.0 ** -7, 2.0 ** -9, 0.0])
