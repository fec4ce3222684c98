"""Routing, the expert layer and the adapters at values and layouts where a kernel's own arithmetic shows.

Picks that are not the largest logits, infinite weights, factors and hidden
values near the ends of f16's range, the error in the mean (not only at its
worst), and calls on another stream.  Tolerances are the oracle's bounds, or
derived beside the test.
"""

import numpy as np
import pytest
import torch

import quantized_gemm_gb300 as qg
from helpers import rand_tensor, to_np
from oracle import select
from test_gpu_select import (U, _check_lowrank_grad, _check_route, _logits, _lowrank_inputs, _moe_inputs, assert_within,  # noqa: F401
                             clean_status, tensor_path)

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS32 = 2.0 ** -24


# ------------------------------------------------------------------ routing


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,G,k", [(5, 8, 2), (9, 64, 4), (3, 256, 8), (2, 300, 20)])
@pytest.mark.parametrize("gap", [5.0, 90.0, 104.0, 300.0])
@pytest.mark.parametrize("normalize", [0, 1])
def test_route_gradient_of_picks_below_the_largest_logit(T, G, k, gap, normalize, dtype):
    """Picks of a biased or capacity-limited router: the row's largest logit, `gap` above the rest, is not among them."""
    rng = np.random.default_rng(G + int(gap))
    l = rng.normal(size=(T, G)) * 2
    idx = np.argsort(rng.random((T, G)), axis=1)[:, :k + 1].astype(np.int32)
    for t in range(T):
        l[t, idx[t, k]] = l[t].max() + gap
    idx = idx[:, :k].copy()
    idx[0, 1:] = -1                                            # dropped picks; a row without any
    idx[1] = -1
    l = torch.from_numpy(l).to(dtype).to(DEV)
    dw = rand_tensor((T, k), F32, 6, DEV)
    got = qg.mm_route_topk_grad(l, torch.from_numpy(idx).to(DEV), dw, normalize)
    want = select.route_topk_grad(to_np(l), idx, to_np(dw), normalize)
    # the terms' sizes: exp's argument is within 40, or (normalize = 0) the share is below 1e-30 anyway
    p, d = np.zeros((T, G)), np.zeros((T, G))
    for t in range(T):
        p[t] = select._softmax_row(to_np(l)[t])[0]
        keep = np.isin(np.arange(G), idx[t])
        if normalize:
            p[t] = np.where(keep, p[t], 0)
            p[t] /= max(p[t].sum(), 1e-300)
        for r in range(k):
            if idx[t, r] >= 0:
                d[t, idx[t, r]] = abs(to_np(dw)[t, r])
    mag = p * (d + (p * d).sum(axis=1, keepdims=True))
    bound = U[dtype] * np.abs(want) + (2 * G + 140) * EPS32 * mag + 2.0 ** -24 * (dtype == F16) + 1e-30
    assert_within(got, want, bound, "gradient")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_route_weights_are_rounded_quotients(dtype):
    """Equal logits: shares of exactly 1, their sum exact, and the weight the fp32 number nearest to the quotient."""
    for G in list(range(1, 130)) + [200, 256, 300, 511, 777, 1024]:
        _, w = qg.mm_route_topk(torch.full((2, G), 0.75, dtype=dtype, device=DEV), 1, 0)
        assert (w.cpu().numpy() == np.float32(1) / np.float32(G)).all(), G
    for k in range(1, 33):
        _, w = qg.mm_route_topk(torch.full((2, 40), -3.0, dtype=dtype, device=DEV), k, 1)
        assert (w.cpu().numpy() == np.float32(1) / np.float32(k)).all(), k


@pytest.mark.parametrize("T,G,k", [(33, 64, 4), (21, 17, 9), (5, 256, 8), (3, 777, 11)])
@pytest.mark.parametrize("normalize", [0, 1])
def test_route_topk_masked_rows_f16(T, G, k, normalize):
    _check_route(_logits(T, G, F16, T * G, masked=True), k, normalize)


_LOWEST = {F32: -3.4028234663852886e38, BF16: -3.3895313892515355e38, F16: -65504.0}
_SUBNORMAL = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("G,k", [(16, 6), (16, 12), (100, 12)])
def test_route_topk_ties_zeros_subnormals_and_lowest_values(dtype, G, k):
    """The order of equal logits, of the two zeros, of the smallest numbers and of the type's most negative ones."""
    inf, tiny, low = float("inf"), _SUBNORMAL[dtype], _LOWEST[dtype]
    rows = [[0.0, -0.0, 1.0, 1.0, 1.0, -0.0, 0.0, 0.5],
            [tiny, 0.0, -tiny, 2 * tiny, -2 * tiny, -0.0, tiny, 3 * tiny],
            [low, -inf, low, float("nan"), low, -1.0, -inf, low],
            [inf, low, -low, inf, -inf, 0.0, float("nan"), -low]]
    l = torch.full((len(rows), G), -inf)
    l[:, G - 8:] = torch.tensor(rows)
    l = l.to(dtype)
    for normalize in (0, 1):
        idx, w = qg.mm_route_topk(l.to(DEV), k, normalize)
        ri, rw = select.route_topk(to_np(l), k, normalize)
        assert idx.cpu().numpy().tolist() == ri.tolist()
        assert_within(w, rw, (G + 60) * EPS32 * rw + 1e-30, "weights")
    idx, w = qg.mm_route_topk(torch.full((4, 200), low, dtype=dtype, device=DEV), k, 0)
    assert idx.cpu().tolist() == [list(range(k))] * 4
    assert torch.allclose(w, torch.full_like(w, 1 / 200))


# ------------------------------------------------------------------ mixture-of-experts layer


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("T,G,S,K,F,N", [(5, 4, 2, 128, 256, 136), (40, 3, 3, 192, 200, 128)])
def test_moe_layer_infinite_weights_of_the_second_product(T, G, S, K, F, N, act, dtype, tensor_path):  # noqa: F811
    """Infinite values of w_down give the infinity or NaN that the formula gives, whatever parts h is held in."""
    x, wg, wu, wd, idx, w = _moe_inputs(T, G, S, K, F, N, dtype, T + F)
    rng = np.random.default_rng(T)
    for e in range(G):
        f = rng.integers(0, F, size=6)
        wd[e, f[0], 3], wd[e, f[1], 7], wd[e, f[2], N - 1] = float("inf"), float("-inf"), float("inf")
        wd[e, f[3], 20], wd[e, f[4], 20] = float("inf"), float("-inf")    # may meet in one sum
    out = to_np(qg.mm_moe_layer(x, wg, wu, wd, idx, w, act))
    assert qg.mm_last_path() == qg.MM_PATH_TENSOR
    args = [to_np(t) for t in (x, wg, wu, wd, idx, w)]
    with np.errstate(invalid="ignore"):
        want = select.moe_layer(*args, activation=act)
    assert np.isinf(want).any()
    assert (np.isnan(out) == np.isnan(want)).all()
    assert (np.isposinf(out) == np.isposinf(want)).all() and (np.isneginf(out) == np.isneginf(want)).all()
    ok = np.isfinite(want)
    args[3] = np.where(np.isfinite(args[3]), args[3], 0.0)
    bound = select.moe_layer_bound(*args, activation=act, u=U[dtype])
    assert (np.abs(out[ok] - want[ok]) <= (bound + 1e-30)[ok]).all()


def _rms(a):
    return float(np.sqrt(np.mean(np.square(a))))


def _rounded(want, dtype):
    return torch.from_numpy(want).to(dtype).double().numpy()


@pytest.mark.parametrize("scale", [4.0, 1.0, 2.0 ** -8, 2.0 ** -24])
def test_moe_layer_hidden_values_over_f16s_range(scale, tensor_path):  # noqa: F811
    """h (not x or the weights) far from 1 in f16: up to half a million, and down to where h itself is below 2^-17."""
    T, G, S, K, F, N = 6, 4, 2, 128, 512, 128
    x, wg, wu, wd, idx, w = _moe_inputs(T, G, S, K, F, N, F16, 17)
    wg, wu = (wg * (180 * scale) ** 0.5).to(F16), (wu * (180 * scale) ** 0.5).to(F16)
    if scale > 1:
        wg, wu, wd = wg * 8, wu * 8, wd * 2.0 ** -10
    elif scale < 1:
        wd = (wd * (2.0 ** 6 if scale > 2.0 ** -10 else 2.0 ** 14)).to(F16)
    out = qg.mm_moe_layer(x, wg, wu, wd, idx, w, "relu")
    assert qg.mm_last_path() == qg.MM_PATH_TENSOR
    args = [to_np(t) for t in (x, wg, wu, wd, idx, w)]
    want = select.moe_layer(*args, activation="relu")
    h = np.concatenate([np.abs(np.maximum(args[0] @ args[1][e], 0) * (args[0] @ args[2][e])).ravel() for e in range(G)])
    assert (h.max() > 65504) == (scale > 1) and h.max() < 2.0 ** 20
    assert (np.sqrt(np.mean(h ** 2)) < 2.0 ** -16) == (scale < 2.0 ** -10)
    assert np.isfinite(to_np(out)).all()
    # h in two parts: an error of at most 2^-22 of h, or 2^-32; the output's own rounding dominates.
    once = _rms(_rounded(want, F16) - want)
    floor = 2.0 ** -32 * _rms(args[3]) * F ** 0.5
    assert _rms(to_np(out) - want) <= 1.05 * (once + floor) + 2.0 ** -19 * _rms(want)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,G,S,K,F,N", [(7, 5, 2, 256, 512, 256), (33, 6, 3, 1024, 768, 520), (4, 2, 2, 2048, 1536, 1024)])
def test_moe_layer_error_in_the_mean_is_one_rounding_of_the_output(T, G, S, K, F, N, dtype, tensor_path):  # noqa: F811
    """h is not rounded to the tensors' type between the products: an h rounded once adds an error of the size of the
    output's own rounding, sqrt(2) of it in the mean; two parts of h and fp32 sums add less than 1 % to it."""
    args = _moe_inputs(T, G, S, K, F, N, dtype, T + F)
    out = to_np(qg.mm_moe_layer(*args))
    want = select.moe_layer(*[to_np(t) for t in args])
    assert _rms(out - want) <= 1.05 * _rms(_rounded(want, dtype) - want)


def test_a_hidden_value_rounded_once_would_be_seen():
    """The check above on the formula with h rounded to the type: it must fail there."""
    for dtype in (BF16, F16):
        x, wg, wu, wd, idx, w = [to_np(t) for t in _moe_inputs(7, 5, 2, 256, 512, 256, dtype, 19)]
        want, got = select.moe_layer(x, wg, wu, wd, idx, w), np.zeros((7, 256))
        for t, s in np.ndindex(*idx.shape):
            e = idx[t, s]
            h = select.activate(x[t] @ wg[e], "silu") * (x[t] @ wu[e])
            got[t] += w[t, s] * (_rounded(h, dtype) @ wd[e])
        got = _rounded(got, dtype)
        assert _rms(got - want) > 1.2 * _rms(_rounded(want, dtype) - want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_moe_layer_gelu_of_negative_values(dtype):
    """g/2 (1 + erf(g / sqrt 2)) where erf is close to -1: the value's own digits, not those left of 1 - 1."""
    F = 64 if dtype == F32 else 256
    K = 1 if dtype == F32 else 64
    g = torch.linspace(-9.0, -2.5, F).to(dtype)
    x = torch.zeros((1, K), dtype=dtype)
    x[0, 0] = 1.0                                               # x w_gate is exact
    wg = torch.zeros((1, K, F), dtype=dtype)
    wg[0, 0] = g
    wd = torch.ones((1, F, 8), dtype=dtype)
    wd[0, :, 1:] = torch.nn.functional.one_hot(torch.arange(F) * 7 // F, 7).to(dtype)    # bands of g, small ones alone
    idx = torch.zeros((1, 1), dtype=torch.int32)
    out = qg.mm_moe_layer(x.to(DEV), wg.to(DEV), None, wd.to(DEV), idx.to(DEV), None, "gelu")
    from math import erfc
    h = np.array([0.5 * v * erfc(-v / np.sqrt(2.0)) for v in g.double().tolist()])
    want = h @ to_np(wd)[0]
    # the argument g / sqrt 2 carries two roundings, which erfc(z) takes 2 z^2 = g^2 times; erfc and the products 8
    # more, h in two parts (bf16) 2^-17, the sum F, the output u
    rel = (2 * 81 + 8 + F) * EPS32 + (2.0 ** -17 + U[BF16] if dtype == BF16 else 0)
    assert_within(out, want[None], rel * np.abs(want)[None])


# ------------------------------------------------------------------ low-rank adapters


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", [(1, 512, 1024), (3, 1024, 520), (17, 512, 1024), (64, 1024, 2048), (130, 512, 520),
                                   (256, 256, 1024)])
def test_projection_adds_what_the_expansion_has_just_written(M, K, N, dtype):
    """Y is written, read and written again within one call while its launches overlap: always with the same output
    memory and other values in it before, the same bits as in fresh memory."""
    X, W, A, B, idx, scales, _ = _lowrank_inputs(M, K, N, 16, 6, dtype, 231)
    inputs = [X * s for s in (1.0, -0.5, 2.0, -4.0)]
    fresh = [qg.mm_lowrank_matmul(x, W, A, B, idx, scales, out=torch.zeros((M, N), dtype=dtype, device=DEV)) for x in inputs]
    out = torch.empty((M, N), dtype=dtype, device=DEV)
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(60):
        qg.mm_lowrank_matmul(inputs[i % 4], W, A, B, idx, scales, out=out)
        differ += (out != fresh[i % 4]).sum()
    assert differ.item() == 0
    args = [to_np(t) for t in (inputs[3], W, A, B, idx, scales)]
    assert_within(fresh[3], select.lowrank_matmul(*args), select.lowrank_matmul_bound(*args, u=U[dtype]))



@pytest.mark.parametrize("M", [40, 200, 300, 700])
def test_lowrank_factors_past_f16s_range(M):
    """X A above f16's largest value, B small: Y lies well inside the range, whichever kernel the row count selects."""
    X, W, A, B, idx, scales, _ = _lowrank_inputs(M, 256, 264, 16, 4, F16, 201)
    X, A, B = X * 64, A * 600, (B * 2.0 ** -10).to(F16)
    args = [to_np(t) for t in (X, W, A, B, idx, scales)]
    z = np.concatenate([args[5][g] * (args[0][args[4] == g] @ args[2][g]) for g in range(4)])
    assert (np.abs(z).max(axis=1) > 65504).any() and (np.abs(z).max(axis=1) < 65504).any()
    assert_within(qg.mm_lowrank_matmul(X, W, A, B, idx, scales), select.lowrank_matmul(*args),
                  select.lowrank_matmul_bound(*args, u=U[F16]))


@pytest.mark.parametrize("M,R,runs", [(300, 16, 0), (700, 40, 1), (1100, 8, 1)])
@pytest.mark.parametrize("big", ["V", "U"])
def test_lowrank_gradients_of_factors_at_both_ends_of_f16s_range(M, R, runs, big):
    """V = s dY B^T above f16's largest value beside U = s X A below its smallest, and the reverse."""
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, 256, 264, R, 4, F16, 211, runs)
    if big == "V":           # dX and dA inside the range through small A and X, dB through a large dY
        dY, B, X, A, scales = dY * 4096, B * 16, X * 2.0 ** -12, A * 2.0 ** -10, scales * 2.0 ** -2
    else:                    # a large U with a small dY, and V below 2^-24
        dY, B, X, A = dY * 2.0 ** -12, (B * 2.0 ** -14).to(F16), X * 4096, A * 64
    W = (W * 2.0 ** -4).to(F16)
    args = [to_np(t) for t in (dY, X, W, A, B, idx, scales)]
    V = np.concatenate([args[6][g] * (args[0][args[5] == g] @ args[4][g].T) for g in range(4)])
    Uf = np.concatenate([args[6][g] * (args[1][args[5] == g] @ args[3][g]) for g in range(4)])
    large, small = (V, Uf) if big == "V" else (Uf, V)
    assert np.abs(large).max() > 65504 and _rms(small) < 2.0 ** -17
    got = qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales)
    for name, g, want, bound in zip(("dX", "dA", "dB"), got, select.lowrank_matmul_grad(*args),
                                    select.lowrank_matmul_grad_bound(*args, u=U[F16])):
        assert_within(g, want, bound, name)
        # in the mean: the output's own rounding and 5 % of it; where V is past the range, dX takes that part of itself
        # as one value of the type, an error of the same size
        most = 1.5 if (name, big) == ("dX", "V") else 1.05
        assert _rms(to_np(g) - want) <= most * _rms(_rounded(want, F16) - want) + 2.0 ** -19 * _rms(want), name


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N,R,G,runs", [(700, 256, 264, 16, 4, 1), (1040, 264, 520, 12, 3, 0), (600, 512, 256, 32, 2, 1)])
def test_lowrank_error_in_the_mean_is_one_rounding_of_the_output(M, K, N, R, G, runs, dtype):
    """Many rows: the factors are not rounded to the tensors' type on their way into the products.  (One rounding of a
    factor adds an error of the size of the output's: sqrt(2) of it in the mean for dA and dB.)"""
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, K, N, R, G, dtype, M + R, runs)
    B = B * 4                                                   # the low-rank part dominates Y and dX
    args = [to_np(t) for t in (X, W, A, B, idx, scales)]
    Y, want = to_np(qg.mm_lowrank_matmul(X, W, A, B, idx, scales)), select.lowrank_matmul(*args)
    assert _rms(Y - want) <= 1.05 * _rms(_rounded(want, dtype) - want)
    got = qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales)
    for name, g, want in zip(("dX", "dA", "dB"), got, select.lowrank_matmul_grad(to_np(dY), *args)):
        assert _rms(to_np(g) - want) <= 1.05 * _rms(_rounded(want, dtype) - want), name


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N,R,G", [(300, 136, 264, 200, 3), (2000, 72, 136, 72, 600), (1100, 264, 72, 8, 1024)])
def test_lowrank_gradients_of_many_adapters_and_ranks(M, K, N, R, G, dtype):
    """Several groups of 64 ranks, more adapters than rows have, all three gradients and each pair."""
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, K, N, R, G, dtype, M + R)
    full = _check_lowrank_grad(dY, X, W, A, B, idx, scales)
    for need in ((True, True, False), (True, False, True), (False, True, True)):
        for f, p in zip(full, qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales, need=need)):
            assert p is None or torch.equal(f, p)


@pytest.mark.parametrize("R", [16, 72])
def test_lowrank_gradients_of_rows_of_very_different_size_f16(R):
    """Rows of one adapter whose factors lie up to 2^20 apart, in no order: each row's part of the sum to its own scale."""
    M, K, N, G = 900, 136, 72, 2
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, K, N, R, G, F16, 241)
    rng = np.random.default_rng(5)
    size = torch.from_numpy(2.0 ** rng.integers(-10, 11, size=(M, 1))).to(DEV)
    X, dY = (X * size).to(F16), (dY / size).to(F16)             # U as large as X, V as small as dY
    W = (W * 2.0 ** -8).to(F16)
    args = [to_np(t) for t in (dY, X, W, A, B, idx, scales)]
    got = qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales)
    for name, g, want, bound in zip(("dX", "dA", "dB"), got, select.lowrank_matmul_grad(*args),
                                    select.lowrank_matmul_grad_bound(*args, u=U[F16])):
        assert_within(g, want, bound, name)
        assert _rms(to_np(g) - want) <= 1.05 * _rms(_rounded(want, F16) - want) + 2.0 ** -19 * _rms(want), name


def _constant(name):
    import os
    import re

    with open(os.path.join(os.path.dirname(qg.__file__), "csrc", "lowrank.cuh")) as f:
        return int(re.search(r"constexpr int %s = (\d+);" % name, f.read()).group(1))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N,R,G", [(3400, 48, 136, 1, 200), (4200, 40, 72, 2500, 100)])
def test_lowrank_rows_past_the_slots_or_the_list_are_rounded_once(M, K, N, R, G, dtype):
    """Rows of more adapters than the product holds copies of, or than a row tile lists: the projection's sum is not
    rounded before the low-rank part joins it."""
    X, W, A, B, idx, scales, _ = _lowrank_inputs(M, K, N, R, G, dtype, M)
    args = [to_np(t) for t in (X, W, A, B, idx, scales)]
    slots, per_tile = _constant("kSlots"), _constant("kSlots")
    while per_tile > 16 and per_tile * ((M + 255) // 256 * 256 * ((R + 63) // 64 * 64) * 2) > 256 << 20:
        per_tile //= 2
    per_tile = min(per_tile, G)
    used = np.unique(args[4][args[4] >= 0])
    named = max(len(np.unique(args[4][t:t + 256][args[4][t:t + 256] >= 0])) for t in range(0, M, 256))
    assert len(used) > slots or named > per_tile
    assert G < (M + 15) // 16                                   # not the few-row kernels
    want = select.lowrank_matmul(*args)
    base, zero = np.abs(args[0]) @ np.abs(args[1]), np.zeros_like(args[1])
    low = select.lowrank_matmul(np.abs(args[0]), zero, np.abs(args[2]), np.abs(args[3]), args[4], args[5])
    u = U[dtype]                     # Y's rounding, and one or two of the low-rank part
    assert_within(qg.mm_lowrank_matmul(X, W, A, B, idx, scales), want,
                  u * np.abs(want) + 2.01 * u * low + (2 * K + R) * EPS32 * (base + low) + 2.0 ** -24)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("layout", ["rows", "columns", "odd"])
@pytest.mark.parametrize("M", [1, 2, 4, 7, 33, 64])
def test_lowrank_error_of_few_rows_in_the_mean_is_one_rounding_of_the_output(M, layout, dtype):
    """Up to 64 rows: the low-rank part is not rounded on its way to the projection (rounded, and as large as the whole,
    it would add an error of the size of the output's own rounding)."""
    K, N = (512, 1032) if layout != "odd" else (509, 1031)
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, K, N, 16, 6, dtype, 251 + M)
    B, idx = B * 4, idx.clamp(min=0)
    if layout == "columns":
        W, A, B = W.t().contiguous().t(), *(t.transpose(1, 2).contiguous().transpose(1, 2) for t in (A, B))
    args = [to_np(t) for t in (X, W, A, B, idx, scales)]
    Y, want = to_np(qg.mm_lowrank_matmul(X, W, A, B, idx, scales)), select.lowrank_matmul(*args)
    assert _rms(Y - want) <= 1.05 * _rms(_rounded(want, dtype) - want)
    dX, want = qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales)[0], select.lowrank_matmul_grad(to_np(dY), *args)[0]
    assert _rms(to_np(dX) - want) <= 1.05 * _rms(_rounded(want, dtype) - want)


@pytest.mark.parametrize("M", [1, 3, 40])
def test_lowrank_part_past_f16s_range_that_the_projection_brings_back(M):
    """The low-rank part alone is above f16's largest value, Y = X W plus it is not."""
    K, N, R = 64, 264, 8
    X, W, A, B = (torch.zeros(s, dtype=F16, device=DEV) for s in ((M, K), (K, N), (1, K, R), (1, R, N)))
    X[:, 0], W[0], A[0, 0, 0], B[0, 0] = 256.0, -160.0, 1.0, 300.0          # -40960 and 76800
    X[:, 1], W[1] = 1.0, torch.arange(N, device=DEV).to(F16)
    idx = torch.zeros(M, dtype=torch.int32, device=DEV)
    want = select.lowrank_matmul(*[to_np(t) for t in (X, W, A, B)], np.zeros(M, int))
    assert (to_np(qg.mm_lowrank_matmul(X, W, A, B, idx)) == _rounded(want, F16)).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("R,chunks", [(1, 1), (8, 1), (16, 3), (72, 1)])
def test_lowrank_gradients_of_infinite_inputs(R, chunks, dtype):
    """Infinite values of X or dY give dA and dB the infinity or NaN of the formula, whatever parts the factors are held
    in, and leave the other adapters', columns' and rows' values alone."""
    M, K, N, G = 300 + 1100 * (chunks - 1), 136, 264, 4
    X, W, A, B, _, scales, dY = _lowrank_inputs(M, K, N, R, G, dtype, 261)
    idx = torch.arange(M, device=DEV) % (G + 1) - 1 if chunks == 1 else torch.where(torch.arange(M, device=DEV) < 4, 1, 0)
    A, B = torch.where(A == 0, 1, A), torch.where(B == 0, 1, B)
    X[dY.abs().amin(dim=1) == 0], dY[dY == 0] = 1, 1
    inf = float("inf")
    for m, c, v in ((6, 3, inf), (6, 9, -inf), (7, 70, inf), (11, 70, -inf), (2, 5, inf)):
        X[m, c] = v                                             # adapter m % 5 - 1, or chunks' adapter 0
    for m, c, v in ((8, 100, inf), (13, 100, inf), (18, 101, -inf), (3, 7, -inf)):
        dY[m, c] = v
    args = [to_np(t) for t in (dY, X, W, A, B, idx, scales)]
    got = qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales)
    with np.errstate(invalid="ignore"):
        wants = select.lowrank_matmul_grad(*args)
    zero = [np.where(np.isfinite(a), a, 0.0) for a in args[:2]] + args[2:]
    bounds = select.lowrank_matmul_grad_bound(*zero, u=U[dtype])
    for name, g, want, bound in zip(("dX", "dA", "dB"), got, wants, bounds):
        g, ok = to_np(g), np.isfinite(want)
        assert not ok.all(), name
        assert (np.isnan(g) == np.isnan(want)).all(), name
        assert (np.isposinf(g) == np.isposinf(want)).all() and (np.isneginf(g) == np.isneginf(want)).all(), name
        assert (np.abs(g[ok] - want[ok]) <= bound[ok]).all(), name


# ------------------------------------------------------------------ streams


@pytest.mark.parametrize("call", ["matmul", "gemm", "qlinear", "grouped", "qweights", "noalloc", "route", "route_grad", "moe",
                                  "lowrank", "lowrank_grad"])
def test_outputs_of_a_call_on_another_stream_are_not_memory_still_in_use(call):
    """Memory freed on the current stream is handed out again at once, ordered by that stream alone: a call on another
    stream that took it would write while the current stream's work still does."""
    x, wg, wu, wd, idx, w = _moe_inputs(64, 4, 2, 256, 256, 256, BF16, 221)
    *lr, dY = _lowrank_inputs(64, 256, 256, 16, 4, BF16, 222)
    q8 = torch.randint(-100, 100, (64, 256), dtype=torch.int8, device=DEV)
    sc, zp = torch.tensor(0.02, device=DEV), torch.tensor(3, dtype=torch.int8, device=DEV)
    wq = torch.randint(-100, 100, (4, 256, 256), dtype=torch.int8, device=DEV)
    ws = torch.rand((4, 1, 256), device=DEV).to(BF16)
    ri, rw = qg.mm_route_topk(x, 4)
    calls = {"matmul": lambda s: qg.mm_matmul(x, wg[0], stream=s),
             "gemm": lambda s: qg.mm_gemm(x, wg[0], stream=s),
             "qlinear": lambda s: qg.mm_qlinear_matmul(q8, sc, zp, q8.t(), sc, zp, sc, zp, stream=s),
             "grouped": lambda s: qg.mm_grouped_matmul(x, wg, idx, stream=s),
             "qweights": lambda s: qg.mm_grouped_matmul_qweights(x, wq, ws, None, 0, idx, stream=s),
             "noalloc": lambda s: qg.mm_grouped_matmul_noalloc(x, wg, idx, stream=s),
             "route": lambda s: qg.mm_route_topk(x, 4, stream=s),
             "route_grad": lambda s: qg.mm_route_topk_grad(x, ri, rw, stream=s),
             "moe": lambda s: qg.mm_moe_layer(x, wg, wu, wd, idx, w, stream=s),
             "lowrank": lambda s: qg.mm_lowrank_matmul(*lr, stream=s),
             "lowrank_grad": lambda s: qg.mm_lowrank_matmul_grad(dY, *lr, stream=s)}

    def run(stream):
        got = calls[call](stream)
        return list(got) if isinstance(got, tuple) else [got]

    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sizes = sorted({t.numel() * t.element_size() for t in want} | {1 << n for n in range(9, 25)})
    junk = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    torch.cuda._sleep(100_000_000)
    for t in junk:
        t.fill_(0xFF)                                    # still to run when the call below is made
    del junk, t
    got = run(side)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    for t in got:                                        # and the outputs are good for the current stream's work
        t.add_(1)


# ------------------------------------------------------------------ the profiles' command


@pytest.mark.parametrize("workload", ["operator_route_decode", "operator_moe_small_g8", "operator_lowrank_grad_ragged"])
def test_the_profiles_command_runs(workload):
    import json
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "bench.py"), "--profile-workload", workload, "--steps", "2",
                        "--warmup", "3"], capture_output=True, text=True, cwd=root)
    assert r.returncode == 0, r.stderr
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["profile_workload"] == workload and line["status"] == "MM_OK"
