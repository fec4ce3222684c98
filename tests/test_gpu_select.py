"""Top-k routing, the mixture-of-experts layer and per-row low-rank adapters against the float64 oracle.

Tolerances are the oracle's bounds: a unit roundoff u of the tensors' type for
each rounding an operator states, plus fp32 sums taken at their worst.
"""

import numpy as np
import pytest
import torch

import quantized_gemm_gb300 as qg
from helpers import rand_tensor, to_np
from oracle import select

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def clean_status():
    qg.mm_get_device_status()
    yield
    assert qg.mm_get_device_status() == "MM_OK"


def assert_within(got, want, bound, what=""):
    got = to_np(got)
    assert np.isfinite(got).all(), what
    worst = np.max(np.abs(got - want) / bound) if got.size else 0.0
    assert worst <= 1.0, "%s: %g of the bound" % (what, worst)


# ------------------------------------------------------------------ routing


def _logits(T, G, dtype, seed, masked):
    l = rand_tensor((T, G), F32, seed, "cpu") * 2
    if masked and T:
        rng = np.random.default_rng(seed)
        l[torch.from_numpy(rng.random((T, G)) < 0.3)] = float("-inf")
        l[torch.from_numpy(rng.random((T, G)) < 0.02)] = float("nan")
        l[T // 2] = float("-inf")
        l[0, G // 2] = float("inf")
    return l.to(dtype).to(DEV)


def _check_route(l, k, normalize):
    G = l.shape[1]
    idx, w = qg.mm_route_topk(l, k, normalize)
    ri, rw = select.route_topk(to_np(l), k, normalize)
    assert np.array_equal(idx.cpu().numpy(), ri)
    # exp's argument is exact to 2^-24 of |l - max| <= 40 here; sums of at most G terms
    assert_within(w, rw, (G + 60) * U[F32] * rw + 1e-30, "weights")
    dw = rand_tensor((l.shape[0], k), F32, 5, DEV)
    for ii in (idx, idx.long()):
        g = qg.mm_route_topk_grad(l, ii, dw, normalize)
        assert g.dtype == l.dtype
        want = select.route_topk_grad(to_np(l), ri, to_np(dw), normalize)
        p, d = np.zeros(l.shape), np.zeros(l.shape)
        for t in range(l.shape[0]):
            p[t] = select._softmax_row(to_np(l)[t])[0]
            if normalize:
                keep = np.isin(np.arange(G), ri[t])
                p[t] = np.where(keep, p[t], 0)
                p[t] /= max(p[t].sum(), 1e-300)
            for r in range(k):
                if ri[t, r] >= 0:
                    d[t, ri[t, r]] = abs(to_np(dw)[t, r])
        mag = p * (d + (p * d).sum(axis=1, keepdims=True))
        assert_within(g, want, U[l.dtype] * np.abs(want) + (2 * G + 140) * U[F32] * mag + 2.0 ** -24 * (l.dtype == F16) +
                      1e-30, "gradient")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,G,k", [(1, 1, 1), (1, 64, 2), (3, 5, 5), (37, 64, 8), (5, 65, 3), (16, 100, 16), (9, 256, 8),
                                   (4, 300, 32), (3, 1000, 7), (2, 1024, 32), (1000, 8, 2), (7, 40, 20)])
@pytest.mark.parametrize("normalize", [0, 1])
def test_route_topk(T, G, k, dtype, normalize):
    _check_route(_logits(T, G, dtype, T + G, masked=False), k, normalize)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,G,k", [(33, 64, 4), (21, 17, 9), (5, 256, 8), (3, 777, 11)])
@pytest.mark.parametrize("normalize", [0, 1])
def test_route_topk_masked_rows(T, G, k, dtype, normalize):
    _check_route(_logits(T, G, dtype, T * G, masked=True), k, normalize)


def test_route_topk_ties_and_signed_zeros():
    l = torch.tensor([[0.0, -0.0, 1.0, 1.0, 1.0, -0.0, 0.0, 0.5]] * 3, device=DEV)
    idx, w = qg.mm_route_topk(l, 6, 1)
    assert idx.cpu().tolist() == [[2, 3, 4, 7, 0, 1]] * 3
    idx, w = qg.mm_route_topk(torch.full((4, 200), -3.4028234663852886e38, device=DEV), 4, 0)
    assert idx.cpu().tolist() == [[0, 1, 2, 3]] * 4
    assert torch.allclose(w, torch.full_like(w, 1 / 200))


def test_route_topk_strided_views():
    base = rand_tensor((40, 90), F32, 8, DEV)
    for l in (base[::2, 3:70], base.t()[:, 1::3], base[1:2].expand(6, 90)):
        _check_route(l, 4, 1)


def test_route_topk_no_rows():
    idx, w = qg.mm_route_topk(torch.empty((0, 16), device=DEV), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    assert qg.mm_route_topk_grad(torch.empty((0, 16), device=DEV), idx, w).shape == (0, 16)


def test_route_gradient_records_an_index_out_of_range():
    l = rand_tensor((2, 8), F32, 9, DEV)
    idx = torch.tensor([[1, 8], [-2, -1]], dtype=torch.int32, device=DEV)
    g = qg.mm_route_topk_grad(l, idx, torch.ones((2, 2), device=DEV), 0)
    assert qg.mm_get_device_status() == "MM_ERR_INDEX_RANGE"
    want = select.route_topk_grad(to_np(l), np.array([[1, -1], [-1, -1]]), np.ones((2, 2)), 0)
    np.testing.assert_allclose(to_np(g), want, atol=1e-6)


# ------------------------------------------------------------------ mixture-of-experts layer


def _moe_inputs(T, G, S, K, F, N, dtype, seed, up=True):
    x = rand_tensor((T, K), dtype, seed, DEV)
    wg = (rand_tensor((G, K, F), F32, seed + 1, DEV) * K ** -0.5).to(dtype)
    wu = (rand_tensor((G, K, F), F32, seed + 2, DEV) * K ** -0.5).to(dtype) if up else None
    wd = (rand_tensor((G, F, N), F32, seed + 3, DEV) * max(F, 1) ** -0.5).to(dtype)
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, G)), axis=1)[:, :S].astype(np.int32)
    w = rng.random((T, S)).astype(np.float32)
    return x, wg, wu, wd, torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV)


def _check_moe(x, wg, wu, wd, idx, w, act="silu", **kw):
    out = qg.mm_moe_layer(x, wg, wu, wd, idx, w, act, **kw)
    args = [None if t is None else to_np(t) for t in (x, wg, wu, wd, idx, w)]
    want = select.moe_layer(*args, activation=act)
    bound = select.moe_layer_bound(*args, activation=act, u=U[x.dtype])
    assert_within(out, want, bound + 1e-30, "moe")
    return out


MOE = [(1, 1, 1, 1, 1, 1), (1, 8, 2, 256, 384, 256), (3, 8, 4, 200, 136, 200), (16, 4, 2, 128, 128, 128),
       (17, 5, 3, 264, 72, 520), (64, 16, 2, 128, 256, 136), (40, 3, 3, 512, 64, 64), (130, 6, 2, 64, 128, 72),
       (5, 7, 2, 33, 19, 21), (2, 40, 8, 1000, 712, 1000)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,G,S,K,F,N", MOE)
def test_moe_layer(T, G, S, K, F, N, dtype):
    _check_moe(*_moe_inputs(T, G, S, K, F, N, dtype, T + K))


@pytest.fixture
def tensor_path():
    qg.mm_set_path_policy(qg.MM_PATH_TENSOR)
    yield
    qg.mm_set_path_policy(qg.MM_PATH_AUTO)


# sizes at the tiles' edges (128 columns, 64 k, 16 tokens, 128 tokens a pass) and shares of a few blocks
MOE_TC = [(1, 1, 1, 8, 8, 8), (1, 3, 1, 64, 128, 128), (2, 2, 2, 72, 136, 8), (15, 9, 4, 128, 120, 248),
          (16, 200, 8, 64, 64, 64), (17, 2, 1, 520, 264, 136), (33, 300, 3, 128, 72, 264), (127, 5, 2, 256, 128, 72),
          (128, 4, 4, 192, 136, 128), (129, 4, 2, 64, 64, 64), (300, 7, 3, 128, 192, 200), (4, 2, 2, 2048, 1536, 1024)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,G,S,K,F,N", MOE_TC)
def test_moe_layer_on_the_tensor_cores(T, G, S, K, F, N, dtype, tensor_path):
    args = _moe_inputs(T, G, S, K, F, N, dtype, T + K + G)
    out = _check_moe(*args)
    assert qg.mm_last_path() == qg.MM_PATH_TENSOR
    for _ in range(2):
        assert torch.equal(out, qg.mm_moe_layer(*args))


def test_moe_layer_uneven_experts_on_the_tensor_cores(tensor_path):
    x, wg, wu, wd, idx, w = _moe_inputs(100, 8, 2, 256, 320, 256, BF16, 23)
    idx[:, 0] = 1                     # one expert with every token, one with a single one, some with none
    idx[:, 1] = torch.where(torch.arange(100, device=DEV) == 77, 6, -1)
    _check_moe(x, wg, wu, wd, idx, w)
    idx[:] = -1
    assert not qg.mm_moe_layer(x, wg, wu, wd, idx, w).any()


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_moe_layer_activations(act, up, dtype):
    _check_moe(*_moe_inputs(9, 6, 2, 192, 320, 192, dtype, 11, up=up), act=act)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_moe_layer_weight_layouts(dtype):
    x, wg, wu, wd, idx, w = _moe_inputs(6, 5, 2, 256, 128, 256, dtype, 21)
    a = qg.mm_moe_layer(x, wg, wu, wd, idx, w)
    both = torch.cat([wg, wu], dim=2)                                   # the halves of one tensor
    assert torch.equal(a, qg.mm_moe_layer(x, both[:, :, :128], both[:, :, 128:], wd, idx.long(), w))
    kt = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (wg, wu, wd)]   # stored [G, out, in]
    _check_moe(x, *kt, idx, w)
    _check_moe(x, kt[0], wu, wd, idx, w)
    _check_moe(x[:, 1:], wg[:, 1:], wu[:, 1:], wd, idx, w)              # misaligned rows of x
    _check_moe(x.t().contiguous().t(), wg, wu, wd, idx.t().contiguous().t(), w)
    wide = torch.zeros((12, 300), dtype=dtype, device=DEV)
    wide[::2, 8:264] = x
    _check_moe(wide[::2, 8:264], wg, wu, wd, idx, w[:, :1].expand(6, 2))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_moe_layer_missing_repeated_and_unweighted_picks(dtype):
    x, wg, wu, wd, idx, w = _moe_inputs(7, 5, 3, 128, 192, 128, dtype, 31)
    idx[2] = -1                       # a token without experts
    idx[3, 1] = -1
    idx[4] = idx[4, 0]                # the same expert three times
    out = _check_moe(x, wg, wu, wd, idx, w)
    assert not out[2].any()
    _check_moe(x, wg, wu, wd, idx, None)
    assert not qg.mm_moe_layer(x, wg, wu, wd, torch.full_like(idx, -1), w).any()
    assert not qg.mm_moe_layer(x, wg, wu, wd, idx[:, :0], w[:, :0]).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_moe_layer_index_out_of_range(dtype):
    x, wg, wu, wd, idx, w = _moe_inputs(4, 5, 2, 128, 128, 128, dtype, 41)
    bad = idx.clone()
    bad[1, 0], bad[2, 1] = 5, -7
    got = qg.mm_moe_layer(x, wg, wu, wd, bad, w)
    assert qg.mm_get_device_status() == "MM_ERR_INDEX_RANGE"
    idx[1, 0] = idx[2, 1] = -1
    assert torch.equal(got, qg.mm_moe_layer(x, wg, wu, wd, idx, w))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [2, 33])
def test_moe_layer_tokens_depend_on_their_own_picks_alone(dtype, T):
    x, wg, wu, wd, idx, w = _moe_inputs(T, 6, 2, 192, 160, 192, dtype, 51)
    idx = torch.where(idx == 5, 4, idx)
    idx[1:][idx[1:] == 3] = 2
    idx[0, 0] = 3                                        # expert 3 serves token 0 alone, expert 5 nobody
    want = qg.mm_moe_layer(x, wg, wu, wd, idx, w)
    for bad in (float("nan"), float("inf")):
        ws = [t.clone() for t in (wg, wu, wd)]
        for t in ws:
            t[3], t[5] = bad, bad
        xb = x.clone()
        xb[0] = bad
        got = qg.mm_moe_layer(xb, *ws, idx, w)
        assert torch.equal(got[1:], want[1:])
        assert not torch.isfinite(got[0].float()).any()


def test_moe_layer_empty_dimensions():
    x, wg, wu, wd, idx, w = _moe_inputs(3, 4, 2, 64, 64, 64, BF16, 61)
    assert qg.mm_moe_layer(x[:0], wg, wu, wd, idx[:0], w[:0]).shape == (0, 64)
    assert not qg.mm_moe_layer(x, wg[:, :, :0], wu[:, :, :0], wd[:, :0], idx, w).any()
    assert not qg.mm_moe_layer(x[:, :0], wg[:, :0], wu[:, :0], wd, idx, w).any()
    assert qg.mm_moe_layer(x, wg, wu, wd[:, :, :0], idx, w).shape == (3, 0)


def test_moe_layer_follows_the_router():
    """A whole routed layer, as a decode step runs it: router product, top-k, experts."""
    x, wg, wu, wd, _, _ = _moe_inputs(12, 16, 4, 256, 128, 256, BF16, 71)
    router = rand_tensor((256, 16), BF16, 72, DEV)
    logits = qg.mm_matmul(x, router)
    idx, w = qg.mm_route_topk(logits, 4)
    out = _check_moe(x, wg, wu, wd, idx, w)
    # the same experts through GroupedMatMul
    g, u = qg.mm_grouped_matmul(x, wg, idx).float(), qg.mm_grouped_matmul(x, wu, idx).float()
    h = (torch.nn.functional.silu(g) * u).to(BF16).reshape(48, 256 // 2)
    y = qg.mm_grouped_matmul(h, wd, idx.reshape(48, 1)).reshape(12, 4, 256).float()
    ref = (y * w[:, :, None]).sum(dim=1)
    assert (out.float() - ref).abs().max() < 0.05 * ref.abs().max()


def test_the_example_runs_the_operators_together():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    import expert_step

    block = expert_step.ExpertBlock(hidden=256, ffn=136, experts=12, picks=3, adapters=4, rank=8)
    x = rand_tensor((21, 256), BF16, 77, DEV)
    adapter = torch.arange(21, device=DEV) % 5 - 1
    y, idx, w, out = block.step(x, adapter)
    n = {k: to_np(getattr(block, k)) for k in ("W", "A", "B", "scales", "gate", "up", "down")}
    a = to_np(adapter)
    args = (to_np(x), n["W"], n["A"], n["B"], a, n["scales"])
    assert_within(y, select.lowrank_matmul(*args), select.lowrank_matmul_bound(*args, u=U[BF16]), "y")
    logits = to_np(qg.mm_matmul(y, block.router))            # each later step on the values it was given
    assert np.array_equal(idx.cpu().numpy(), select.route_topk(logits, 3, 1)[0])
    args = (to_np(y), n["gate"], n["up"], n["down"], idx.cpu().numpy(), to_np(w))
    assert_within(out, select.moe_layer(*args), select.moe_layer_bound(*args, u=U[BF16]) + 1e-30, "out")
    dy = rand_tensor((21, 256), BF16, 78, DEV)
    args = (to_np(dy), to_np(x), n["W"], n["A"], n["B"], a, n["scales"])
    for g, want, bound in zip(block.adapter_gradients(dy, x, adapter), select.lowrank_matmul_grad(*args),
                              select.lowrank_matmul_grad_bound(*args, u=U[BF16])):
        assert_within(g, want, bound)
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "expert_step.py"), "--steps", "3"],
                       capture_output=True, text=True)
    assert r.returncode == 0 and "us a step" in r.stdout, r.stderr


# ------------------------------------------------------------------ low-rank adapters


def _lowrank_inputs(M, K, N, R, G, dtype, seed, runs=False):
    X = rand_tensor((M, K), dtype, seed, DEV)
    W = (rand_tensor((K, N), F32, seed + 1, DEV) * K ** -0.5).to(dtype)
    A = (rand_tensor((G, K, R), F32, seed + 2, DEV) * K ** -0.5).to(dtype)
    B = rand_tensor((G, R, N), dtype, seed + 3, DEV)
    rng = np.random.default_rng(seed)
    idx = rng.integers(-1, G, size=M)
    if runs:
        idx = np.sort(idx)[::-1].copy()
    scales = torch.from_numpy(rng.uniform(0.5, 2.0, G).astype(np.float32)).to(DEV)
    dY = rand_tensor((M, N), dtype, seed + 4, DEV)
    return X, W, A, B, torch.from_numpy(idx.astype(np.int32)).to(DEV), scales, dY


def _check_lowrank(X, W, A, B, idx, scales, **kw):
    Y = qg.mm_lowrank_matmul(X, W, A, B, idx, scales, **kw)
    args = [None if t is None else to_np(t) for t in (X, W, A, B, idx, scales)]
    assert_within(Y, select.lowrank_matmul(*args), select.lowrank_matmul_bound(*args, u=U[X.dtype]), "lowrank")
    return Y


def _check_lowrank_grad(dY, X, W, A, B, idx, scales, **kw):
    got = qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales, **kw)
    args = [None if t is None else to_np(t) for t in (dY, X, W, A, B, idx, scales)]
    want, bound = select.lowrank_matmul_grad(*args), select.lowrank_matmul_grad_bound(*args, u=U[X.dtype])
    for name, g, w, b in zip(("dX", "dA", "dB"), got, want, bound):
        assert_within(g, w, b, name)
    return got


LOWRANK = [(1, 256, 264, 16, 4, 0), (1, 1, 1, 1, 1, 0), (5, 200, 136, 8, 3, 0), (61, 512, 520, 32, 20, 0),
           (64, 264, 256, 12, 2, 1), (129, 256, 300, 5, 6, 1), (300, 512, 256, 16, 5, 1), (777, 128, 264, 64, 3, 1),
           (515, 1024, 512, 16, 40, 0), (33, 77, 35, 3, 4, 0), (257, 1032, 648, 24, 300, 0), (600, 1024, 272, 128, 2, 1),
           (1030, 264, 520, 8, 300, 0), (530, 200, 200, 12, 9, 1)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,K,N,R,G,runs", LOWRANK)
def test_lowrank_matmul(M, K, N, R, G, runs, dtype):
    X, W, A, B, idx, scales, _ = _lowrank_inputs(M, K, N, R, G, dtype, M + K, runs)
    _check_lowrank(X, W, A, B, idx, scales)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,K,N,R,G,runs", LOWRANK)
def test_lowrank_gradients(M, K, N, R, G, runs, dtype):
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, K, N, R, G, dtype, M + K, runs)
    _check_lowrank_grad(dY, X, W, A, B, idx, scales)


@pytest.mark.parametrize("M", [4, 300])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lowrank_layouts(M, dtype):
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, 256, 384, 16, 4, dtype, 81)
    Wt = W.t().contiguous().t()                             # stored [N, K]
    At, Bt = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (A, B))
    for w, a, b in ((Wt, A, B), (W, At, B), (W, A, Bt), (Wt, At, Bt)):
        _check_lowrank(X, w, a, b, idx, scales)
        _check_lowrank_grad(dY, X, w, a, b, idx, scales)
    Xt, dYt = X.t().contiguous().t(), dY.t().contiguous().t()
    _check_lowrank(Xt, W, A, B, idx.long(), None)
    _check_lowrank_grad(dYt, Xt, W, A, B, idx.long(), None)
    _check_lowrank(X[:, 1:], W[1:], A[:, 1:, 1:], B[:, 1:], idx, scales)          # misaligned rows
    _check_lowrank_grad(dY[:, 3:], X[:, 1:], W[1:, 3:], A[:, 1:, 1:], B[:, 1:, 3:], idx, scales[:1].expand(4))
    both = torch.stack([idx, idx], dim=1)
    _check_lowrank(X, W, A, B, both[:, 0], scales)


@pytest.mark.parametrize("M", [3, 200])
def test_lowrank_rows_without_adapter(M):
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, 256, 264, 16, 3, BF16, 91)
    none = torch.full_like(idx, -1)
    _check_lowrank(X, W, A, B, none, scales)
    dX, dA, dB = _check_lowrank_grad(dY, X, W, A, B, none, scales)
    assert not dA.any() and not dB.any()
    one = torch.full_like(idx, 1)                            # adapters 0 and 2 without rows
    bad = [t.clone() for t in (A, B)]
    for t in bad:
        t[0], t[2] = float("nan"), float("inf")
    assert torch.equal(qg.mm_lowrank_matmul(X, W, *bad, one, scales), qg.mm_lowrank_matmul(X, W, A, B, one, scales))
    for a, b in zip(qg.mm_lowrank_matmul_grad(dY, X, W, *bad, one, scales),
                    qg.mm_lowrank_matmul_grad(dY, X, W, A, B, one, scales)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [6, 300])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lowrank_rows_depend_on_their_own_adapter_alone(M, dtype):
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, 256, 264, 16, 3, dtype, 95)
    idx[0], idx[1:] = 2, torch.where(idx[1:] == 2, 1, idx[1:])
    want, gw = qg.mm_lowrank_matmul(X, W, A, B, idx, scales), qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales)
    for bad in (float("nan"), float("inf")):
        Ab, Bb, Xb, dYb = A.clone(), B.clone(), X.clone(), dY.clone()
        Ab[2], Bb[2], Xb[0], dYb[0] = bad, bad, bad, bad
        got = qg.mm_lowrank_matmul(Xb, W, Ab, Bb, idx, scales)
        assert torch.equal(got[1:], want[1:]) and not torch.isfinite(got[0].float()).any()
        gx, ga, gb = qg.mm_lowrank_matmul_grad(dYb, Xb, W, Ab, Bb, idx, scales)
        assert torch.equal(gx[1:], gw[0][1:]) and torch.equal(ga[:2], gw[1][:2]) and torch.equal(gb[:2], gw[2][:2])


@pytest.mark.parametrize("M", [5, 260])
def test_lowrank_index_out_of_range(M):
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, 128, 136, 8, 3, BF16, 101)
    bad = idx.clone()
    bad[1], bad[3] = 3, -2
    Y, g = qg.mm_lowrank_matmul(X, W, A, B, bad, scales), qg.mm_lowrank_matmul_grad(dY, X, W, A, B, bad, scales)
    assert qg.mm_get_device_status() == "MM_ERR_INDEX_RANGE"
    idx[1] = idx[3] = -1
    assert torch.equal(Y, qg.mm_lowrank_matmul(X, W, A, B, idx, scales))
    for a, b in zip(g, qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_lowrank_rows_past_their_tile_list_are_rounded_once(dtype):
    """Rows of more adapters than a row tile lists: the projection's sum is not rounded before the low-rank part joins it."""
    X, W, A, B, idx, scales, _ = _lowrank_inputs(700, 48, 520, 1, 71, dtype, 105)
    args = [to_np(t) for t in (X, W, A, B, idx, scales)]
    want = select.lowrank_matmul(*args)
    base, zero = np.abs(args[0]) @ np.abs(args[1]), np.zeros_like(args[1])
    low = select.lowrank_matmul(np.abs(args[0]), zero, np.abs(args[2]), np.abs(args[3]), args[4], args[5])
    u = U[dtype]                     # Y's rounding, and one or two of the low-rank part
    assert_within(qg.mm_lowrank_matmul(X, W, A, B, idx, scales), want,
                  u * np.abs(want) + 2.01 * u * low + 2 * 48 * U[F32] * (base + low) + 2.0 ** -24)


# Rows in random order name most adapters in every row tile: more than a warp
# of them, more than the product holds copies of, and (ranks this large) more
# than a tile lists.
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N,R,G", [(1040, 264, 520, 24, 40), (2100, 256, 264, 16, 131), (2600, 136, 272, 72, 160),
                                       (1100, 64, 264, 2048, 68), (1200, 256, 264, 16, 80)])
def test_lowrank_many_adapters_in_every_tile(M, K, N, R, G, dtype):
    X, W, A, B, idx, scales, dY = _lowrank_inputs(M, K, N, R, G, dtype, M + G)
    _check_lowrank(X, W, A, B, idx, scales)
    _check_lowrank_grad(dY, X, W, A, B, idx, scales)


def test_lowrank_empty_dimensions():
    X, W, A, B, idx, scales, dY = _lowrank_inputs(6, 64, 72, 8, 3, BF16, 111)
    assert qg.mm_lowrank_matmul(X[:0], W, A, B, idx[:0], scales).shape == (0, 72)
    _, dA, dB = qg.mm_lowrank_matmul_grad(dY[:0], X[:0], W, A, B, idx[:0], scales)
    assert not dA.any() and not dB.any()
    _check_lowrank(X, W, A[:, :, :0], B[:, :0], idx, scales)
    assert qg.mm_lowrank_matmul(X, W[:, :0], A, B[:, :, :0], idx, scales).shape == (6, 0)
    none = torch.full_like(idx, -1)
    assert torch.equal(qg.mm_lowrank_matmul(X, W, A[:0], B[:0], none, scales[:0]),
                       qg.mm_lowrank_matmul(X, W, A, B, none, scales))
    assert not qg.mm_lowrank_matmul(X[:, :0], W[:0], A[:, :0], B, idx, scales).any()


def test_lowrank_wanted_gradients_only():
    X, W, A, B, idx, scales, dY = _lowrank_inputs(50, 128, 136, 8, 3, BF16, 121)
    full = qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
        part = qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales, need=need)
        for f, p, n in zip(full, part, need):
            assert (p is not None) == n and (p is None or torch.equal(f, p))


def test_lowrank_gradient_against_differences():
    """The kernels' gradients in a random direction against differences of the float64 forward form."""
    X, W, A, B, idx, scales, dY = _lowrank_inputs(70, 96, 104, 8, 3, F32, 131)
    grads = qg.mm_lowrank_matmul_grad(dY, X, W, A, B, idx, scales)
    n = [to_np(t) for t in (X, W, A, B, idx, scales)]
    rng = np.random.default_rng(7)
    for at, g in zip((0, 2, 3), grads):
        d = rng.normal(size=n[at].shape)
        hi, lo = list(n), list(n)
        hi[at], lo[at] = n[at] + 1e-6 * d, n[at] - 1e-6 * d
        diff = ((select.lowrank_matmul(*hi) - select.lowrank_matmul(*lo)) * to_np(dY)).sum() / 2e-6
        size = np.sqrt((to_np(g) ** 2).sum())      # <g, d> has standard deviation |g|
        assert abs((to_np(g) * d).sum() - diff) < 1e-4 * size


# ------------------------------------------------------------------ streams, graphs, repeatability


def _all_ops(x, wg, wu, wd, idx, w, lr, dY, stream=None):
    X, W, A, B, ai, sc = lr
    l = x[:, :64]
    ri, rw = qg.mm_route_topk(l, 3, stream=stream)
    return [ri, rw, qg.mm_route_topk_grad(l, ri, rw, stream=stream),
            qg.mm_moe_layer(x, wg, wu, wd, idx, w, stream=stream),
            qg.mm_lowrank_matmul(X, W, A, B, ai, sc, stream=stream),
            *qg.mm_lowrank_matmul_grad(dY, X, W, A, B, ai, sc, stream=stream)]


@pytest.mark.parametrize("M", [8, 300])
def test_streams_graphs_and_repeats_give_the_same_bits(M):
    moe = _moe_inputs(20, 6, 2, 256, 320, 256, BF16, 141)
    *lr, dY = _lowrank_inputs(M, 1024, 520, 16, 4, BF16, 142)
    want = _all_ops(*moe, lr, dY)
    for _ in range(3):
        for a, b in zip(want, _all_ops(*moe, lr, dY)):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _all_ops(*moe, lr, dY)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _all_ops(*moe, lr, dY)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    moe[0].mul_(-0.5)                       # new values in the same buffers
    lr[0].mul_(-0.5)
    want = _all_ops(*moe, lr, dY)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_memory_of_a_call_on_another_stream_is_not_reused_early():
    """Outputs and workspaces belong to the current stream's pool; a call given another stream must keep them from it."""
    moe = _moe_inputs(20, 6, 2, 256, 320, 256, BF16, 161)
    *lr, dY = _lowrank_inputs(300, 1024, 520, 16, 4, BF16, 162)
    want = [t.clone() for t in _all_ops(*moe, lr, dY)]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                    # the calls' work waits here
        got = _all_ops(*moe, lr, dY, stream=side)
        # whatever the calls let go of is written over on the current stream
        junk = [torch.full((1 << n,), 0xFF, dtype=torch.uint8, device=DEV) for n in range(9, 27) for _ in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        del junk


def test_given_workspace_and_outputs():
    x, wg, wu, wd, idx, w = _moe_inputs(5, 4, 2, 128, 128, 128, BF16, 151)
    n = qg.mm_moe_layer_workspace_size(x, wg, wu, wd, idx)
    ws, out = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV), torch.empty((5, 128), dtype=BF16, device=DEV)
    assert qg.mm_moe_layer(x, wg, wu, wd, idx, w, workspace=ws, out=out) is out
    assert torch.equal(out, qg.mm_moe_layer(x, wg, wu, wd, idx, w))
    with pytest.raises(qg.MMError) as e:
        qg.mm_moe_layer(x, wg, wu, wd, idx, w, workspace=ws[:n - 1])
    assert e.value.name == "MM_ERR_WORKSPACE"
    X, W, A, B, ai, sc, dY = _lowrank_inputs(70, 128, 136, 8, 3, BF16, 152)
    for size, call in ((qg.mm_lowrank_matmul_workspace_size, lambda v: qg.mm_lowrank_matmul(X, W, A, B, ai, sc, workspace=v)),
                       (qg.mm_lowrank_matmul_grad_workspace_size,
                        lambda v: qg.mm_lowrank_matmul_grad(dY, X, W, A, B, ai, sc, workspace=v)[1])):
        n = size(X, W, A, B)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
        first = call(ws)
        assert torch.equal(first, call(ws)) and torch.equal(first, call(None))
        with pytest.raises(qg.MMError) as e:
            call(ws[:n - 1])
        assert e.value.name == "MM_ERR_WORKSPACE"
