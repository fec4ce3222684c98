"""8-bit products, the router's balance loss and the orthogonalised update against the float64 oracle.

Tolerances are the oracle's bounds: a unit roundoff of the tensors' type for each rounding that an operator states, plus
fp32 sums taken at their worst."""

import numpy as np
import pytest
import torch

import quantized_gemm_gb300 as qg
from helpers import rand_tensor, to_np
from oracle import layer, select

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
MUON = (3.4445, -4.7750, 2.0315)


@pytest.fixture(autouse=True)
def clean_status():
    qg.mm_get_device_status()
    yield
    assert qg.mm_get_device_status() == "MM_OK"


@pytest.fixture(params=["auto", "simt", "tensor"])
def path(request):
    which = {"auto": qg.MM_PATH_AUTO, "simt": qg.MM_PATH_SIMT, "tensor": qg.MM_PATH_TENSOR}[request.param]
    qg.mm_set_path_policy(which)
    yield which
    qg.mm_set_path_policy(qg.MM_PATH_AUTO)


def assert_within(got, want, bound, what=""):
    got = to_np(got)
    assert np.isfinite(got).all(), what
    worst = np.max(np.abs(got - want) / bound) if got.size else 0.0
    assert worst <= 1.0, "%s: %g of the bound" % (what, worst)


# ------------------------------------------------------------------ quantisation of rows


def _check_quantize(x):
    q, s = qg.mm_quantize_rows(x)
    assert q.dtype == torch.int8 and s.dtype == F32
    wq, ws = layer.quantize_rows(to_np(x))
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    np.testing.assert_array_equal(q.cpu().numpy(), wq)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (3, 7), (5, 64), (130, 1000), (9, 1024), (7, 1032), (4, 4104), (3, 16384),
                                 (2, 16392), (2, 40000), (33, 129), (2, 0)])
def test_quantize_rows(M, K, dtype):
    x = rand_tensor((M, K), F32, M + K, "cpu") * torch.exp(3 * rand_tensor((M, 1), F32, K, "cpu"))
    _check_quantize(x.to(dtype).to(DEV))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_ties_and_near_ties(dtype):
    """Rows whose scale is a power of two, so that quotients end in exactly one half, and their neighbours."""
    base = torch.arange(-127, 128, dtype=F32)
    x = torch.cat([base, base + 0.5, base.clamp(-126, 126) + 0.5, base * (1 + 2.0 ** -11)]).clamp(-127, 127)
    x = torch.cat([x, torch.zeros((-x.numel()) % 8)])
    _check_quantize((x[None, :] * torch.tensor([[1.0], [2.0 ** -7], [2.0 ** 5]])).to(dtype).to(DEV))


def test_quantize_special_rows():
    rows = [[0.0] * 8, [-0.0] * 8, [float("inf")] + [1.0] * 7, [float("nan")] * 8, [1.0] * 7 + [float("-inf")],
            [2.0 ** -149] * 8, [2.0 ** -149 * k for k in (1, 64, 127, 128, 190, 191, 254, 300)], [2.0 ** -126] * 7 + [1e-40],
            [3.4e38, -3.4e38, 1e38, 1.0, 0, 0, 0, 0], [2.0 ** 120] * 8, [127 * 2.0 ** -126, 63.5 * 2.0 ** -126] + [0.0] * 6]
    _check_quantize(torch.tensor(rows, dtype=torch.float64).to(F32).to(DEV))
    half = torch.tensor([[65504.0, 1, -2, 6e-8, 0, 0, 0, 0], [6e-8] * 8, [float("nan")] + [0.0] * 7, [float("-inf")] * 8], dtype=F32)
    _check_quantize(half.to(F16).to(DEV))
    _check_quantize(half.to(BF16).to(DEV))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_strided_views(dtype):
    base = rand_tensor((200, 328), dtype, 3, DEV)
    for x in (base[::3], base[:, 1:], base[:, ::2], base.t(), base.t()[1:, 3:], base[4:5].expand(6, 328), base[:, :0], base[:0],
              base[:, 7:8], base.t()[:33]):
        _check_quantize(x)


# ------------------------------------------------------------------ 8-bit product


def _int8_inputs(M, K, N, dtype, seed, bias=True, full=False):
    rng = np.random.default_rng(seed)
    A = rng.integers(-128, 128, (M, K)).astype(np.int8)
    B = rng.integers(-128, 128, (N, K)).astype(np.int8)
    if full:                     # one sign, every sum at its largest
        A[:], B[:] = 127, 127
        A[::2] = -128
    sa, sb = rng.uniform(0.003, 0.02, M).astype(np.float32), rng.uniform(0.001, 0.01, N).astype(np.float32)
    b = rand_tensor((N,), dtype, seed + 1, DEV) if bias else None
    return [torch.from_numpy(v).to(DEV) for v in (A, B, sa, sb)] + [b]


def _check_int8(A, B, sa, sb, bias, dtype, **kw):
    Y = qg.mm_int8_matmul(A, B, sa, sb, bias, dtype=dtype, **kw)
    assert Y.dtype == dtype and Y.shape == (A.shape[0], B.shape[1])
    args = [to_np(t).astype(np.float64) if t is not None and t.is_floating_point() else None if t is None else to_np(t)
            for t in (A, B, sa, sb, bias)]
    want, bound = layer.int8_matmul(*args), layer.int8_matmul_bound(*args, u=U[dtype])
    # What is more than half a step above the type's largest number is infinite (65504 and 65520 for f16).
    top = torch.finfo(dtype).max * (1 + U[dtype] / 2)
    past, fits, got = np.abs(want) - bound > top, np.abs(want) + bound < top, to_np(Y)
    assert (got[past] == np.sign(want[past]) * np.inf).all()
    assert_within(torch.from_numpy(got[fits]), want[fits], bound[fits], "int8")
    return Y


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,K,N", [(1, 16, 1), (1, 4096, 300), (2, 512, 129), (3, 48, 1000), (5, 1040, 77), (8, 2048, 515), (9, 2048, 515),
                                   (16, 256, 256), (17, 1000, 333), (61, 1024, 1001), (64, 96, 4096), (100, 515, 264), (129, 2048, 250),
                                   (200, 333, 1), (257, 64, 513), (1, 7, 5), (300, 1, 40), (384, 1280, 640)])
@pytest.mark.parametrize("nk", [0, 1])
def test_int8(M, K, N, nk, dtype, path):
    A, B, sa, sb, bias = _int8_inputs(M, K, N, dtype, M * 7 + K + N, bias=(M + N) % 2 == 0)
    _check_int8(A, B.t() if nk else B.t().contiguous(), sa, sb, bias, dtype)


@pytest.mark.parametrize("M", [1, 4, 40, 200, 520])
def test_int8_sums_at_their_largest(M, path):
    for K in (1024, 9000):
        _check_int8(*(lambda A, B, *r: (A, B.t(), *r))(*_int8_inputs(M, K, 264, F32, 5, bias=False, full=True)), F32)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("K", [1, 6, 127, 1023, 1024, 1029, 4099])
@pytest.mark.parametrize("N", [1, 3, 130, 1157])
def test_int8_a_few_rows_at_any_address(M, K, N):
    """Weights as [N, K] and as [K, N], rows of every alignment."""
    rng = np.random.default_rng(M * K + N)
    for skip in range(4):
        A = torch.from_numpy(rng.integers(-128, 128, (M, K + 7)).astype(np.int8)).to(DEV)[:, skip:skip + K]
        kn = torch.from_numpy(rng.integers(-128, 128, (K, N + 9)).astype(np.int8)).to(DEV)[:, skip:skip + N]
        nk = torch.from_numpy(rng.integers(-128, 128, (N, K + 5)).astype(np.int8)).to(DEV)[:, skip:skip + K]
        sa, sb = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
        dtype = (BF16, F16, F32)[skip % 3]
        bias = rand_tensor((N,), dtype, skip, DEV)
        for B in (kn, nk.t(), kn.contiguous(), nk.contiguous().t()):
            _check_int8(A, B, sa, sb, bias if skip & 1 else None, dtype)
            assert M > 4 or qg.mm_last_path() == qg.MM_PATH_VECTOR


@pytest.mark.parametrize("K", [(1 << 17) - 1, 1 << 17])
def test_int8_longest_sums_of_a_few_rows_of_kn_weights(K):
    A = torch.full((2, K), -128, dtype=torch.int8, device=DEV)
    Y = qg.mm_int8_matmul(A, torch.full((K, 8), -128, dtype=torch.int8, device=DEV), torch.ones(2, device=DEV),
                          torch.ones(8, device=DEV), dtype=F32)
    few = qg.mm_last_path() == qg.MM_PATH_VECTOR
    assert few == (K < 1 << 17)
    assert float((Y.double() / (2.0 ** 14 * K) - 1).abs().max()) <= (2.0 ** -23 if few else (K / 16 + 1) * 2.0 ** -23)


@pytest.mark.parametrize("K", [8191 * 512, 8191 * 512 + 16, 8192 * 512 - 16, 8192 * 512])
def test_int8_longest_sums_of_a_few_rows(K):
    """Every product 2^14: the integer sums of the few-row form just fit, then other forms take over."""
    A = torch.full((1, K), -128, dtype=torch.int8, device=DEV)
    one = torch.ones(2, device=DEV)
    Y = qg.mm_int8_matmul(A, A.expand(2, K).contiguous().t(), one[:1], one, dtype=F32)
    # exact lanes and 31 fp32 additions, or the fp32 additions of the tensor cores
    few = qg.mm_last_path() == qg.MM_PATH_VECTOR
    assert few == (K <= 8191 * 512)
    assert float((Y.double() / (2.0 ** 14 * K) - 1).abs().max()) <= (37 * 2.0 ** -24 if few else (K / 16 + 1) * 2.0 ** -23)


def test_int8_strided_views(path):
    A, B, sa, sb, bias = _int8_inputs(90, 300, 400, F32, 11)
    for a in (A, A[::2], A[:, 5:], A[:, ::3], A.t().contiguous().t(), A[3:4].expand(20, 300), A[:1], A[5:7, 1:]):
        for b in (B.t(), B[:, 3:].t(), B[::2].t(), B.t().contiguous(), B.t().contiguous()[:, 1:], B[:, ::2].t(), B[2:3].expand(50, 300).t()):
            k = min(a.shape[1], b.shape[0])
            a2, b2 = a[:, :k], b[:k]
            _check_int8(a2, b2, sa[:a2.shape[0]], sb[:b2.shape[1]], bias[:b2.shape[1]], F32)
    _check_int8(A[:45], B[:200].t(), sa[::2], sb[::2], bias[1::2], F32)


def test_int8_columns_that_overlap(path):
    """Weights whose columns lie 16 bytes apart and are 64 long: windows over one array."""
    A, B, sa, sb, bias = _int8_inputs(300, 64, 264, BF16, 12)
    windows = B.reshape(-1).as_strided((64, 264), (1, 16))
    for M in (5, 40, 300):
        _check_int8(A[:M], windows, sa[:M], sb, bias, BF16)


def test_int8_rows_depend_on_themselves_alone(path):
    """A row of NaN scale (quantised from an infinity) is NaN, and the others are what they were."""
    A, B, sa, sb, bias = _int8_inputs(70, 256, 264, BF16, 21)
    for M in (3, 70):
        want = qg.mm_int8_matmul(A[:M], B.t(), sa[:M], sb, bias)
        s = sa[:M].clone()
        s[1] = float("nan")
        got = qg.mm_int8_matmul(A[:M], B.t(), s, sb, bias)
        assert got[1].isnan().all()
        keep = [m for m in range(M) if m != 1]
        assert torch.equal(got[keep], want[keep])


def test_int8_scales_far_apart(path):
    """Scales whose product leaves fp32's range are applied one after the other."""
    A, B, sa, sb, _ = _int8_inputs(40, 512, 264, F32, 22)
    for fa, fb in ((1e-25, 1e25), (1e30, 1e-30), (1e-30, 1e30)):
        _check_int8(A, B.t(), sa * fa, sb * fb, None, F32)


def test_int8_empty(path):
    A, B = torch.zeros((0, 16), dtype=torch.int8, device=DEV), torch.zeros((8, 16), dtype=torch.int8, device=DEV)
    s = torch.ones(8, device=DEV)
    assert qg.mm_int8_matmul(A, B.t(), s[:0], s).shape == (0, 8)
    assert qg.mm_int8_matmul(B, A.t(), s, s[:0]).shape == (8, 0)
    if path != qg.MM_PATH_TENSOR:
        bias = rand_tensor((8,), F32, 1, DEV)
        y = qg.mm_int8_matmul(A.t()[:8, :0], B.t()[:0], s, s, bias, dtype=F32)
        assert torch.equal(y, bias.expand(8, 8))


def test_int8_after_quantisation_is_close_to_the_product():
    x, w = rand_tensor((33, 1024), BF16, 31, DEV), rand_tensor((1024, 520), BF16, 32, DEV)
    q, s = qg.mm_quantize_rows(x)
    wq, ws = qg.mm_quantize_rows(w.t())
    y = _check_int8(q, wq.t(), s, ws, None, BF16)
    want = to_np(x) @ to_np(w)
    # each factor is off by at most half a step, s / 2: |dy| <= sum (s_x/2 |w| + s_w/2 |x|) + s_x s_w / 4 a term
    ax, aw = np.abs(to_np(x)), np.abs(to_np(w))
    sx, sw = to_np(s)[:, None], to_np(ws)[None, :]
    bound = sx / 2 * aw.sum(axis=0) + ax.sum(axis=1, keepdims=True) * sw / 2 + 1024 * sx * sw / 4 + U[BF16] * np.abs(want)
    assert (np.abs(to_np(y) - want) <= 1.02 * bound).all()


# ------------------------------------------------------------------ balance loss


def _balance_inputs(T, G, k, dtype, seed, masked):
    rng = np.random.default_rng(seed)
    l = rand_tensor((T, G), F32, seed, "cpu") * 2
    idx = np.argsort(rng.random((T, G)), axis=1)[:, :k].astype(np.int32)
    if masked and T:
        l[torch.from_numpy(rng.random((T, G)) < 0.3)] = float("-inf")
        l[torch.from_numpy(rng.random((T, G)) < 0.02)] = float("nan")
        l[T // 2] = float("-inf")
        l[0, G // 2] = float("inf")
        idx[rng.random((T, k)) < 0.2] = -1
        idx[T // 2] = -1
    return l.to(dtype).to(DEV), torch.from_numpy(idx).to(DEV)


def _check_balance(l, idx, base_seed=9):
    T, G = l.shape
    loss, counts, mean = qg.mm_route_balance(l, idx)
    wl, wc, wm = layer.route_balance(to_np(l), to_np(idx))
    np.testing.assert_array_equal(counts.cpu().numpy(), wc)
    # exp: 2 ulp and |l - max| 2^-23 (times p, at most 2^-23 in all), its sum G terms, a quotient; then T terms
    rel = (G + T + 40) * 2.0 ** -24 + 2.0 ** -21
    assert_within(mean, wm, rel * wm + T * 2.0 ** -23 / max(1, wc[G]) + 1e-30, "mean")
    assert_within(loss, np.array([wl]), (rel + G * 2.0 ** -23) * abs(wl) + 2.0 ** -22 * G + 1e-30, "loss")
    d = torch.tensor([0.37 * max(1, T)], device=DEV)
    for base in (None, rand_tensor((T, G), l.dtype, base_seed, DEV)):
        got = qg.mm_route_balance_grad(l, counts, d, base=base)
        assert got.dtype == l.dtype
        want = layer.route_balance_grad(to_np(l), wc, to_np(d)[0], None if base is None else to_np(base))
        p = np.stack([select._softmax_row(r)[0] for r in to_np(l)]) if T else np.zeros((0, G))
        share = wc[:G] / max(1, wc[:G].sum())
        mag = to_np(d)[0] * G / max(1, wc[G]) * p * (share + (p @ share)[:, None])
        assert_within(got, want, U[l.dtype] * np.abs(want) + ((2 * G + 60) * 2.0 ** -24 + 2.0 ** -21) * mag +
                      to_np(d)[0] * G / max(1, wc[G]) * 2.0 ** -40 + 2.0 ** -25 * (l.dtype == F16) + 1e-30, "gradient")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,G,k", [(1, 1, 1), (1, 64, 2), (3, 5, 5), (37, 64, 8), (5, 65, 3), (16, 100, 16), (257, 256, 8), (4, 300, 32),
                                   (3, 1000, 7), (2, 1024, 32), (1000, 8, 2), (7, 40, 40), (1200, 24, 2)])
@pytest.mark.parametrize("masked", [0, 1])
def test_balance(T, G, k, dtype, masked):
    _check_balance(*_balance_inputs(T, G, k, dtype, T + G, masked))


def test_balance_many_rows():
    """More rows than one round of blocks takes: counts to the last, column sums against fp64."""
    for T, G, k, dtype in ((70001, 64, 2, BF16), (50000, 160, 8, F16), (40003, 33, 3, F32)):
        l, idx = _balance_inputs(T, G, k, dtype, G, masked=1)
        loss, counts, mean = qg.mm_route_balance(l, idx)
        d = torch.where(l.isnan(), float("-inf"), l.double())
        p = torch.softmax(torch.where(d.isinf() & (d > 0), 1e300, d), dim=1)
        p = torch.where(d.amax(dim=1, keepdim=True) > float("-inf"), p, 0.0)
        alive = int((d.amax(dim=1) > float("-inf")).sum())
        want = torch.bincount(idx[idx >= 0].long(), minlength=G)
        assert counts[:G].tolist() == want.tolist() and int(counts[G]) == alive
        wm = p.sum(dim=0) / alive
        # each block adds T / (3 SMs) terms, then the blocks' sums: far fewer than 4000 roundings of 2^-24
        assert_within(mean, wm.cpu().numpy(), (4000 * 2.0 ** -24 + 2.0 ** -21) * wm.cpu().numpy() + 2.0 ** -23)
        share = want.double() / want.sum()
        assert abs(float(loss) - float(G * (share * wm).sum())) < 1e-3
        g = qg.mm_route_balance_grad(l, counts, torch.full((1,), float(T), device=DEV))
        wg = T * G / alive * p * (share - (p * share).sum(dim=1, keepdim=True))
        mag = (T * G / alive * p * (share + (p * share).sum(dim=1, keepdim=True))).cpu().numpy()
        assert_within(g, wg.cpu().numpy(), U[dtype] * np.abs(wg.cpu().numpy()) + (G + 60) * 2.0 ** -23 * mag + 1e-7)


def test_balance_strided_views_and_int64():
    base = rand_tensor((40, 90), F32, 8, DEV)
    ids = torch.randint(-1, 30, (40, 9), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    for l in (base[::2, 3:70], base.t()[:36, 1:32], base[1:2].expand(6, 90), base[:, 4:68]):
        for i in (ids[:l.shape[0], :3], ids.int()[:l.shape[0], ::4], ids[:l.shape[0]]):
            _check_balance(l, i)


def test_balance_nothing_to_count():
    l = torch.full((5, 12), float("-inf"), device=DEV)
    idx = torch.full((5, 2), -1, dtype=torch.int32, device=DEV)
    _check_balance(l, idx)
    _check_balance(torch.zeros((5, 12), device=DEV), idx)
    _check_balance(torch.zeros((0, 12), device=DEV), idx[:0])


def test_balance_records_an_index_out_of_range():
    l = rand_tensor((3, 8), F32, 4, DEV)
    idx = torch.tensor([[1, 8], [-2, -1], [7, 1 << 30]], dtype=torch.int32, device=DEV)
    _, counts, _ = qg.mm_route_balance(l, idx)
    assert qg.mm_get_device_status() == "MM_ERR_INDEX_RANGE"
    assert counts.tolist() == [0, 1, 0, 0, 0, 0, 0, 1, 3]


def test_balance_results_repeat():
    l, idx = _balance_inputs(30000, 96, 4, BF16, 3, 0)
    first = qg.mm_route_balance(l, idx)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, qg.mm_route_balance(l, idx)))


# ------------------------------------------------------------------ orthogonalised update


def _operand(X):
    """The products' operands: two f16 values, or one for larger bf16 matrices."""
    return 2.0 ** -11 if X.dtype == BF16 and min(X.shape[-2:]) > 512 else 3 * 2.0 ** -22


def _check_ortho(X, steps=5, coefficients=MUON, eps=1e-7, scale=1.0):
    Y = qg.mm_orthogonalize(X, steps, coefficients, eps, scale)
    assert Y.shape == X.shape and Y.dtype == X.dtype
    per = [coefficients] * steps if steps and not isinstance(coefficients[0], tuple) else list(coefficients)[:steps]
    x = to_np(X).reshape((-1,) + X.shape[-2:])
    y = to_np(Y).reshape((-1,) + X.shape[-2:])
    assert np.isfinite(y).all()
    for a, b in zip(x, y):
        want = layer.orthogonalize(a, per, eps, scale)
        bound = layer.orthogonalize_bound(a, per, eps, scale, _operand(X), U[X.dtype])
        off = np.linalg.norm(b - want)
        assert off <= bound, "%g of the bound" % (off / bound)
    return Y


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (9, 1), (2, 2), (3, 40), (40, 3), (16, 16), (61, 100), (64, 64), (100, 61), (130, 136),
                                   (65, 300), (300, 65), (96, 1000), (256, 256), (200, 520), (520, 264)])
def test_orthogonalize(shape, dtype):
    _check_ortho(rand_tensor(shape, dtype, sum(shape), DEV))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(2, 2), (16, 16), (61, 100), (100, 61), (64, 64), (65, 300), (300, 65), (130, 136), (256, 256), (257, 600),
                                   (385, 129), (520, 264), (3, 20, 33), (5, 130, 64), (3, 136, 264), (2, 300, 1100), (513, 513),
                                   (520, 777), (1030, 523), (2, 516, 600)])
def test_orthogonalize_on_the_tensor_cores(shape, dtype):
    """The chain of products for sizes that a cluster would take; tiles that end inside, and on both sides of the diagonal."""
    qg.mm_set_path_policy(qg.MM_PATH_TENSOR)
    try:
        _check_ortho(rand_tensor(shape, dtype, sum(shape) + 1, DEV), scale=1.5)
        assert qg.mm_last_path() == qg.MM_PATH_TENSOR
        _check_ortho(rand_tensor(shape, dtype, sum(shape) + 2, DEV), steps=1)
    finally:
        qg.mm_set_path_policy(qg.MM_PATH_AUTO)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(300, 520), (2, 260, 200), (129, 1300)])
def test_orthogonalize_on_the_cuda_cores(shape, dtype):
    """The chain in fp32: larger than a cluster's shared memory, and coefficients that leave the f16 operands' range."""
    X = rand_tensor(shape, dtype, 9, DEV)
    qg.mm_set_path_policy(qg.MM_PATH_SIMT)
    try:
        _check_ortho(X)
        assert qg.mm_last_path() == qg.MM_PATH_SIMT
    finally:
        qg.mm_set_path_policy(qg.MM_PATH_AUTO)
    _check_ortho(X, 5, (40.0, 0.0, 0.0))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(8, 16), (31, 31), (32, 5000), (33, 1000), (1000, 33), (64, 4000), (65, 999), (128, 1024), (1024, 127),
                                   (90, 11, 7), (200, 40, 64), (30, 128, 130)])
def test_orthogonalize_in_a_cluster(shape, dtype):
    """Slabs of every size, stacks with fewer CTAs a matrix."""
    _check_ortho(rand_tensor(shape, dtype, sum(shape) + 3, DEV), scale=0.3)
    assert qg.mm_last_path() == qg.MM_PATH_SIMT


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(3, 20, 33), (2, 2, 70, 30), (5, 130, 64), (1, 1, 8), (40, 17, 17), (3, 136, 264)])
def test_orthogonalize_stacks(shape, dtype):
    X = rand_tensor(shape, dtype, sum(shape), DEV)
    _check_ortho(X, scale=0.7)
    # alone, a matrix may take other kernels (the choice goes by the work of the stack): the same bound, not the same bits
    _check_ortho(X.reshape((-1,) + shape[-2:])[:1], scale=0.7)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalize_strided_views(dtype):
    base = rand_tensor((4, 90, 120), dtype, 5, DEV)
    for x in (base[0, ::2, 3:], base[:, :, ::2], base.transpose(1, 2), base.permute(1, 2, 0)[:3], base[1, :1].expand(8, 120),
              base[0].expand(2, 90, 120), base[::2, 1:, 1:]):
        _check_ortho(x, steps=3)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalize_other_coefficients(dtype):
    X = rand_tensor((48, 80), dtype, 6, DEV)
    _check_ortho(X, 3, [(1.5, -0.5, 0.0), (1.875, -1.25, 0.375), MUON], eps=0.5, scale=-2.0)
    _check_ortho(X, 0)
    _check_ortho(X, 1, (0.0, 0.0, 0.0))
    _check_ortho(X, 2, (10.0, -20.0, 15.0))
    _check_ortho(X, 8, (1.5, -0.5, 0.0))
    L = rand_tensor((300, 520), dtype, 10, DEV)          # the chain of products
    for coefficients, steps in (((0.0, 0.0, 0.0), 2), ((2.0, 0.0, 0.0), 2), ((0.0, 1.0, 0.0), 1), ((1.5, -0.5, 0.0), 6), (MUON, 0)):
        _check_ortho(L, steps, coefficients, scale=-0.5)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalize_more_matrices_than_a_grid_axis_holds(dtype):
    X = rand_tensor((66000, 40, 48), dtype, 13, DEV)
    for which in (qg.MM_PATH_AUTO, qg.MM_PATH_SIMT, qg.MM_PATH_TENSOR):
        qg.mm_set_path_policy(which)
        try:
            Y = qg.mm_orthogonalize(X)
        finally:
            qg.mm_set_path_policy(qg.MM_PATH_AUTO)
        for i in (0, 65535, 65536, 65999):
            want = layer.orthogonalize(to_np(X[i]), [MUON] * 5, 1e-7)
            bound = layer.orthogonalize_bound(to_np(X[i]), [MUON] * 5, 1e-7, 1.0, _operand(X), U[dtype])
            assert np.linalg.norm(to_np(Y[i]) - want) <= bound


def test_orthogonalize_many_tiny_matrices():
    X = rand_tensor((3000, 6, 7), BF16, 12, DEV)
    Y = qg.mm_orthogonalize(X)
    assert qg.mm_last_path() == qg.MM_PATH_SIMT
    pick = [0, 1, 1499, 2999]
    for i in pick:
        want = layer.orthogonalize(to_np(X[i]), [MUON] * 5, 1e-7)
        bound = layer.orthogonalize_bound(to_np(X[i]), [MUON] * 5, 1e-7, 1.0, U[F32], U[BF16])
        assert np.linalg.norm(to_np(Y[i]) - want) <= bound


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalize_range_of_values(dtype):
    """The norm's squares leave fp32's range on both sides.  (The bits may differ between exponents: values below
    2^-126 lose digits when they are stored, and squares on both sides of the ranges' borders are added apart.)"""
    X = rand_tensor((40, 64), dtype, 7, DEV)
    for e in (-120, -70, -40, 40, 70, 118):
        _check_ortho((X.double() * 2.0 ** e).to(dtype), eps=0.0)
    tiny = (X.double() * 2.0 ** -146).to(dtype)
    if dtype == BF16:       # |x| < 2^-143 < 2^-134, half of bf16's least value: all zeros, 0 / 0
        assert qg.mm_orthogonalize(tiny, eps=0.0).isnan().all()
    else:                   # subnormal
        _check_ortho(tiny, eps=0.0)
    mixed = X.clone()
    mixed[0, 0] = 2.0 ** 100
    _check_ortho(mixed)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_orthogonalize_zeros_and_nan(dtype):
    X = rand_tensor((4, 70, 80), dtype, 8, DEV)
    want = qg.mm_orthogonalize(X)
    Z = X.clone()
    Z[0] = 0
    Z[2, 3, 4] = float("nan")
    Z[3, 1, 1] = float("inf")
    got = qg.mm_orthogonalize(Z)
    assert (got[0] == 0).all() and torch.equal(got[1], want[1])
    assert got[2].isnan().all() and got[3].isnan().all()
    assert qg.mm_orthogonalize(Z[:1], eps=0.0).isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalize_strong_directions(dtype):
    """A few directions far above the rest: the iteration magnifies what is small, and rounding of the state with it."""
    g = torch.Generator().manual_seed(4)
    X = 0.02 * torch.randn((192, 320), generator=g)
    for i in range(6):
        X += 0.5 ** i * torch.randn((192, 1), generator=g) @ torch.randn((1, 320), generator=g)
    _check_ortho(X.to(dtype).to(DEV))


def test_orthogonalize_results_repeat():
    for shape, dtype in (((300, 520), BF16), ((2, 700, 300), F32), ((60, 60), F32)):
        X = rand_tensor(shape, dtype, 3, DEV)
        first = qg.mm_orthogonalize(X)
        for _ in range(3):
            assert torch.equal(qg.mm_orthogonalize(X), first)


# ------------------------------------------------------------------ streams, graphs, workspaces


def _all_ops(stream=None):
    """Every entry point on both sides of its choices; the inputs are remade the same."""
    out = []
    for M in (3, 40, 300):
        A, B, sa, sb, bias = _int8_inputs(M, 512, 264, BF16, M)
        out += [lambda A=A, B=B, sa=sa, sb=sb, bias=bias: qg.mm_int8_matmul(A, B.t(), sa, sb, bias, stream=stream)]
    x = rand_tensor((70, 1000), BF16, 61, DEV)
    out += [lambda: qg.mm_quantize_rows(x, stream=stream), lambda: qg.mm_quantize_rows(x.t(), stream=stream)]
    l, idx = _balance_inputs(500, 64, 2, BF16, 62, 1)
    d = torch.ones(1, device=DEV)

    def balance():
        loss, counts, mean = qg.mm_route_balance(l, idx, stream=stream)
        return loss, counts, mean, qg.mm_route_balance_grad(l, counts, d, base=l, stream=stream)
    out += [balance]
    for shape, dtype in (((61, 200), F32), ((2, 300, 264), BF16), ((400, 260), F32)):
        X = rand_tensor(shape, dtype, 63, DEV)
        out += [lambda X=X: qg.mm_orthogonalize(X, stream=stream)]
    return out


def _flat(results):
    return [t for r in results for t in (r if isinstance(r, tuple) else (r,))]


def _same(a, b):
    return a.dtype == b.dtype and torch.equal(a.view(torch.uint8) if a.dim() else a, b.view(torch.uint8) if b.dim() else b)


def test_memory_of_a_call_on_another_stream_is_not_reused_early():
    want = [t.clone() for t in _flat([f() for f in _all_ops()])]
    side = torch.cuda.Stream()
    calls = _all_ops(stream=side)
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                    # the calls' work waits here
        got = _flat([f() for f in calls])
        junk = [torch.full((1 << n,), 0xFF, dtype=torch.uint8, device=DEV) for n in range(9, 25) for _ in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert _same(a, b)
        del junk


def test_graphs_replay_on_new_values():
    """Captured once the calls have run; replays follow the inputs' memory."""
    l, idx = _balance_inputs(3000, 64, 2, BF16, 71, 1)
    A, B, sa, sb, bias = _int8_inputs(200, 512, 264, BF16, 72)
    X = rand_tensor((2, 200, 300), BF16, 73, DEV)
    R = rand_tensor((40, 90), F32, 74, DEV)
    d = torch.ones(1, device=DEV)

    def step():
        loss, counts, mean = qg.mm_route_balance(l, idx)
        g = qg.mm_route_balance_grad(l, counts, d)
        q, s = qg.mm_quantize_rows(X[0])
        return loss, counts, mean, g, q, s, qg.mm_int8_matmul(A, B.t(), sa, sb, bias), qg.mm_int8_matmul(
            A[:5], B.t(), sa[:5], sb, bias), qg.mm_int8_matmul(A[:30], B.t(), sa[:30], sb), qg.mm_orthogonalize(
            X), qg.mm_orthogonalize(R)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (81, 82):
        l2, idx2 = _balance_inputs(3000, 64, 2, BF16, seed, 1)
        A2, B2, sa2, sb2, bias2 = _int8_inputs(200, 512, 264, BF16, seed)
        for a, b in ((l, l2), (idx, idx2), (A, A2), (B, B2), (sa, sa2), (sb, sb2), (bias, bias2),
                     (X, rand_tensor((2, 200, 300), BF16, seed, DEV)), (R, rand_tensor((40, 90), F32, seed, DEV))):
            a.copy_(b)
        graph.replay()
        for a, b in zip(step(), got):
            assert _same(a, b)


def test_given_workspaces_and_outputs():
    """A workspace full of garbage gives the same results, and one byte too few is refused."""
    assert qg.mm_orthogonalize_workspace_size(torch.empty((60, 80), device=DEV)) == 0
    l, idx = _balance_inputs(300, 40, 2, F32, 91, 0)
    A, B, sa, sb, _ = _int8_inputs(300, 512, 264, F32, 92)
    X = rand_tensor((300, 264), BF16, 93, DEV)
    R = rand_tensor((400, 264), F32, 94, DEV)
    for size, call in ((qg.mm_route_balance_workspace_size(l, idx), lambda w: qg.mm_route_balance(l, idx, workspace=w)),
                       (qg.mm_int8_matmul_workspace_size(A, B.t(), F32), lambda w: qg.mm_int8_matmul(A, B.t(), sa, sb, dtype=F32, workspace=w)),
                       (qg.mm_orthogonalize_workspace_size(X), lambda w: qg.mm_orthogonalize(X, workspace=w)),
                       (qg.mm_orthogonalize_workspace_size(R), lambda w: qg.mm_orthogonalize(R, workspace=w))):
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
        want, got = call(None), call(ws)
        assert all(_same(a, b) for a, b in zip(_flat([want]), _flat([got])))
        with pytest.raises(qg.MMError) as e:
            call(ws[:size - 1])
        assert e.value.name == "MM_ERR_WORKSPACE"
    out = torch.empty_like(X)
    assert qg.mm_orthogonalize(X, out=out) is out and torch.equal(out, qg.mm_orthogonalize(X))


# ------------------------------------------------------------------ offsets past 32 bits


def test_large_quantisation_and_product():
    """2.2e9 values in, 2.2e9 products out; the last rows against the oracle."""
    x = torch.zeros((17000, 131072), dtype=BF16, device=DEV)
    x[-3:] = rand_tensor((3, 131072), BF16, 5, DEV)
    q, s = qg.mm_quantize_rows(x)
    wq, ws = layer.quantize_rows(to_np(x[-3:]))
    np.testing.assert_array_equal(q[-3:].cpu().numpy(), wq)
    np.testing.assert_array_equal(s[-3:].cpu().numpy(), ws)
    assert not q[:-3].any()
    del x
    # the long array as weights of 17000 channels, and as tokens
    A, B = q[-300:, :64].contiguous(), q[:, :64]
    sa = torch.ones(300, device=DEV)
    for M in (3, 40, 300):
        Y = qg.mm_int8_matmul(A[-M:], B.t(), sa[-M:], s)
        want = A[-M:].double() @ B[-3:].double().t() * s[-3:].double()
        assert float((Y[:, -3:].double() - want).abs().max()) <= U[BF16] * 1.01 * float(want.abs().max()) + 1e-12
    C = torch.randint(-128, 128, (131072, 64), dtype=torch.int8, device=DEV)
    Y = qg.mm_int8_matmul(q[:, :64], C.t(), s, torch.ones(131072, device=DEV))
    want = q[-3:, :64].double() @ C.double().t() * s[-3:, None].double()
    assert float(((Y[-3:].double() - want).abs() - U[BF16] * 1.01 * want.abs()).max()) <= 1e-12
    assert not Y[:-3].any()


def test_large_balance():
    T, G = 2200000, 1024
    l = torch.zeros((T, G), dtype=BF16, device=DEV)
    l[-1] = rand_tensor((G,), BF16, 6, DEV)
    idx = (torch.arange(T, device=DEV, dtype=torch.int32) % G)[:, None].contiguous()
    loss, counts, mean = qg.mm_route_balance(l, idx)
    assert torch.equal(counts[:G].long(), torch.bincount(idx[:, 0].long(), minlength=G)) and int(counts[G]) == T
    # each block adds T / 304 equal terms in fp32 to a lane's sum, off by half an ulp each
    assert float((mean * G - 1).abs().max()) < T / 304 * 2.0 ** -24 + 1e-5 and abs(float(loss) - 1) < 1e-3
    g = qg.mm_route_balance_grad(l, counts, torch.full((1,), float(T), device=DEV), base=l)
    p, share = torch.softmax(l[-1].double(), 0), counts[:G].double() / T
    want = G * p * (share - (p * share).sum()) + l[-1].double()
    assert float((g[-1].double() - want).abs().max()) < U[BF16] * float(want.abs().max()) + 1e-3 * 2.0 ** -8


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_stack(dtype):
    X = torch.zeros((9000, 240, 1024), dtype=dtype, device=DEV)
    X[-1] = rand_tensor((240, 1024), dtype, 7, DEV)
    Y = qg.mm_orthogonalize(X)
    want = layer.orthogonalize(to_np(X[-1]), [MUON] * 5, 1e-7)
    bound = layer.orthogonalize_bound(to_np(X[-1]), [MUON] * 5, 1e-7, 1.0, _operand(X), U[dtype])
    assert np.linalg.norm(to_np(Y[-1]) - want) <= bound
    assert not Y[:-1].any()


# ------------------------------------------------------------------ together


def test_the_example_trains_and_serves():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, root)
    from examples import train_and_serve
    block = train_and_serve.ExpertLayer(hidden=128, ffn=136, experts=6, picks=2)
    x = rand_tensor((40, 128), F32, 111, DEV)
    logits, idx, weights = block.route(x)
    assert np.array_equal(to_np(idx), select.route_topk(to_np(logits), 2, 1)[0])
    dw = rand_tensor((40, 2), F32, 112, DEV) / 40
    loss, counts, dlogits = block.router_gradient(logits, idx, dw, balance=0.05)
    l64 = to_np(logits)
    want = select.route_topk_grad(l64, to_np(idx), to_np(dw)) + layer.route_balance_grad(l64, to_np(counts), 0.05)
    assert abs(float(loss) - layer.route_balance(l64, to_np(idx))[0]) < 1e-5
    assert_within(dlogits, want, 1e-5 * np.abs(want) + 1e-8, "router gradient")
    # against a difference of the two losses' sum
    def total(l):
        _, w = select.route_topk(l, 2, 1)
        return (w * to_np(dw)).sum() + 0.05 * layer.route_balance(l, to_np(idx))[0]
    for t, j in ((0, 1), (7, 3), (39, 5)):
        d = np.zeros_like(l64)
        d[t, j] = 1e-5
        assert abs((total(l64 + d) - total(l64 - d)) / 2e-5 - want[t, j]) < 1e-6
    before = block.experts.clone()
    block.update(x, dlogits, rand_tensor(block.experts.shape, BF16, 113, DEV), rate=0.02)
    assert not torch.equal(before, block.experts) and torch.isfinite(block.experts.float()).all()
    served = block.serve()
    y = served(x.to(BF16), 3)
    q, s = layer.quantize_rows(to_np(x.to(BF16)))
    wq, ws = layer.quantize_rows(to_np(block.experts[3]).T)
    want = layer.int8_matmul(q, wq.T, s.astype(np.float64), ws.astype(np.float64))
    assert_within(y, want, layer.int8_matmul_bound(q, wq.T, s.astype(np.float64), ws.astype(np.float64), u=U[BF16]), "served")
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "train_and_serve.py"), "--steps", "2"],
                       capture_output=True, text=True)
    assert r.returncode == 0 and "us a step" in r.stdout, r.stderr


def test_a_training_step_and_its_8_bit_layer():
    """Route, balance loss and gradients, the orthogonalised update of router and experts, then the experts in 8 bits."""
    T, K, G, F, k = 96, 128, 8, 136, 2
    x, router = rand_tensor((T, K), F32, 101, DEV), rand_tensor((K, G), F32, 102, DEV) * K ** -0.5
    w, dw_pick = rand_tensor((G, K, F), BF16, 103, DEV), rand_tensor((T, k), F32, 104, DEV) / T
    logits = qg.mm_matmul(x, router)
    idx, weights = qg.mm_route_topk(logits, k)
    loss, counts, mean = qg.mm_route_balance(logits, idx)
    assert int(counts[:G].sum()) == T * k and int(counts[G]) == T
    through = qg.mm_route_topk_grad(logits, idx, dw_pick)
    dl = qg.mm_route_balance_grad(logits, counts, torch.full((1,), 0.01, device=DEV), base=through)
    l64 = to_np(logits)
    want = select.route_topk_grad(l64, to_np(idx), to_np(dw_pick)) + layer.route_balance_grad(l64, to_np(counts), 0.01)
    assert_within(dl, want, 1e-5 * np.abs(want) + 1e-8, "dlogits")
    up = qg.mm_orthogonalize(qg.mm_matmul(x.t(), dl))
    assert up.shape == router.shape
    s = np.linalg.svd(to_np(up), compute_uv=False)
    assert s.max() < 1.3 and s.min() > 0.0
    ups = qg.mm_orthogonalize(rand_tensor((G, K, F), BF16, 105, DEV), scale=0.2)
    w = (w - ups).contiguous()
    q, sx = qg.mm_quantize_rows(x.to(BF16))
    for e in (0, G - 1):
        wq, sw = qg.mm_quantize_rows(w[e].t())
        _check_int8(q, wq.t(), sx, sw, None, BF16)
