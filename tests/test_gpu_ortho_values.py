"""The orthogonalised update over its range of values, against the formula in 64 bits.

How far a result may be off is worked out for each matrix, not limited from far away: half a step of its type at every value
(the output's rounding), plus what the stated roundings of operands, sums and state do to this matrix in an emulation on
the CPU (oracle.layer.orthogonalize_emulated).  The kernels' roundings are others of the same size, so twice the emulated
distance is allowed where the operands' 11 bits set it, and four times where the truncation of the tensor cores' sums does,
whose spare bits are not documented.  Each 32 x 32 box is held to the same with a factor of 3 more for what it
may stand out from the rest, so that a lost or misplaced box fails."""

import numpy as np
import pytest
import torch

import quantized_gemm_gb300 as qg
from helpers import rand_tensor, to_np
from oracle import layer

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


def _box_norms(x):
    p = np.pad(x * x, [(0, -n % 32) for n in x.shape])
    return np.sqrt(p.reshape(p.shape[0] // 32, 32, p.shape[1] // 32, 32).sum(axis=(1, 3)))


def check(got, X, coefficients, eps=1e-7, scale=1.0, form=None):
    """One matrix X (fp64 of the input's values) and its result; ``form``: of the products, where it is not the usual one."""
    form = form or ("single" if got.dtype == BF16 and min(X.shape) > 512 else "pairs")
    y, u = to_np(got), U[got.dtype]
    want = layer.orthogonalize(X, coefficients, eps, scale)
    off = np.linalg.norm(layer.orthogonalize_emulated(X, coefficients, eps, scale, form) - want)
    off = (2 if form == "single" else 4) * off + 8 * 2.0 ** -24 * np.linalg.norm(want)
    assert np.isfinite(y).all()
    err, bound = np.linalg.norm(y - want), np.linalg.norm(layer.half_steps(want, u)) + off
    assert err <= bound, "off by %g of the bound, %g of the result" % (err / bound, err / np.linalg.norm(want))
    share = np.sqrt(min(1.0, 1024 / want.size))
    over = _box_norms(y - want) / (_box_norms(layer.half_steps(want, u)) + 3 * off * share + 1e-300)
    worst = float(over.max())
    assert worst <= 1.0, "box %s is off by %g of its bound" % (np.unravel_index(over.argmax(), over.shape), worst)


def strong(shape, seed):
    """A few directions far above the rest: the iteration magnifies what is small, and rounding of the state with it."""
    g = torch.Generator().manual_seed(seed)
    X = 0.02 * torch.randn(shape, generator=g)
    for i in range(6):
        X += 0.5 ** i * torch.randn(shape[:-1] + (1,), generator=g) @ torch.randn(shape[:-2] + (1,) + shape[-1:], generator=g)
    return X


# ------------------------------------------------------------------ norms far below eps


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(520, 777), (600, 514), (40, 64), (200, 330)])
def test_matrices_of_a_stack_whose_norms_are_far_apart(shape, dtype):
    """Expert gradients that have died away: X / (norm + eps) is then far below 1, beside others that are 1."""
    sizes = [1.0, 1e-7, 1e-13, 1e-14, 1e-15, 1e-16, 1e-20]
    X = rand_tensor((len(sizes),) + shape, F32, 5, "cpu").double()
    X = (X / X.pow(2).sum(dim=(1, 2), keepdim=True).sqrt() * torch.tensor(sizes, dtype=torch.float64)[:, None, None]).to(dtype)
    got = qg.mm_orthogonalize(X.to(DEV))
    for x, y in zip(to_np(X), got):
        check(y, x, [MUON] * 5)


# ------------------------------------------------------------------ coefficients


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(520, 600), (200, 330), (40, 64)])
@pytest.mark.parametrize("steps,coefficients", [(3, (0.0, 1.0, 0.0)), (2, (0.0, 0.0, 1.0)), (5, (1e-3, 0.0, 0.0)),
                                                (4, (1e-4, 1e-5, 0.0)), (6, (0.02, 0.9, 0.0)), (2, (0.0, 0.0, 0.0))])
def test_coefficients_that_shrink(shape, dtype, steps, coefficients):
    """Singular values that end far below their bound, without a term a X to carry them or with a small one: the chain
    of MatMul's products, in fp32."""
    X = rand_tensor(shape, dtype, 21, DEV)
    Y = qg.mm_orthogonalize(X, steps, coefficients)
    fp32 = qg.mm_last_path() == qg.MM_PATH_TENSOR and coefficients[0] < 0.01 and any(coefficients)
    check(Y, to_np(X), [coefficients] * steps, form="matmul" if fp32 else None)


# ------------------------------------------------------------------ infinities


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(2, 520, 600), (2, 200, 330), (2, 40, 64)])
@pytest.mark.parametrize("steps", [0, 1, 3])
def test_an_infinity_makes_its_matrix_nan(shape, dtype, steps):
    X = rand_tensor(shape, dtype, 23, DEV)
    want = qg.mm_orthogonalize(X, steps)
    X[1, 3, 5] = float("inf")
    X[1, 7, 9] = float("-inf")
    Y = qg.mm_orthogonalize(X, steps)
    assert Y[1].isnan().all() and torch.equal(Y[0], want[0])


# ------------------------------------------------------------------ several steps


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("steps", [2, 5])
@pytest.mark.parametrize("shape", [(513, 513), (520, 777), (1030, 523), (640, 900), (300, 520), (520, 264), (129, 1300), (61, 100), (100, 61),
                                   (64, 64), (128, 256), (1000, 33)])
def test_errors_are_those_of_the_stated_roundings(shape, steps, dtype):
    """Row counts that end inside tiles of 128 and 256 rows, one launch and the chain of products, wide and tall."""
    X = rand_tensor(shape, dtype, 25, DEV)
    check(qg.mm_orthogonalize(X, steps, scale=1.5), to_np(X), [MUON] * steps, scale=1.5)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(520, 777), (900, 513), (192, 320), (300, 140), (64, 200)])
def test_strong_directions(shape, dtype):
    """A state that lost its lower bits would show here first (4e-2 for one of 11 bits)."""
    X = strong(shape, 4).to(dtype).to(DEV)
    check(qg.mm_orthogonalize(X), to_np(X), [MUON] * 5)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(3, 640, 520), (2, 300, 264), (3, 2, 130, 200)])
def test_stacks_of_unlike_matrices(shape, dtype):
    """Random, strong and small matrices side by side: each is held to its own bound."""
    X = rand_tensor(shape, F32, 27, "cpu").reshape((-1,) + shape[-2:])
    X[0] = strong(shape[-2:], 5)
    X[1] *= 2.0 ** -10
    X = X.reshape(shape).to(dtype).to(DEV)
    Y = qg.mm_orthogonalize(X, 3)
    for x, y in zip(to_np(X).reshape((-1,) + shape[-2:]), Y.reshape((-1,) + shape[-2:])):
        check(y, x, [MUON] * 3)


STEEP = (8.287 / 1.01, -23.596 / 1.01 ** 3, 17.300 / 1.01 ** 5)
THEN = (4.107 / 1.01, -2.948 / 1.01 ** 3, 0.545 / 1.01 ** 5)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(520, 777), (300, 520), (60, 200)])
def test_coefficients_that_change_from_step_to_step(shape, dtype):
    """A schedule that is steep just above 1; its bound leaves the f16 operands' range with five steps, not with two."""
    for steps in (2, 5):
        coefficients = [STEEP] + [THEN] * (steps - 1)
        X = rand_tensor(shape, dtype, 26, DEV)
        Y = qg.mm_orthogonalize(X, steps, coefficients)
        fp32 = steps == 5 and qg.mm_last_path() == qg.MM_PATH_TENSOR
        check(Y, to_np(X), coefficients, form="matmul" if fp32 else None)
