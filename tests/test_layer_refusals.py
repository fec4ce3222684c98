"""What the 8-bit, balance-loss and orthogonalising entry points refuse (no GPU: every call fails validation first)."""

import ctypes
import math

import pytest
import torch

import quantized_gemm_gb300 as qg
from quantized_gemm_gb300 import build as qbuild
from test_abi import T

BF16, F16, F32, F64, I32, I64, I8, U8 = 0, 1, 2, 3, 4, 5, 8, 9
INVALID, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qg._lib()


def ref(t):
    return None if t is None else ctypes.byref(t)


@pytest.mark.parametrize("change,want", [
    ({"x": T((4, 8), dtype=F64)}, DTYPE), ({"x": T((4, 8), dtype=I8)}, DTYPE), ({"x": T((4, 8, 1))}, SHAPE), ({"x": None}, INVALID),
    ({"x": T((4, 8), data=None)}, INVALID), ({"x": T((4, 8), strides=(-8, 1))}, INVALID), ({"q": T((4, 8), dtype=U8)}, DTYPE),
    ({"q": T((4, 7), dtype=I8)}, SHAPE), ({"q": T((4, 8), dtype=I8, strides=(1, 4))}, SHAPE), ({"q": None}, INVALID),
    ({"s": T((4,), dtype=F16)}, DTYPE), ({"s": T((3,))}, SHAPE), ({"s": T((4, 1))}, SHAPE), ({"s": T((4,), strides=(2,))}, SHAPE),
])
def test_quantize_refusals(lib, change, want):
    a = {"x": T((4, 8)), "q": T((4, 8), dtype=I8), "s": T((4,))}
    a.update(change)
    assert lib.mm_quantize_rows(ref(a["x"]), ref(a["q"]), ref(a["s"]), None) == want


@pytest.mark.parametrize("change,want", [
    ({"A": T((5, 16), dtype=U8)}, DTYPE), ({"B": T((16, 24), dtype=BF16)}, DTYPE), ({"B": T((15, 24), dtype=I8)}, SHAPE),
    ({"A": T((2, 5, 16), dtype=I8)}, SHAPE), ({"A": None}, INVALID), ({"B": None}, INVALID), ({"sa": T((5,), dtype=F16)}, DTYPE),
    ({"sa": T((5, 1))}, SHAPE), ({"sa": T((1,))}, SHAPE), ({"sb": T((5,))}, SHAPE), ({"sb": None}, INVALID),
    ({"bias": T((24,), dtype=F32)}, DTYPE), ({"bias": T((23,), dtype=BF16)}, SHAPE), ({"Y": T((5, 24), dtype=F64)}, DTYPE),
    ({"Y": T((5, 24), dtype=I8)}, DTYPE), ({"Y": T((5, 23), dtype=BF16)}, SHAPE), ({"Y": T((5, 24), dtype=BF16, strides=(25, 1))}, SHAPE),
    ({"Y": None}, INVALID), ({"A": T((5, 1 << 31), dtype=I8), "B": T((1 << 31, 24), dtype=I8)}, UNSUPPORTED),
])
def test_int8_refusals(lib, change, want):
    a = {"A": T((5, 16), dtype=I8), "B": T((16, 24), dtype=I8), "sa": T((5,)), "sb": T((24,)), "bias": T((24,), dtype=BF16),
         "Y": T((5, 24), dtype=BF16)}
    a.update(change)
    assert lib.mm_int8_matmul(ref(a["A"]), ref(a["B"]), ref(a["sa"]), ref(a["sb"]), ref(a["bias"]), ref(a["Y"]), 0x10000, 1 << 30,
                              None) == want


def test_int8_size_refusals(lib):
    n = ctypes.c_size_t()
    A, B = T((5, 16), dtype=I8), T((16, 24), dtype=I8)
    assert lib.mm_int8_matmul_workspace_size(ref(A), ref(B), F64, ctypes.byref(n)) == DTYPE
    assert lib.mm_int8_matmul_workspace_size(ref(A), ref(B), BF16, None) == INVALID
    assert lib.mm_int8_matmul_workspace_size(ref(A), ref(T((0, 24), dtype=I8)), BF16, ctypes.byref(n)) == SHAPE


@pytest.mark.parametrize("change,want", [
    ({"l": T((4, 8), dtype=F64)}, DTYPE), ({"l": T((8,))}, SHAPE), ({"l": T((4, 0))}, SHAPE), ({"l": T((4, 1025))}, UNSUPPORTED),
    ({"i": T((4, 2), dtype=F32)}, DTYPE), ({"i": T((3, 2), dtype=I32)}, SHAPE), ({"i": T((4, 0), dtype=I32)}, SHAPE),
    ({"i": None}, INVALID), ({"l": T((1 << 30, 8)), "i": T((1 << 30, 2), dtype=I32)}, UNSUPPORTED),
    ({"loss": T((1,), dtype=BF16)}, DTYPE), ({"loss": T((2,))}, SHAPE), ({"loss": T(())}, SHAPE), ({"counts": T((8,), dtype=I32)}, SHAPE),
    ({"counts": T((9,), dtype=I64)}, DTYPE), ({"mean": T((9,))}, SHAPE), ({"mean": T((8,), strides=(2,))}, SHAPE),
    ({"mean": None}, INVALID), ({"ws": 0}, WORKSPACE), ({"ws": 0x10010}, WORKSPACE), ({"bytes": 3}, WORKSPACE),
])
def test_balance_refusals(lib, change, want):
    a = {"l": T((4, 8)), "i": T((4, 2), dtype=I32), "loss": T((1,)), "counts": T((9,), dtype=I32), "mean": T((8,)),
         "ws": 0x10000, "bytes": 1 << 30}
    a.update(change)
    assert lib.mm_route_balance(ref(a["l"]), ref(a["i"]), ref(a["loss"]), ref(a["counts"]), ref(a["mean"]), a["ws"], a["bytes"],
                                None) == want


@pytest.mark.parametrize("change,want", [
    ({"l": T((4, 8), dtype=I32)}, DTYPE), ({"l": T((4, 8, 1), dtype=BF16)}, SHAPE), ({"c": T((8,), dtype=I32)}, SHAPE), ({"c": T((9,))}, DTYPE),
    ({"c": None}, INVALID), ({"d": T((2,))}, SHAPE), ({"d": T((1,), dtype=BF16)}, DTYPE), ({"b": T((4, 8))}, DTYPE),
    ({"b": T((4, 7), dtype=BF16)}, SHAPE), ({"o": T((4, 8))}, DTYPE), ({"o": T((4, 8), dtype=BF16, strides=(1, 4))}, SHAPE),
    ({"o": None}, INVALID), ({"l": T((4, 1025), dtype=BF16), "c": T((1026,), dtype=I32), "b": None, "o": T((4, 1025), dtype=BF16)}, UNSUPPORTED),
])
def test_balance_grad_refusals(lib, change, want):
    a = {"l": T((4, 8), dtype=BF16), "c": T((9,), dtype=I32), "d": T((1,)), "b": T((4, 8), dtype=BF16), "o": T((4, 8), dtype=BF16)}
    a.update(change)
    assert lib.mm_route_balance_grad(ref(a["l"]), ref(a["c"]), ref(a["d"]), ref(a["b"]), ref(a["o"]), None) == want


@pytest.mark.parametrize("change,want", [
    ({"X": T((8,))}, SHAPE), ({"X": T((4, 8), dtype=F64)}, DTYPE), ({"X": T((4, 8), strides=(8, -1))}, INVALID), ({"X": None}, INVALID),
    ({"Y": T((4, 8), dtype=BF16)}, DTYPE), ({"Y": T((1, 4, 8))}, SHAPE), ({"Y": T((8, 4))}, SHAPE), ({"Y": T((4, 8), strides=(1, 4))}, SHAPE),
    ({"steps": -1}, INVALID), ({"steps": 65}, INVALID), ({"coef": None}, INVALID), ({"coef": (1.0, math.inf, 0.0)}, INVALID),
    ({"coef": (1.0, 0.0, math.nan)}, INVALID), ({"eps": -1e-9}, INVALID), ({"eps": math.nan}, INVALID), ({"scale": math.inf}, INVALID),
])
def test_orthogonalize_refusals(lib, change, want):
    a = {"X": T((4, 8)), "Y": T((4, 8)), "steps": 1, "coef": (1.5, -0.5, 0.0), "eps": 1e-7, "scale": 1.0, "ws": 0x10000, "bytes": 1 << 30}
    a.update(change)
    coef = None if a["coef"] is None else (ctypes.c_float * 3)(*a["coef"])
    assert lib.mm_orthogonalize(ref(a["X"]), a["steps"], coef, a["eps"], a["scale"], ref(a["Y"]), a["ws"], a["bytes"], None) == want


def test_orthogonalize_binding_refuses_coefficients_for_another_number_of_steps(lib):
    x = torch.zeros((4, 8))
    for bad in ([(1.5, -0.5, 0.0)] * 2, (1.5, -0.5)):
        with pytest.raises(ValueError):
            qg.mm_orthogonalize(x, steps=3, coefficients=bad)


def test_int8_binding_refuses_a_type_it_does_not_know(lib):
    a = torch.zeros((4, 8), dtype=torch.int8)
    with pytest.raises(TypeError):
        qg.mm_int8_matmul_workspace_size(a, a.t(), torch.complex64)
    with pytest.raises(qg.MMError) as e:
        qg.mm_int8_matmul_workspace_size(a, a.t(), torch.float64)
    assert e.value.name == "MM_ERR_DTYPE"
