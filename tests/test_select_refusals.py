"""What the routing, expert-layer and low-rank entry points refuse (no GPU: every call fails validation first)."""

import ctypes

import pytest

import quantized_gemm_gb300 as qg
from quantized_gemm_gb300 import build as qbuild
from test_abi import T

BF16, F16, F32, F64, I32, I64, I8 = 0, 1, 2, 3, 4, 5, 8
INVALID, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qg._lib()


def ref(t):
    return None if t is None else ctypes.byref(t)


@pytest.mark.parametrize("change,want", [
    ({"logits": T((4, 8), dtype=F64)}, DTYPE), ({"logits": T((4, 8, 1))}, SHAPE), ({"logits": T((4, 8), data=None)}, INVALID),
    ({"logits": None}, INVALID), ({"indices": T((4, 2), dtype=I64)}, DTYPE), ({"indices": T((3, 2), dtype=I32)}, SHAPE),
    ({"weights": T((4, 2), dtype=BF16)}, DTYPE), ({"weights": T((4, 3))}, SHAPE),
    ({"weights": T((4, 2), strides=(1, 4))}, SHAPE),
    ({"indices": T((4, 9), dtype=I32), "weights": T((4, 9))}, SHAPE),
    ({"indices": T((4, 0), dtype=I32), "weights": T((4, 0))}, SHAPE),
    ({"logits": T((4, 40)), "indices": T((4, 33), dtype=I32), "weights": T((4, 33))}, SHAPE),
    ({"logits": T((4, 1025))}, UNSUPPORTED),
])
def test_route_refusals(lib, change, want):
    a = {"logits": T((4, 8)), "indices": T((4, 2), dtype=I32), "weights": T((4, 2))}
    a.update(change)
    assert lib.mm_route_topk(ref(a["logits"]), 1, ref(a["indices"]), ref(a["weights"]), None) == want


@pytest.mark.parametrize("change,want", [
    ({"indices": T((4, 2), dtype=I8)}, DTYPE), ({"dw": T((4, 2), dtype=BF16)}, DTYPE), ({"dw": T((4, 3))}, SHAPE),
    ({"out": T((4, 8), dtype=BF16)}, DTYPE), ({"out": T((4, 7))}, SHAPE), ({"indices": T((5, 2), dtype=I32)}, SHAPE),
    ({"out": None}, INVALID),
])
def test_route_grad_refusals(lib, change, want):
    a = {"logits": T((4, 8)), "indices": T((4, 2), dtype=I32), "dw": T((4, 2)), "out": T((4, 8))}
    a.update(change)
    assert lib.mm_route_topk_grad(ref(a["logits"]), ref(a["indices"]), ref(a["dw"]), 1, ref(a["out"]), None) == want


@pytest.mark.parametrize("change,want", [
    ({"x": T((3, 16), dtype=F64)}, DTYPE), ({"x": T((3, 15), dtype=BF16)}, SHAPE), ({"wg": T((4, 16, 8), dtype=F16)}, DTYPE),
    ({"wu": T((4, 16, 9), dtype=BF16)}, SHAPE), ({"wu": T((4, 16, 8), dtype=F32)}, DTYPE),
    ({"wd": T((4, 9, 24), dtype=BF16)}, SHAPE), ({"wd": T((3, 8, 24), dtype=BF16)}, SHAPE),
    ({"gi": T((3, 2), dtype=F32)}, DTYPE), ({"gi": T((2, 2), dtype=I32)}, SHAPE), ({"gi": None}, INVALID),
    ({"ew": T((3, 2), dtype=BF16)}, DTYPE), ({"ew": T((3, 1))}, SHAPE), ({"act": 3}, INVALID), ({"act": -1}, INVALID),
    ({"out": T((3, 23), dtype=BF16)}, SHAPE), ({"out": T((3, 24))}, DTYPE),
    ({"out": T((3, 24), dtype=BF16, strides=(25, 1))}, SHAPE), ({"x": T((3, 16), dtype=BF16, strides=(-16, 1))}, INVALID),
    ({"ws": 0}, WORKSPACE), ({"ws": 0x1010}, WORKSPACE), ({"bytes": 3}, WORKSPACE),
])
def test_moe_refusals(lib, change, want):
    a = {"x": T((3, 16), dtype=BF16), "wg": T((4, 16, 8), dtype=BF16), "wu": T((4, 16, 8), dtype=BF16),
         "wd": T((4, 8, 24), dtype=BF16), "gi": T((3, 2), dtype=I32), "ew": T((3, 2)), "act": 0,
         "out": T((3, 24), dtype=BF16), "ws": 0x10000, "bytes": 1 << 30}
    a.update(change)
    if want == WORKSPACE:      # checked after the status word's device address is known
        import torch
        if not torch.cuda.is_available():
            pytest.skip("needs a device")
    assert lib.mm_moe_layer(ref(a["x"]), ref(a["wg"]), ref(a["wu"]), ref(a["wd"]), ref(a["gi"]), ref(a["ew"]), a["act"],
                            ref(a["out"]), a["ws"], a["bytes"], None) == want


@pytest.mark.parametrize("change,want", [
    ({"X": T((5, 16), dtype=F64)}, DTYPE), ({"W": T((15, 24), dtype=BF16)}, SHAPE), ({"W": T((16, 24), dtype=F16)}, DTYPE),
    ({"A": T((3, 15, 4), dtype=BF16)}, SHAPE), ({"A": T((2, 16, 4), dtype=BF16)}, SHAPE),
    ({"B": T((3, 5, 24), dtype=BF16)}, SHAPE), ({"B": T((3, 4, 23), dtype=BF16)}, SHAPE),
    ({"idx": T((5, 1), dtype=I32)}, SHAPE), ({"idx": T((4,), dtype=I32)}, SHAPE), ({"idx": T((5,), dtype=F32)}, DTYPE),
    ({"idx": None}, INVALID), ({"scales": T((3,), dtype=BF16)}, DTYPE), ({"scales": T((2,))}, SHAPE),
    ({"ws": 0}, WORKSPACE), ({"ws": 0x1010}, WORKSPACE), ({"bytes": 3}, WORKSPACE),
])
def test_lowrank_refusals(lib, change, want):
    a = {"X": T((5, 16), dtype=BF16), "W": T((16, 24), dtype=BF16), "A": T((3, 16, 4), dtype=BF16),
         "B": T((3, 4, 24), dtype=BF16), "idx": T((5,), dtype=I32), "scales": T((3,)), "ws": 0x10000, "bytes": 1 << 30}
    a.update(change)
    common = [ref(a[n]) for n in ("X", "W", "A", "B", "idx", "scales")]
    assert lib.mm_lowrank_matmul(*common, ref(T((5, 24), dtype=BF16)), a["ws"], a["bytes"], None) == want
    outs = [ref(T(s, dtype=BF16)) for s in ((5, 16), (3, 16, 4), (3, 4, 24))]
    assert lib.mm_lowrank_matmul_grad(ref(T((5, 24), dtype=BF16)), *common, *outs, a["ws"], a["bytes"], None) == want


def test_lowrank_output_refusals(lib):
    common = [ref(T((5, 16), dtype=BF16)), ref(T((16, 24), dtype=BF16)), ref(T((3, 16, 4), dtype=BF16)),
              ref(T((3, 4, 24), dtype=BF16)), ref(T((5,), dtype=I32)), None]
    assert lib.mm_lowrank_matmul(*common, ref(T((5, 23), dtype=BF16)), 0x10000, 1 << 30, None) == SHAPE
    assert lib.mm_lowrank_matmul(*common, ref(T((5, 24))), 0x10000, 1 << 30, None) == DTYPE
    good = [T((5, 16), dtype=BF16), T((3, 16, 4), dtype=BF16), T((3, 4, 24), dtype=BF16)]
    for at, bad, want in ((0, T((5, 17), dtype=BF16), SHAPE), (1, T((3, 16, 4)), DTYPE),
                          (2, T((3, 4, 24), dtype=BF16, strides=(96, 1, 4)), SHAPE)):
        outs = [bad if i == at else t for i, t in enumerate(good)]
        assert lib.mm_lowrank_matmul_grad(ref(T((5, 24), dtype=BF16)), *common, *[ref(t) for t in outs], 0x10000,
                                          1 << 30, None) == want
    assert lib.mm_lowrank_matmul_grad(ref(T((5, 23), dtype=BF16)), *common, None, None, None, 0x10000, 1 << 30,
                                      None) == SHAPE


def test_workspace_queries(lib):
    n = ctypes.c_size_t()
    args = [T((3, 16), dtype=BF16), T((4, 16, 8), dtype=BF16), None, T((4, 8, 24), dtype=BF16), T((3, 2), dtype=I32)]
    assert lib.mm_moe_layer_workspace_size(*[ref(t) for t in args], ctypes.byref(n)) == 0 and n.value > 0
    assert lib.mm_moe_layer_workspace_size(*[ref(t) for t in args], None) == INVALID
    lr = [T((5, 16), dtype=BF16), T((16, 24), dtype=BF16), T((3, 16, 4), dtype=BF16), T((3, 4, 24), dtype=BF16)]
    assert lib.mm_lowrank_matmul_workspace_size(*[ref(t) for t in lr], ctypes.byref(n)) == 0 and n.value > 0
    assert lib.mm_lowrank_matmul_grad_workspace_size(*[ref(t) for t in lr], ctypes.byref(n)) == 0 and n.value > 0
    lr[2] = T((3, 15, 4), dtype=BF16)
    assert lib.mm_lowrank_matmul_workspace_size(*[ref(t) for t in lr], ctypes.byref(n)) == SHAPE
