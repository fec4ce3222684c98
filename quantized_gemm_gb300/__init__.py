"""Python binding of the GB300 ONNX matrix-product library (include/mm.h).

Argument marshalling only: every function below turns torch tensors into the
C ABI's ``mm_tensor`` descriptors (device pointer, type, shape, element
strides), allocates the output (and, where the fast path needs one, the
workspace) with torch's allocator, and calls the library's entry point of the
same name on the current CUDA stream.  All arithmetic runs in the library's
CUDA kernels; there is no fallback of any kind, and importing a function whose
shared library was not built raises immediately.
"""

import ctypes
import os
import struct

import torch

__all__ = [
    "MMError", "mm_matmul", "mm_gemm", "mm_qlinear_matmul", "mm_grouped_matmul",
    "mm_get_device_status", "mm_set_path_policy", "mm_last_path", "mm_set_wait_limit_ns", "mm_version",
    "library_path",
    "mm_qlinear_matmul_workspace_size", "mm_grouped_matmul_workspace_size", "mm_grouped_matmul_noalloc",
    "mm_grouped_matmul_qweights", "mm_grouped_matmul_qweights_workspace_size",
    "MM_PATH_AUTO", "MM_PATH_SIMT", "MM_PATH_TENSOR", "MM_PATH_NONE", "MM_PATH_VECTOR", "mm_stream_probe",
    "mm_alu_probe", "MM_ALU_CHAINS",
    "mm_route_topk", "mm_route_topk_grad", "mm_moe_layer", "mm_moe_layer_workspace_size",
    "mm_lowrank_matmul", "mm_lowrank_matmul_workspace_size", "mm_lowrank_matmul_grad",
    "mm_lowrank_matmul_grad_workspace_size",
    "mm_route_balance", "mm_route_balance_workspace_size", "mm_route_balance_grad",
    "mm_quantize_rows", "mm_int8_matmul", "mm_int8_matmul_workspace_size",
    "mm_orthogonalize", "mm_orthogonalize_workspace_size",
]

MM_MAX_DIMS = 8
MM_PATH_AUTO, MM_PATH_SIMT, MM_PATH_TENSOR, MM_PATH_NONE, MM_PATH_VECTOR = 0, 1, 2, 3, 4
_STATUS = ["MM_OK", "MM_ERR_INVALID_ARG", "MM_ERR_SHAPE", "MM_ERR_DTYPE", "MM_ERR_UNSUPPORTED",
           "MM_ERR_WORKSPACE", "MM_ERR_CUDA", "MM_ERR_TIMEOUT", "MM_ERR_INDEX_RANGE"]

_DTYPES = {
    torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float64: 3,
    torch.int32: 4, torch.int64: 5, torch.uint32: 6, torch.uint64: 7,
    torch.int8: 8, torch.uint8: 9,
}
# 4-bit types (include/mm.h MM_I4 / MM_U4), which torch has no dtype for:
# passed as uint8 bytes holding two values each (see _desc4).
_PACKED4 = {"int4": 10, "uint4": 11}


def library_path():
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqgemm_gb300.so")


class MMTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * MM_MAX_DIMS), ("strides", ctypes.c_int64 * MM_MAX_DIMS)]


class _Descriptor:
    """Argument type of a descriptor: its packed bytes as they are (see _packed), a pointer to an MMTensor, or None."""

    @classmethod
    def from_param(cls, d):
        return d if d is None or isinstance(d, bytes) else ctypes.POINTER(MMTensor).from_param(d)


class MMError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        self.name = _STATUS[status] if 0 <= status < len(_STATUS) else "unknown"
        super().__init__("%s: %s" % (where, _lib().mm_status_string(status).decode()))


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError("the CUDA library %s is not built; run __graft_entry__.build() "
                               "(or python -m quantized_gemm_gb300.build)" % path)
        lib = ctypes.CDLL(path)
        P, I32, I64, F, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        T = ctypes.POINTER(MMTensor)
        D = _Descriptor                # an MMTensor's bytes, or a pointer to one
        sigs = {
            "mm_status_string": ([I32], ctypes.c_char_p),
            "mm_version": ([], ctypes.c_char_p),
            "mm_set_path_policy": ([I32], I32),
            "mm_last_path": ([], I32),
            "mm_matmul_output_shape": ([T, T, ctypes.POINTER(I32), ctypes.POINTER(I64)], I32),
            "mm_matmul": ([T, T, T, P], I32),
            "mm_gemm_output_shape": ([T, T, I64, I64, ctypes.POINTER(I32), ctypes.POINTER(I64)], I32),
            "mm_gemm": ([T, T, T, F, F, I64, I64, T, P], I32),
            "mm_qlinear_matmul_workspace_size": ([T, T, ctypes.POINTER(SZ)], I32),
            "mm_qlinear_matmul": ([T, T, T, T, T, T, T, T, T, P, SZ, P], I32),
            "mm_grouped_matmul_workspace_size": ([T, T, T, ctypes.POINTER(SZ)], I32),
            "mm_grouped_matmul": ([T, T, T, T, T, P, SZ, P], I32),
            "mm_get_device_status": ([P], I32),
            "mm_grouped_matmul_noalloc_max_scratch": ([], SZ),
            "mm_set_wait_limit_ns": ([ctypes.c_uint64], I32),
            "mm_grouped_matmul_noalloc": ([T, T, T, T, T, P], I32),
            "mm_grouped_matmul_qweights_workspace_size": ([T, T, T, T, I64, T, ctypes.POINTER(SZ)], I32),
            "mm_grouped_matmul_qweights": ([T, T, T, T, I64, T, T, T, P, SZ, P], I32),
            "mm_stream_probe": ([P, P, SZ, I32, P], I32),
            "mm_alu_probe": ([I32, P, I64, P, P], I32),
            "mm_route_topk": ([T, I32, T, T, P], I32),
            "mm_route_topk_grad": ([T, T, T, I32, T, P], I32),
            "mm_moe_layer_workspace_size": ([T, T, T, T, T, ctypes.POINTER(SZ)], I32),
            "mm_moe_layer": ([T, T, T, T, T, T, I32, T, P, SZ, P], I32),
            "mm_lowrank_matmul_workspace_size": ([T, T, T, T, ctypes.POINTER(SZ)], I32),
            "mm_lowrank_matmul": ([T, T, T, T, T, T, T, P, SZ, P], I32),
            "mm_lowrank_matmul_grad_workspace_size": ([T, T, T, T, ctypes.POINTER(SZ)], I32),
            "mm_route_balance_workspace_size": ([D, D, ctypes.POINTER(SZ)], I32),
            "mm_route_balance": ([D, D, D, D, D, P, SZ, P], I32),
            "mm_route_balance_grad": ([D, D, D, D, D, P], I32),
            "mm_quantize_rows": ([D, D, D, P], I32),
            "mm_int8_matmul_workspace_size": ([D, D, I32, ctypes.POINTER(SZ)], I32),
            "mm_int8_matmul": ([D, D, D, D, D, D, P, SZ, P], I32),
            "mm_orthogonalize_workspace_size": ([D, ctypes.POINTER(SZ)], I32),
            "mm_orthogonalize": ([D, I32, ctypes.POINTER(F), F, F, D, P, SZ, P], I32),
            "mm_lowrank_matmul_grad": ([T, T, T, T, T, T, T, T, T, T, P, SZ, P], I32),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _LIB = lib
    return _LIB


# MMTensor's bytes: pointer, dtype, ndim, shape[8], strides[8] (packed in one
# call, which is cheaper than filling the ctypes arrays element by element; one
# format per rank, whose pad bytes are the unused entries' zeros).
_MM_TENSOR_BYTES = struct.Struct("<Qii%dq%dq" % (MM_MAX_DIMS, MM_MAX_DIMS))
_PACK = [struct.Struct("<Qii%dq%dx%dq%dx" % (n, 8 * (MM_MAX_DIMS - n), n, 8 * (MM_MAX_DIMS - n))).pack
         for n in range(MM_MAX_DIMS + 1)]
_TENSOR_OF = MMTensor.from_buffer_copy
_ZEROS = (0,) * MM_MAX_DIMS


def _desc(t):
    """mm_tensor describing torch tensor ``t`` (None -> NULL)."""
    if t is None:
        return None
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError("unsupported dtype %s" % t.dtype)
    nd = t.dim()
    if nd > MM_MAX_DIMS:
        raise ValueError("at most %d dimensions" % MM_MAX_DIMS)
    return _TENSOR_OF(_PACK[nd](t.data_ptr() if t.numel() > 0 else 0, dt, nd, *t.shape, *t.stride()))


def _packed(t):
    """The same as bytes, which ctypes passes on without building a structure."""
    if t is None:
        return None
    nd = t.dim()
    if nd > MM_MAX_DIMS:
        raise ValueError("at most %d dimensions" % MM_MAX_DIMS)
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError("unsupported dtype %s" % t.dtype)
    return _PACK[nd](t.data_ptr(), dt, nd, *t.shape, *t.stride())


def _desc4(t, kind):
    """mm_tensor of 4-bit values stored packed in uint8 tensor ``t`` [..., N/2]:
    logical shape [..., N], element strides twice the byte strides (the last
    one 1); the even element of a byte is its low nibble."""
    if t is None:
        return None
    if kind not in _PACKED4:
        raise ValueError("packed4 must be 'int4' or 'uint4'")
    if t.dtype != torch.uint8 or t.dim() < 1 or t.stride(-1) != 1:
        raise ValueError("packed 4-bit values arrive as a uint8 tensor with a unit stride in its last dimension")
    nd = t.dim()
    shape = tuple(t.shape[:-1]) + (2 * t.shape[-1],)
    strides = tuple(2 * st for st in t.stride()[:-1]) + (1,)
    return MMTensor.from_buffer_copy(_MM_TENSOR_BYTES.pack(
        t.data_ptr() if t.numel() > 0 else 0, _PACKED4[kind], nd, *(shape + _ZEROS[nd:]), *(strides + _ZEROS[nd:])))


def _ref(d):
    return None if d is None else ctypes.byref(d)


# The current stream's handle for a device index, without building a
# torch.cuda.Stream object (the public route below when torch lacks it).
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t, stream):
    if stream is None:
        if _RAW_STREAM is not None and t.is_cuda:
            return ctypes.c_void_p(_RAW_STREAM(t.get_device()))
        stream = torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(stream.cuda_stream)


def _handle(t, stream):
    """The stream's handle as a number."""
    if stream is None and _RAW_STREAM is not None and t.is_cuda:
        return _RAW_STREAM(t.get_device())
    return _stream(t, stream).value


def _empty(shape, dtype, like, stream):
    """Memory for a call on ``stream`` (None: the current one), of that stream's own: what torch hands out on the current
    stream may still be in use by work queued there, which another stream does not wait for.  The current stream may
    then use it until it is freed, too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    current = torch.cuda.current_stream(like.device)
    if stream == current:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(current)
    return t


def _check(status, where):
    if status != 0:
        raise MMError(status, where)


def _out_shape(fn, *args):
    nd = ctypes.c_int32()
    shape = (ctypes.c_int64 * MM_MAX_DIMS)()
    _check(fn(*args, ctypes.byref(nd), shape), fn.__name__)
    return tuple(shape[i] for i in range(nd.value))


def _workspace(nbytes, like, stream, given=None):
    """(tensor, size) of a workspace of at least ``nbytes``: ``given`` when it is large enough."""
    if nbytes == 0:
        return None, 0
    if given is not None:
        if given.numel() * given.element_size() < nbytes:
            raise ValueError("workspace of %d bytes is smaller than the %d required" % (given.numel(), nbytes))
        return given, given.numel() * given.element_size()
    return _empty(nbytes, torch.uint8, like, stream), nbytes


def mm_qlinear_matmul_workspace_size(a, b):
    nbytes = ctypes.c_size_t()
    _check(_lib().mm_qlinear_matmul_workspace_size(_ref(_desc(a)), _ref(_desc(b)), ctypes.byref(nbytes)),
           "mm_qlinear_matmul_workspace_size")
    return nbytes.value


def mm_grouped_matmul_workspace_size(input, weights, group_indices):
    nbytes = ctypes.c_size_t()
    _check(_lib().mm_grouped_matmul_workspace_size(_ref(_desc(input)), _ref(_desc(weights)), _ref(_desc(group_indices)),
                                                   ctypes.byref(nbytes)), "mm_grouped_matmul_workspace_size")
    return nbytes.value


def mm_version():
    return _lib().mm_version().decode()


def mm_set_path_policy(policy):
    _check(_lib().mm_set_path_policy(policy), "mm_set_path_policy")


def mm_last_path():
    return _lib().mm_last_path()


def mm_set_wait_limit_ns(ns):
    """Limit of each tensor-core pipeline wait, in ns (0 = default 2 s)."""
    _check(_lib().mm_set_wait_limit_ns(int(ns)), "mm_set_wait_limit_ns")


def mm_stream_probe(dst, src=None, mode=0, stream=None):
    """Memory-stream measurement kernel on the bytes of ``dst``: mode 0 writes
    them, 1 copies ``src`` into them (same size), 2 writes them with bulk (TMA)
    stores."""
    nbytes = dst.numel() * dst.element_size()
    if src is not None and src.numel() * src.element_size() != nbytes:
        raise ValueError("src and dst must have the same size in bytes")
    _check(_lib().mm_stream_probe(dst.data_ptr(), None if src is None else src.data_ptr(), nbytes, int(mode),
                                  _stream(dst, stream)), "mm_stream_probe")


# Independent multiply-add chains per thread of mm_alu_probe (include/mm.h).
MM_ALU_CHAINS = 16


def mm_alu_probe(op, iters, out=None, stream=None):
    """Arithmetic-rate probe (op 0 int32 multiply-add, 1 fp64 FMA, 2 fp32 FMA):
    returns the number of multiply-adds the launch performs; with ``out`` (a
    device tensor of at least that many / (MM_ALU_CHAINS * iters) 8-byte
    elements, one per thread) it also launches the probe on the current stream."""
    n = ctypes.c_int64(0)
    ptr = None if out is None else out.data_ptr()
    st = None if out is None else _stream(out, stream)
    _check(_lib().mm_alu_probe(int(op), ptr, int(iters), ctypes.byref(n), st), "mm_alu_probe")
    return n.value


def mm_matmul(A, B, out=None, stream=None):
    """Y = A @ B with numpy.matmul semantics (MatMul, opset 13)."""
    lib = _lib()
    dA, dB = _desc(A), _desc(B)
    # A given output is checked by the library itself (MM_ERR_SHAPE).
    Y = out if out is not None else _empty(_out_shape(lib.mm_matmul_output_shape, _ref(dA), _ref(dB)), A.dtype, A, stream)
    _check(lib.mm_matmul(_ref(dA), _ref(dB), _ref(_desc(Y)), _stream(A, stream)), "mm_matmul")
    return Y


def mm_gemm(A, B, C=None, alpha=1.0, beta=1.0, transA=0, transB=0, out=None, stream=None):
    """Y = alpha * A' @ B' + beta * C (Gemm, opset 13)."""
    lib = _lib()
    dA, dB = _desc(A), _desc(B)
    Y = out if out is not None else _empty(
        _out_shape(lib.mm_gemm_output_shape, _ref(dA), _ref(dB), int(transA), int(transB)), A.dtype, A, stream)
    _check(lib.mm_gemm(_ref(dA), _ref(dB), _ref(_desc(C)), float(alpha), float(beta), int(transA), int(transB),
                       _ref(_desc(Y)), _stream(A, stream)), "mm_gemm")
    return Y


def mm_qlinear_matmul(a, a_scale, a_zero_point, b, b_scale, b_zero_point, y_scale, y_zero_point,
                      out=None, stream=None, workspace=None):
    """Quantized matmul of int8/uint8 tensors (QLinearMatMul, opset 10); y has y_zero_point's type."""
    lib = _lib()
    da, db = _desc(a), _desc(b)
    y = out if out is not None else _empty(_out_shape(lib.mm_matmul_output_shape, _ref(da), _ref(db)),
                                           y_zero_point.dtype, a, stream)
    nbytes = ctypes.c_size_t()
    _check(lib.mm_qlinear_matmul_workspace_size(_ref(da), _ref(db), ctypes.byref(nbytes)),
           "mm_qlinear_matmul_workspace_size")
    ws, wsb = _workspace(nbytes.value, a, stream, workspace)
    _check(lib.mm_qlinear_matmul(_ref(da), _ref(_desc(a_scale)), _ref(_desc(a_zero_point)), _ref(db),
                                 _ref(_desc(b_scale)), _ref(_desc(b_zero_point)), _ref(_desc(y_scale)),
                                 _ref(_desc(y_zero_point)), _ref(_desc(y)),
                                 None if ws is None else ws.data_ptr(), wsb, _stream(a, stream)),
           "mm_qlinear_matmul")
    return y


def mm_grouped_matmul(input, weights, group_indices, bias=None, out=None, stream=None, workspace=None):
    """output[m, i] = input[m] @ weights[group_indices[m, i]] (+ bias[g]) (GroupedMatMul, opset 29)."""
    lib = _lib()
    dx, dw, dg = _desc(input), _desc(weights), _desc(group_indices)
    M, S, N = input.shape[0], group_indices.shape[1], weights.shape[2]
    y = _empty((M, S, N), input.dtype, input, stream) if out is None else out
    nbytes = ctypes.c_size_t()
    _check(lib.mm_grouped_matmul_workspace_size(_ref(dx), _ref(dw), _ref(dg), ctypes.byref(nbytes)),
           "mm_grouped_matmul_workspace_size")
    ws, wsb = _workspace(nbytes.value, input, stream, workspace)
    _check(lib.mm_grouped_matmul(_ref(dx), _ref(dw), _ref(dg), _ref(_desc(bias)), _ref(_desc(y)),
                                 None if ws is None else ws.data_ptr(), wsb, _stream(input, stream)),
           "mm_grouped_matmul")
    return y


def _qdesc(t, packed4):
    return _desc(t) if packed4 is None else _desc4(t, packed4)


def mm_grouped_matmul_qweights_workspace_size(input, weights_q, w_scale, w_zero_point, block_size, group_indices,
                                              packed4=None):
    nbytes = ctypes.c_size_t()
    _check(_lib().mm_grouped_matmul_qweights_workspace_size(
        _ref(_desc(input)), _ref(_qdesc(weights_q, packed4)), _ref(_desc(w_scale)),
        _ref(_qdesc(w_zero_point, packed4)), int(block_size), _ref(_desc(group_indices)), ctypes.byref(nbytes)),
        "mm_grouped_matmul_qweights_workspace_size")
    return nbytes.value


def mm_grouped_matmul_qweights(input, weights_q, w_scale, w_zero_point, block_size, group_indices, bias=None,
                               out=None, stream=None, workspace=None, packed4=None):
    """GroupedMatMul of quantized experts: input[m] @ W[g] (+ bias[g]) with
    W = DequantizeLinear(weights_q, w_scale, w_zero_point) in blocks of
    ``block_size`` rows of K (0: one scale per group and column), fused.
    weights_q and w_zero_point are int8/uint8 tensors, or with ``packed4``
    ('int4' or 'uint4') uint8 tensors [G, K, N/2] / [G, Kb, N/2] holding two
    4-bit values per byte (the even column in the low nibble)."""
    lib = _lib()
    M, S = input.shape[0], group_indices.shape[1]
    N = weights_q.shape[2] * (2 if packed4 is not None else 1)
    y = _empty((M, S, N), input.dtype, input, stream) if out is None else out
    ws, wsb = _workspace(mm_grouped_matmul_qweights_workspace_size(input, weights_q, w_scale, w_zero_point,
                                                                   block_size, group_indices, packed4),
                         input, stream, workspace)
    _check(lib.mm_grouped_matmul_qweights(_ref(_desc(input)), _ref(_qdesc(weights_q, packed4)), _ref(_desc(w_scale)),
                                          _ref(_qdesc(w_zero_point, packed4)), int(block_size),
                                          _ref(_desc(group_indices)),
                                          _ref(_desc(bias)), _ref(_desc(y)), None if ws is None else ws.data_ptr(),
                                          wsb, _stream(input, stream)),
           "mm_grouped_matmul_qweights")
    return y


def mm_grouped_matmul_noalloc(input, weights, group_indices, bias=None, out=None, stream=None):
    """GroupedMatMul for callers that cannot allocate device memory per call.

    Same result as mm_grouped_matmul, computed with scratch taken from a fixed
    array the library keeps on each device (no workspace argument, no
    allocation by the library).  ``out`` must be given by such callers; when
    it is None this binding allocates it with torch for convenience.
    """
    y = _empty((input.shape[0], group_indices.shape[1], weights.shape[2]), input.dtype, input,
               stream) if out is None else out
    _check(_lib().mm_grouped_matmul_noalloc(_ref(_desc(input)), _ref(_desc(weights)), _ref(_desc(group_indices)),
                                            _ref(_desc(bias)), _ref(_desc(y)), _stream(input, stream)),
           "mm_grouped_matmul_noalloc")
    return y


# The calls below take a few microseconds on the device for small sizes, as
# long as their marshalling: it is written out, without lists or helpers on
# the way of a call that passes its workspace.


def mm_route_topk(logits, k, normalize=1, indices=None, weights=None, stream=None):
    """Top-k routing of logits [T, G]: (indices int32 [T, k], weights fp32 [T, k]), the largest logits first, ties to
    the lowest index; weights are the softmax over all experts, divided by the picks' sum when ``normalize``."""
    lib = _LIB or _lib()
    if indices is None:
        indices = _empty((logits.shape[0], k), torch.int32, logits, stream)
    elif indices.shape[-1] != k:
        raise ValueError("indices for %d picks, k is %d" % (indices.shape[-1], k))
    if weights is None:
        weights = _empty((logits.shape[0], k), torch.float32, logits, stream)
    status = lib.mm_route_topk(_ref(_desc(logits)), int(normalize), _ref(_desc(indices)), _ref(_desc(weights)),
                               _stream(logits, stream))
    if status:
        raise MMError(status, "mm_route_topk")
    return indices, weights


def mm_route_topk_grad(logits, indices, grad_weights, normalize=1, out=None, stream=None):
    """Gradient of mm_route_topk's weights with respect to the logits (in the logits' type)."""
    lib = _LIB or _lib()
    y = _empty(logits.shape, logits.dtype, logits, stream) if out is None else out
    status = lib.mm_route_topk_grad(_ref(_desc(logits)), _ref(_desc(indices)), _ref(_desc(grad_weights)),
                                    int(normalize), _ref(_desc(y)), _stream(logits, stream))
    if status:
        raise MMError(status, "mm_route_topk_grad")
    return y


def mm_route_balance_workspace_size(logits, indices):
    return _room(_lib().mm_route_balance_workspace_size, _packed(logits), _packed(indices))


def _room(fn, *args):
    """Bytes of workspace that ``fn`` names."""
    nbytes = ctypes.c_size_t()
    _check(fn(*args, ctypes.byref(nbytes)), fn.__name__)
    return nbytes.value


def _work(workspace, like, stream, fn, *args):
    """(tensor, address, size) of the workspace: the caller's (the library checks its size), or one of the size ``fn``
    names; the tensor keeps the memory until the call has been made."""
    if workspace is None:
        workspace, nbytes = _workspace(_room(fn, *args), like, stream)
        return workspace, None if workspace is None else workspace.data_ptr(), nbytes
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def mm_route_balance(logits, indices, loss=None, counts=None, mean_probs=None, stream=None, workspace=None):
    """The router's balance loss: (loss fp32 [1], counts int32 [G + 1], mean_probs fp32 [G]) with loss = G * sum_g
    (counts[g] / all picks) * mean_probs[g]; the last place of counts holds the rows that take part (a row of -inf
    alone is padding)."""
    lib = _LIB or _lib()
    G = logits.shape[1]
    dl, di = _packed(logits), _packed(indices)
    if loss is None:
        loss = _empty((1,), torch.float32, logits, stream)
    if counts is None:
        counts = _empty((G + 1,), torch.int32, logits, stream)
    if mean_probs is None:
        mean_probs = _empty((G,), torch.float32, logits, stream)
    ws, at, nbytes = _work(workspace, logits, stream, lib.mm_route_balance_workspace_size, dl, di)
    status = lib.mm_route_balance(dl, di, _packed(loss), _packed(counts), _packed(mean_probs), at, nbytes,
                                  _handle(logits, stream))
    if status:
        raise MMError(status, "mm_route_balance")
    return loss, counts, mean_probs


def mm_route_balance_grad(logits, counts, grad_loss, base=None, out=None, stream=None):
    """Gradient of mm_route_balance's loss with respect to the logits, times grad_loss (one fp32 value on the device),
    plus ``base``, another gradient of the logits."""
    lib = _LIB or _lib()
    y = _empty(logits.shape, logits.dtype, logits, stream) if out is None else out
    status = lib.mm_route_balance_grad(_packed(logits), _packed(counts), _packed(grad_loss), _packed(base), _packed(y),
                                       _handle(logits, stream))
    if status:
        raise MMError(status, "mm_route_balance_grad")
    return y


_ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}


def _sized(fn, *descs):
    nbytes = ctypes.c_size_t()
    _check(fn(*[_ref(d) for d in descs], ctypes.byref(nbytes)), fn.__name__)
    return nbytes.value


def _given_or_sized(workspace, like, stream, fn, *descs):
    """(tensor, size) of the workspace: the caller's (the library checks its size), or one of the size ``fn`` names."""
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    return _workspace(_sized(fn, *descs), like, stream)


def mm_moe_layer_workspace_size(x, w_gate, w_up, w_down, expert_indices):
    return _sized(_lib().mm_moe_layer_workspace_size, _desc(x), _desc(w_gate), _desc(w_up), _desc(w_down),
                  _desc(expert_indices))


def mm_moe_layer(x, w_gate, w_up, w_down, expert_indices, expert_weights=None, activation="silu", out=None,
                 stream=None, workspace=None):
    """The mixture-of-experts layer for a few tokens: out[t] = sum_s expert_weights[t, s] * (act(x[t] @ w_gate[e]) *
    (x[t] @ w_up[e])) @ w_down[e], e = expert_indices[t, s] (-1: no pick).  ``activation`` is 'silu', 'gelu' or
    'relu'; w_up None leaves the second factor out."""
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be one of %s" % ", ".join(sorted(_ACTIVATIONS)))
    lib = _LIB or _lib()
    dx, dg, du, dd, di = _desc(x), _desc(w_gate), _desc(w_up), _desc(w_down), _desc(expert_indices)
    y = _empty((x.shape[0], w_down.shape[2]), x.dtype, x, stream) if out is None else out
    ws, wsb = _given_or_sized(workspace, x, stream, lib.mm_moe_layer_workspace_size, dx, dg, du, dd, di)
    status = lib.mm_moe_layer(_ref(dx), _ref(dg), _ref(du), _ref(dd), _ref(di),
                              _ref(_desc(expert_weights)), act, _ref(_desc(y)),
                              None if ws is None else ws.data_ptr(), wsb, _stream(x, stream))
    if status:
        raise MMError(status, "mm_moe_layer")
    return y


def mm_lowrank_matmul_workspace_size(X, W, A, B):
    return _sized(_lib().mm_lowrank_matmul_workspace_size, _desc(X), _desc(W), _desc(A), _desc(B))


def mm_lowrank_matmul(X, W, A, B, adapter_indices, scales=None, out=None, stream=None, workspace=None):
    """X @ W plus each row's low-rank adapter: Y[m] = X[m] @ W + scales[g] * (X[m] @ A[g]) @ B[g],
    g = adapter_indices[m] (-1: no adapter)."""
    lib = _LIB or _lib()
    dX, dW, dA, dB = _desc(X), _desc(W), _desc(A), _desc(B)
    y = _empty((X.shape[0], W.shape[1]), X.dtype, X, stream) if out is None else out
    ws, wsb = _given_or_sized(workspace, X, stream, lib.mm_lowrank_matmul_workspace_size, dX, dW, dA, dB)
    status = lib.mm_lowrank_matmul(_ref(dX), _ref(dW), _ref(dA), _ref(dB), _ref(_desc(adapter_indices)),
                                   _ref(_desc(scales)), _ref(_desc(y)),
                                   None if ws is None else ws.data_ptr(), wsb, _stream(X, stream))
    if status:
        raise MMError(status, "mm_lowrank_matmul")
    return y


def mm_lowrank_matmul_grad_workspace_size(X, W, A, B):
    return _sized(_lib().mm_lowrank_matmul_grad_workspace_size, _desc(X), _desc(W), _desc(A), _desc(B))


def mm_lowrank_matmul_grad(dY, X, W, A, B, adapter_indices, scales=None, need=(True, True, True), stream=None,
                           workspace=None):
    """Gradients (dX, dA, dB) of mm_lowrank_matmul for a frozen W; ``need`` says which are wanted (None in the
    others' place)."""
    lib = _LIB or _lib()
    d = [_desc(t) for t in (X, W, A, B)]
    dX = _empty(X.shape, X.dtype, X, stream) if need[0] else None
    dA = _empty(A.shape, A.dtype, X, stream) if need[1] else None
    dB = _empty(B.shape, B.dtype, X, stream) if need[2] else None
    ws, wsb = _given_or_sized(workspace, X, stream, lib.mm_lowrank_matmul_grad_workspace_size, *d)
    status = lib.mm_lowrank_matmul_grad(_ref(_desc(dY)), *[_ref(t) for t in d], _ref(_desc(adapter_indices)),
                                        _ref(_desc(scales)), _ref(_desc(dX)), _ref(_desc(dA)), _ref(_desc(dB)),
                                        None if ws is None else ws.data_ptr(), wsb, _stream(X, stream))
    if status:
        raise MMError(status, "mm_lowrank_matmul_grad")
    return dX, dA, dB


def mm_quantize_rows(x, out=None, scales=None, stream=None):
    """Rows of x [M, K] as int8 with a scale each: (q int8 [M, K], scales fp32 [M]), x ~ q * scales[:, None].  For
    weights [K, N] pass their transpose: a scale per output channel."""
    lib = _LIB or _lib()
    q = _empty(x.shape, torch.int8, x, stream) if out is None else out
    if scales is None:
        scales = _empty(x.shape[:1], torch.float32, x, stream)
    status = lib.mm_quantize_rows(_packed(x), _packed(q), _packed(scales), _handle(x, stream))
    if status:
        raise MMError(status, "mm_quantize_rows")
    return q, scales


def _type_of(dtype):
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("unsupported dtype %s" % dtype)
    return dt


def mm_int8_matmul_workspace_size(A, B, dtype=torch.bfloat16):
    return _room(_lib().mm_int8_matmul_workspace_size, _packed(A), _packed(B), _type_of(dtype))


def mm_int8_matmul(A, B, a_scale, b_scale, bias=None, dtype=torch.bfloat16, out=None, stream=None, workspace=None):
    """Product of int8 tensors scaled per row of A and per column of B: Y[m, n] = sum_k A[m, k] B[k, n] * a_scale[m] *
    b_scale[n] + bias[n], in ``dtype`` (or the type of ``out``).  Weights quantised as [N, K] rows are passed transposed."""
    lib = _LIB or _lib()
    dA, dB = _packed(A), _packed(B)
    y = _empty((A.shape[0], B.shape[1]), dtype, A, stream) if out is None else out
    ws, at, nbytes = _work(workspace, A, stream, lib.mm_int8_matmul_workspace_size, dA, dB, _type_of(y.dtype))
    status = lib.mm_int8_matmul(dA, dB, _packed(a_scale), _packed(b_scale), _packed(bias), _packed(y), at, nbytes,
                                _handle(A, stream))
    if status:
        raise MMError(status, "mm_int8_matmul")
    return y


def mm_orthogonalize_workspace_size(X):
    return _room(_lib().mm_orthogonalize_workspace_size, _packed(X))


def mm_orthogonalize(X, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0, out=None, stream=None,
                     workspace=None):
    """Each matrix of X [..., M, N] divided by its Frobenius norm (plus eps) and driven towards the nearest orthogonal
    one by ``steps`` of X = a X + (b X X^T + c (X X^T)^2) X, times ``scale``.  ``coefficients`` is one (a, b, c) for all
    steps, or a sequence of them, one a step."""
    lib = _LIB or _lib()
    steps = int(steps)
    if steps and isinstance(coefficients[0], (tuple, list)):
        if len(coefficients) != steps:
            raise ValueError("coefficients for %d steps, steps is %d" % (len(coefficients), steps))
        flat = [v for step in coefficients for v in step]
    else:
        flat = list(coefficients) * steps
    if len(flat) != 3 * max(0, steps):
        raise ValueError("three coefficients a step")
    dX = _packed(X)
    y = _empty(X.shape, X.dtype, X, stream) if out is None else out
    ws, at, nbytes = _work(workspace, X, stream, lib.mm_orthogonalize_workspace_size, dX)
    status = lib.mm_orthogonalize(dX, steps, (ctypes.c_float * max(1, len(flat)))(*flat), eps, scale, _packed(y), at,
                                  nbytes, _handle(X, stream))
    if status:
        raise MMError(status, "mm_orthogonalize")
    return y


def mm_get_device_status(stream=None, device=None):
    """Synchronise the stream; return (and clear) the device-side status name, e.g. 'MM_OK'."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    s = _lib().mm_get_device_status(ctypes.c_void_p(stream.cuda_stream))
    return _STATUS[s]
