"""Python binding of the layer operators of libiqcodec.so (``include/iq_layers.h``):
products in 8-bit integers with a scale per token and per channel, dense and
with a weight per expert, and the routing of tokens to experts and back with
its gradients.

Like the rest of the binding it only marshals: it checks tensors, allocates the
outputs that were not given, and calls the library on the current HIP stream.
Matrices are two-dimensional with consecutive values in a row; rows may have a
stride of their own (slices of larger tensors are taken as they are).
"""

from __future__ import annotations

import ctypes
import sys

import torch

# The package, whose helpers and loaded library the calls below use (it imports
# this module before it defines them).
iq = sys.modules[__package__]

# iq_dtype_t of the values these operators take.
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_CHOICE_BYTES = {torch.int32: 4, torch.int64: 8}
_DEVICES = [torch.device("cuda", i) for i in range(64)]


def declare(L):
    """Argument types of the entry points of ``include/iq_layers.h``."""
    P, i64, i32, c = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    for name, args in {
        "iq_quantize_rows": [c, P, i64, i64, i64, P, i64, P, P, P],
        "iq_int8_matmul": [P, i64, P, P, i64, P, i64, i64, i64, c, P, i64, P],
        "iq_int8_linear": [c, P, i64, P, i64, P, i64, i64, i64, P, i64, P, i64, P, P],
        "iq_int8_expert_matmul": [P, i64, P, i64, P, i32, P, i32, i64, P, i64, i64, P, i64, i64,
                                  c, P, i64, P],
        "iq_expert_sort": [P, i32, i64, i32, i32, P, P, P, P, i64, P, P],
        "iq_expert_dispatch": [c, P, i64, i64, i64, P, i32, P, i32, P, i64, P],
        "iq_expert_dispatch_backward": [c, P, i64, i64, i64, P, i32, P, i32, P, i64, P],
        "iq_expert_combine": [c, P, i64, i64, i64, P, i32, P, i32, P, P, i64, P],
        "iq_expert_combine_backward": [c, P, i64, P, i64, i64, i64, P, i32, P, i32, P, P, i64, P,
                                       P],
    }.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, c
    for name, args in {"iq_int8_linear_workspace": [i64, i64],
                       "iq_expert_sort_workspace": [i64, i32]}.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, i64


def _on_gpu(t, name):
    """The index of a tensor's GPU, which has to be the current device: that is
    where the kernels are launched."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    index = t.get_device()
    if index < 0:
        raise ValueError("%s must be on the GPU" % name)
    if index != torch._C._cuda_getDevice():
        raise ValueError("%s is on cuda:%d, which is not the current device" % (name, index))
    return index


def _refuse(t, name, index):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    raise ValueError("%s must be on cuda:%d" % (name, index))


def _row_stride(t, name, dtype):
    """The row stride of a two-dimensional tensor with consecutive values in a row."""
    if dtype is None:
        if t.dtype not in _DTYPES:
            raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, t.dtype))
    elif t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    stride = t.stride()
    if len(stride) != 2:
        raise ValueError("%s must have two dimensions" % name)
    if stride[1] != 1 and t.shape[1] != 1:
        raise ValueError("%s must have consecutive values in a row" % name)
    return stride[0]


def _first(t, name, dtype=None):
    """A call's first matrix: the GPU it is on, and its row stride."""
    return _on_gpu(t, name), _row_stride(t, name, dtype)


def _matrix(t, name, index, dtype=None):
    """A further matrix, on that GPU: its row stride."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _refuse(t, name, index)
    return _row_stride(t, name, dtype)


def _vector(t, dtype, shape, name, index):
    """The address of a contiguous tensor of the given shape on that GPU."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _refuse(t, name, index)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of shape %s" % (name, tuple(shape)))
    return t.data_ptr()


# The current stream's handle, without the Stream object that
# torch.cuda.current_stream builds around it (1.1 us a call).
_stream = torch._C._cuda_getCurrentRawStream


def _output(out, rows, cols, like, index, name):
    """The result of a call, a matrix like the tensor `like` or of the type it
    is, and its row stride."""
    if out is None:
        if isinstance(like, torch.Tensor):
            return like.new_empty((rows, cols)), cols
        return torch.empty((rows, cols), dtype=like, device=_DEVICES[index]), cols
    dtype = like.dtype if isinstance(like, torch.Tensor) else like
    stride = _matrix(out, name, index, dtype)
    if out.shape != (rows, cols):
        raise ValueError("%s must be [%d, %d]" % (name, rows, cols))
    return out, stride


def _status(status, check, index):
    """The address of the status word to pass (None: the library waits and
    returns the data error), and the tensor behind it."""
    if status is None:
        if check:
            return None, None
        status = torch.zeros(1, dtype=torch.int32, device=_DEVICES[index])
        return status.data_ptr(), status
    return _vector(status, torch.int32, status.shape, "status", index), status


def quantize_rows(x, *, status=None, check=True):
    """Rows of ``x`` [rows, cols] (fp32, bf16 or fp16) as 8-bit integers with a scale each.

    Returns (codes int8 [rows, cols], scale fp32 [rows]) with
    scale = max|row| * (1/127) and code = the integer nearest to value / scale
    (halves to even).  A weight's rows are its output channels, so this also
    makes the weight of the products below.  A row with a NaN or an infinity is
    reported (IQ_ERR_NONFINITE) and written as zeros.
    """
    index, ldx = _first(x, "x")
    rows, cols = x.shape
    word, status = _status(status, check, index)
    device = _DEVICES[index]
    q = torch.empty((rows, cols), dtype=torch.int8, device=device)
    scale = torch.empty((rows,), dtype=torch.float32, device=device)
    code = iq.load().iq_quantize_rows(
        _DTYPES[x.dtype], x.data_ptr(), ldx, rows, cols, q.data_ptr(), cols, scale.data_ptr(),
        word, _stream(index))
    iq._check(code, "iq_quantize_rows")
    iq._raise_on_status(status, check, "iq_quantize_rows")
    return q, scale


def int8_matmul(x, x_scale, w, w_scale, *, dtype=torch.bfloat16, out=None):
    """``(x @ w.T) * x_scale[:, None] * w_scale`` in 8-bit integers.

    ``x`` int8 [tokens, depth] with ``x_scale`` fp32 [tokens], ``w`` int8
    [channels, depth] with ``w_scale`` fp32 [channels] (both as
    ``quantize_rows`` gives them).  The sums are exact.  Returns
    [tokens, channels] in ``dtype`` (or in the type of ``out``).
    """
    index, ldx = _first(x, "x", torch.int8)
    ldw = _matrix(w, "w", index, torch.int8)
    tokens, depth = x.shape
    channels, w_depth = w.shape
    if w_depth != depth:
        raise ValueError("w must be [channels, %d]" % depth)
    xs = _vector(x_scale, torch.float32, (tokens,), "x_scale", index)
    ws = _vector(w_scale, torch.float32, (channels,), "w_scale", index)
    if out is not None:
        dtype = out.dtype
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % (dtype,))
    y, ldy = _output(out, tokens, channels, dtype, index, "out")
    code = iq.load().iq_int8_matmul(
        x.data_ptr(), ldx, xs, w.data_ptr(), ldw, ws, tokens, channels, depth, _DTYPES[dtype],
        y.data_ptr(), ldy, _stream(index))
    iq._check(code, "iq_int8_matmul")
    return y


def int8_linear(x, w, w_scale, *, out=None, status=None, check=True):
    """A layer served in 8-bit integers: ``int8_matmul(*quantize_rows(x), w, w_scale)``.

    ``x`` [tokens, depth] in fp32, bf16 or fp16; the result [tokens, channels]
    has its type.  A token with a NaN or an infinity is reported
    (IQ_ERR_NONFINITE) and answered with zeros.
    """
    index, ldx = _first(x, "x")
    ldw = _matrix(w, "w", index, torch.int8)
    tokens, depth = x.shape
    channels, w_depth = w.shape
    if w_depth != depth:
        raise ValueError("w must be [channels, %d]" % depth)
    ws = _vector(w_scale, torch.float32, (channels,), "w_scale", index)
    y, ldy = _output(out, tokens, channels, x, index, "out")
    word, status = _status(status, check, index)
    L = iq.load()
    need, work, space = L.iq_int8_linear_workspace(tokens, depth), None, None
    if need:
        work = torch.empty((need,), dtype=torch.uint8, device=_DEVICES[index])
        space = work.data_ptr()
    code = L.iq_int8_linear(
        _DTYPES[x.dtype], x.data_ptr(), ldx, w.data_ptr(), ldw, ws, tokens, channels, depth,
        y.data_ptr(), ldy, space, need, word, _stream(index))
    iq._check(code, "iq_int8_linear")
    iq._raise_on_status(status, check, "iq_int8_linear")
    return y


def int8_expert_matmul(x, x_scale, w, w_scale, offsets, order=None, *, top_k=1,
                       dtype=torch.bfloat16, out=None):
    """``int8_matmul`` with a weight per expert, on rows in the order of their experts.

    ``w`` int8 [experts, channels, depth] with ``w_scale`` fp32 [experts,
    channels]; ``offsets`` and ``order`` int32 as ``expert_sort`` gives them.
    Row p of the result, offsets[e] <= p < offsets[e+1], is token
    ``order[p] // top_k`` of ``x`` times the weight of expert e; without
    ``order`` it is row p of ``x`` (already dispatched).  Rows of dropped
    choices are zeros.
    """
    index, ldx = _first(x, "x", torch.int8)
    tokens, depth = x.shape
    if not isinstance(w, torch.Tensor) or w.get_device() != index:
        _refuse(w, "w", index)
    if w.dtype != torch.int8:
        raise TypeError("w must be torch.int8, got %s" % (w.dtype,))
    if w.dim() != 3 or w.shape[2] != depth or (w.stride(2) != 1 and depth != 1):
        raise ValueError("w must be [experts, channels, %d] with consecutive values in a row" % depth)
    experts, channels, _ = w.shape
    w_stride, ldw, _ = w.stride()
    xs = _vector(x_scale, torch.float32, (tokens,), "x_scale", index)
    ws = _vector(w_scale, torch.float32, (experts, channels), "w_scale", index)
    ends = _vector(offsets, torch.int32, (experts + 1,), "offsets", index)
    rows, places = tokens, None
    if order is not None:
        rows = tokens * top_k
        places = _vector(order, torch.int32, (rows,), "order", index)
    if out is not None:
        dtype = out.dtype
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % (dtype,))
    y, ldy = _output(out, rows, channels, dtype, index, "out")
    code = iq.load().iq_int8_expert_matmul(
        x.data_ptr(), ldx, xs, tokens, places, top_k, ends, experts, rows, w.data_ptr(), ldw,
        w_stride, ws, channels, depth, _DTYPES[dtype], y.data_ptr(), ldy, _stream(index))
    iq._check(code, "iq_int8_expert_matmul")
    return y


def expert_sort(experts_of, num_experts, *, status=None, check=True):
    """Choices sorted by expert.

    ``experts_of`` [tokens, top_k] int32 or int64: each choice's expert, or -1
    where it was dropped.  Returns int32 tensors: ``order`` [tokens * top_k],
    the choice (token * top_k + slot) at each place; ``position`` [tokens,
    top_k], the place of each choice; ``offsets`` [num_experts + 1], each
    expert's first place.  Equal choices keep their order, dropped ones come
    last, from offsets[num_experts] on.
    """
    index = _on_gpu(experts_of, "experts_of")
    if experts_of.dtype not in _CHOICE_BYTES:
        raise TypeError("experts_of must be int32 or int64, got %s" % (experts_of.dtype,))
    if experts_of.dim() != 2 or not experts_of.is_contiguous():
        raise ValueError("experts_of must be a contiguous [tokens, top_k] tensor")
    tokens, top_k = experts_of.shape
    n, device = tokens * top_k, _DEVICES[index]
    order = torch.empty((n,), dtype=torch.int32, device=device)
    position = torch.empty((tokens, top_k), dtype=torch.int32, device=device)
    offsets = torch.empty((max(num_experts, 0) + 1,), dtype=torch.int32, device=device)
    word, status = _status(status, check, index)
    L = iq.load()
    need, work, space = L.iq_expert_sort_workspace(n, num_experts), None, None
    if need:
        work = torch.empty((need,), dtype=torch.uint8, device=device)
        space = work.data_ptr()
    code = L.iq_expert_sort(
        experts_of.data_ptr(), _CHOICE_BYTES[experts_of.dtype], tokens, top_k, num_experts,
        order.data_ptr(), position.data_ptr(), offsets.data_ptr(), space, need, word,
        _stream(index))
    iq._check(code, "iq_expert_sort")
    iq._raise_on_status(status, check, "iq_expert_sort")
    return order, position, offsets


def _places(t, name, dims, index):
    """The address of a contiguous int32 tensor of that many dimensions on that GPU."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _refuse(t, name, index)
    if t.dtype != torch.int32:
        raise TypeError("%s must be %s, got %s" % (name, torch.int32, t.dtype))
    if t.dim() != dims or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of %d dimensions" % (name, dims))
    return t.data_ptr()


def _route(position, offsets, index):
    """Checks of expert_sort's answers: (tokens, top_k, experts, their addresses)."""
    places, ends = _places(position, "position", 2, index), _places(offsets, "offsets", 1, index)
    tokens, top_k = position.shape
    experts = offsets.shape[0] - 1
    if experts < 1:
        raise ValueError("offsets must be [num_experts + 1]")
    return tokens, top_k, experts, places, ends


def _has_rows(t, name, rows):
    if t.shape[0] != rows:
        raise ValueError("%s must have %d rows" % (name, rows))


def expert_dispatch(x, position, offsets, *, out=None):
    """Tokens copied to the places of their choices: [tokens * top_k, width],
    row position[t, j] holding ``x[t]`` (zeros where the choice was dropped)."""
    index, ldx = _first(x, "x")
    tokens, top_k, experts, places, ends = _route(position, offsets, index)
    _has_rows(x, "x", tokens)
    width = x.shape[1]
    out, ldo = _output(out, tokens * top_k, width, x, index, "out")
    code = iq.load().iq_expert_dispatch(
        _DTYPES[x.dtype], x.data_ptr(), ldx, tokens, width, places, top_k, ends, experts,
        out.data_ptr(), ldo, _stream(index))
    iq._check(code, "iq_expert_dispatch")
    return out


def expert_dispatch_backward(grad, position, offsets, *, out=None):
    """The gradient of ``expert_dispatch``: for the gradient of its result, that
    of ``x``, the sum over each token's kept choices."""
    index, ldg = _first(grad, "grad")
    tokens, top_k, experts, places, ends = _route(position, offsets, index)
    _has_rows(grad, "grad", tokens * top_k)
    width = grad.shape[1]
    out, ldo = _output(out, tokens, width, grad, index, "out")
    code = iq.load().iq_expert_dispatch_backward(
        _DTYPES[grad.dtype], grad.data_ptr(), ldg, tokens, width, places, top_k, ends, experts,
        out.data_ptr(), ldo, _stream(index))
    iq._check(code, "iq_expert_dispatch_backward")
    return out


def expert_combine(y, position, offsets, weights, *, out=None):
    """Rows brought back to their tokens: out[t] = the sum over the kept choices
    j of weights[t, j] * y[position[t, j]] (``weights`` fp32 [tokens, top_k])."""
    index, ldy = _first(y, "y")
    tokens, top_k, experts, places, ends = _route(position, offsets, index)
    _has_rows(y, "y", tokens * top_k)
    width = y.shape[1]
    factors = _vector(weights, torch.float32, position.shape, "weights", index)
    out, ldo = _output(out, tokens, width, y, index, "out")
    code = iq.load().iq_expert_combine(
        _DTYPES[y.dtype], y.data_ptr(), ldy, tokens, width, places, top_k, ends, experts, factors,
        out.data_ptr(), ldo, _stream(index))
    iq._check(code, "iq_expert_combine")
    return out


def expert_combine_backward(grad, y, position, offsets, weights):
    """The gradients of ``expert_combine`` for the gradient ``grad`` [tokens,
    width] of its result: (that of ``y``, that of ``weights``)."""
    index, ldy = _first(y, "y")
    tokens, top_k, experts, places, ends = _route(position, offsets, index)
    _has_rows(y, "y", tokens * top_k)
    width, dtype = y.shape[1], y.dtype
    ldo = _matrix(grad, "grad", index, dtype)
    if grad.shape != (tokens, width):
        raise ValueError("grad must be [%d, %d]" % (tokens, width))
    factors = _vector(weights, torch.float32, position.shape, "weights", index)
    y_grad = y.new_empty((tokens * top_k, width))
    weights_grad = weights.new_empty((tokens, top_k))
    code = iq.load().iq_expert_combine_backward(
        _DTYPES[dtype], grad.data_ptr(), ldo, y.data_ptr(), ldy, tokens, width, places, top_k,
        ends, experts, factors, y_grad.data_ptr(), width, weights_grad.data_ptr(), _stream(index))
    iq._check(code, "iq_expert_combine_backward")
    return y_grad, weights_grad
