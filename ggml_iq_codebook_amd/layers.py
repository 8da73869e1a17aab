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


def _matrix(t, name, dtype=None):
    """A two-dimensional GPU tensor with consecutive values in a row; its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    if dtype is None:
        if t.dtype not in _DTYPES:
            raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, t.dtype))
    elif t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 2:
        raise ValueError("%s must have two dimensions" % name)
    stride, step = t.stride()
    if step != 1 and t.shape[1] != 1:
        raise ValueError("%s must have consecutive values in a row" % name)
    return stride


def _vector(t, dtype, shape, name):
    """A contiguous GPU tensor of the given shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of shape %s" % (name, tuple(shape)))


def _same_device(first, *others):
    """Kernels are launched on the current device, which has to hold every tensor."""
    index = first.device.index
    for t in others:
        if t is not None and t.device.index != index:
            raise ValueError("all tensors must be on one GPU")
    if index != torch.cuda.current_device():
        raise ValueError("the tensors are on cuda:%d, which is not the current device" % index)
    return index


# The current stream's handle, without the Stream object that
# torch.cuda.current_stream builds around it (1.1 us a call).
_stream = torch._C._cuda_getCurrentRawStream


def _output(out, rows, cols, dtype, device, name):
    if out is None:
        return torch.empty((rows, cols), dtype=dtype, device=device), cols
    stride = _matrix(out, name, dtype)
    if out.shape != (rows, cols):
        raise ValueError("%s must be [%d, %d]" % (name, rows, cols))
    return out, stride


def quantize_rows(x, *, status=None, check=True):
    """Rows of ``x`` [rows, cols] (fp32, bf16 or fp16) as 8-bit integers with a scale each.

    Returns (codes int8 [rows, cols], scale fp32 [rows]) with
    scale = max|row| * (1/127) and code = the integer nearest to value / scale
    (halves to even).  A weight's rows are its output channels, so this also
    makes the weight of the products below.  A row with a NaN or an infinity is
    reported (IQ_ERR_NONFINITE) and written as zeros.
    """
    ldx = _matrix(x, "x")
    rows, cols = x.shape
    index = _same_device(x, status)
    q = torch.empty((rows, cols), dtype=torch.int8, device=x.device)
    scale = torch.empty((rows,), dtype=torch.float32, device=x.device)
    status = iq._status_arg(status, check, x.device)
    code = iq.load().iq_quantize_rows(
        _DTYPES[x.dtype], x.data_ptr(), ldx, rows, cols, q.data_ptr(), cols, scale.data_ptr(),
        None if status is None else status.data_ptr(), _stream(index))
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
    ldx, ldw = _matrix(x, "x", torch.int8), _matrix(w, "w", torch.int8)
    tokens, depth = x.shape
    channels = w.shape[0]
    if w.shape[1] != depth:
        raise ValueError("w must be [channels, %d]" % depth)
    _vector(x_scale, torch.float32, (tokens,), "x_scale")
    _vector(w_scale, torch.float32, (channels,), "w_scale")
    dtype = dtype if out is None else out.dtype
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % (dtype,))
    index = _same_device(x, x_scale, w, w_scale, out)
    y, ldy = _output(out, tokens, channels, dtype, x.device, "out")
    code = iq.load().iq_int8_matmul(
        x.data_ptr(), ldx, x_scale.data_ptr(), w.data_ptr(), ldw, w_scale.data_ptr(), tokens,
        channels, depth, _DTYPES[dtype], y.data_ptr(), ldy, _stream(index))
    iq._check(code, "iq_int8_matmul")
    return y


def int8_linear(x, w, w_scale, *, out=None, status=None, check=True):
    """A layer served in 8-bit integers: ``int8_matmul(*quantize_rows(x), w, w_scale)``.

    ``x`` [tokens, depth] in fp32, bf16 or fp16; the result [tokens, channels]
    has its type.  A token with a NaN or an infinity is reported
    (IQ_ERR_NONFINITE) and answered with zeros.
    """
    ldx, ldw = _matrix(x, "x"), _matrix(w, "w", torch.int8)
    tokens, depth = x.shape
    channels = w.shape[0]
    if w.shape[1] != depth:
        raise ValueError("w must be [channels, %d]" % depth)
    _vector(w_scale, torch.float32, (channels,), "w_scale")
    index = _same_device(x, w, w_scale, out, status)
    y, ldy = _output(out, tokens, channels, x.dtype, x.device, "out")
    L = iq.load()
    need = L.iq_int8_linear_workspace(tokens, depth)
    work = torch.empty((need,), dtype=torch.uint8, device=x.device) if need else None
    status = iq._status_arg(status, check, x.device)
    code = L.iq_int8_linear(
        _DTYPES[x.dtype], x.data_ptr(), ldx, w.data_ptr(), ldw, w_scale.data_ptr(), tokens,
        channels, depth, y.data_ptr(), ldy, None if work is None else work.data_ptr(), need,
        None if status is None else status.data_ptr(), _stream(index))
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
    ldx = _matrix(x, "x", torch.int8)
    tokens, depth = x.shape
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor")
    if not w.is_cuda:
        raise ValueError("w must be on the GPU")
    if w.dtype != torch.int8:
        raise TypeError("w must be torch.int8, got %s" % (w.dtype,))
    if w.dim() != 3 or w.shape[2] != depth or (w.stride(2) != 1 and depth != 1):
        raise ValueError("w must be [experts, channels, %d] with consecutive values in a row" % depth)
    experts, channels, _ = w.shape
    _vector(x_scale, torch.float32, (tokens,), "x_scale")
    _vector(w_scale, torch.float32, (experts, channels), "w_scale")
    _vector(offsets, torch.int32, (experts + 1,), "offsets")
    rows = tokens
    if order is not None:
        _vector(order, torch.int32, (tokens * top_k,), "order")
        rows = tokens * top_k
    dtype = dtype if out is None else out.dtype
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % (dtype,))
    index = _same_device(x, x_scale, w, w_scale, offsets, order, out)
    y, ldy = _output(out, rows, channels, dtype, x.device, "out")
    code = iq.load().iq_int8_expert_matmul(
        x.data_ptr(), ldx, x_scale.data_ptr(), tokens, None if order is None else order.data_ptr(),
        top_k, offsets.data_ptr(), experts, rows, w.data_ptr(), w.stride(1), w.stride(0),
        w_scale.data_ptr(), channels, depth, _DTYPES[dtype], y.data_ptr(), ldy, _stream(index))
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
    if not isinstance(experts_of, torch.Tensor):
        raise TypeError("experts_of must be a torch.Tensor")
    if not experts_of.is_cuda:
        raise ValueError("experts_of must be on the GPU")
    if experts_of.dtype not in (torch.int32, torch.int64):
        raise TypeError("experts_of must be int32 or int64, got %s" % (experts_of.dtype,))
    if experts_of.dim() != 2 or not experts_of.is_contiguous():
        raise ValueError("experts_of must be a contiguous [tokens, top_k] tensor")
    tokens, top_k = experts_of.shape
    n, device = tokens * top_k, experts_of.device
    index = _same_device(experts_of, status)
    order = torch.empty((n,), dtype=torch.int32, device=device)
    position = torch.empty((tokens, top_k), dtype=torch.int32, device=device)
    offsets = torch.empty((max(num_experts, 0) + 1,), dtype=torch.int32, device=device)
    L = iq.load()
    need = L.iq_expert_sort_workspace(n, num_experts)
    work = torch.empty((need,), dtype=torch.uint8, device=device) if need else None
    status = iq._status_arg(status, check, device)
    code = L.iq_expert_sort(
        experts_of.data_ptr(), experts_of.element_size(), tokens, top_k, num_experts,
        order.data_ptr(), position.data_ptr(), offsets.data_ptr(),
        None if work is None else work.data_ptr(), need,
        None if status is None else status.data_ptr(), _stream(index))
    iq._check(code, "iq_expert_sort")
    iq._raise_on_status(status, check, "iq_expert_sort")
    return order, position, offsets


def _route(position, offsets):
    """Checks of expert_sort's answers; returns (tokens, top_k, experts)."""
    if not isinstance(position, torch.Tensor) or position.dim() != 2:
        raise ValueError("position must be [tokens, top_k]")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be [num_experts + 1]")
    _vector(position, torch.int32, position.shape, "position")
    _vector(offsets, torch.int32, offsets.shape, "offsets")
    return position.shape[0], position.shape[1], offsets.shape[0] - 1


def expert_dispatch(x, position, offsets, *, out=None):
    """Tokens copied to the places of their choices: [tokens * top_k, width],
    row position[t, j] holding ``x[t]`` (zeros where the choice was dropped)."""
    ldx = _matrix(x, "x")
    tokens, top_k, experts = _route(position, offsets)
    if x.shape[0] != tokens:
        raise ValueError("x must have %d rows" % tokens)
    width = x.shape[1]
    index = _same_device(x, position, offsets, out)
    out, ldo = _output(out, tokens * top_k, width, x.dtype, x.device, "out")
    code = iq.load().iq_expert_dispatch(
        _DTYPES[x.dtype], x.data_ptr(), ldx, tokens, width, position.data_ptr(), top_k,
        offsets.data_ptr(), experts, out.data_ptr(), ldo, _stream(index))
    iq._check(code, "iq_expert_dispatch")
    return out


def _sorted(t, name, tokens, top_k):
    ld = _matrix(t, name)
    if t.shape[0] != tokens * top_k:
        raise ValueError("%s must have %d rows" % (name, tokens * top_k))
    return ld


def expert_dispatch_backward(grad, position, offsets, *, out=None):
    """The gradient of ``expert_dispatch``: for the gradient of its result, that
    of ``x``, the sum over each token's kept choices."""
    tokens, top_k, experts = _route(position, offsets)
    ldg = _sorted(grad, "grad", tokens, top_k)
    width = grad.shape[1]
    index = _same_device(grad, position, offsets, out)
    out, ldo = _output(out, tokens, width, grad.dtype, grad.device, "out")
    code = iq.load().iq_expert_dispatch_backward(
        _DTYPES[grad.dtype], grad.data_ptr(), ldg, tokens, width, position.data_ptr(), top_k,
        offsets.data_ptr(), experts, out.data_ptr(), ldo, _stream(index))
    iq._check(code, "iq_expert_dispatch_backward")
    return out


def expert_combine(y, position, offsets, weights, *, out=None):
    """Rows brought back to their tokens: out[t] = the sum over the kept choices
    j of weights[t, j] * y[position[t, j]] (``weights`` fp32 [tokens, top_k])."""
    tokens, top_k, experts = _route(position, offsets)
    ldy = _sorted(y, "y", tokens, top_k)
    width = y.shape[1]
    _vector(weights, torch.float32, position.shape, "weights")
    index = _same_device(y, position, offsets, weights, out)
    out, ldo = _output(out, tokens, width, y.dtype, y.device, "out")
    code = iq.load().iq_expert_combine(
        _DTYPES[y.dtype], y.data_ptr(), ldy, tokens, width, position.data_ptr(), top_k,
        offsets.data_ptr(), experts, weights.data_ptr(), out.data_ptr(), ldo, _stream(index))
    iq._check(code, "iq_expert_combine")
    return out


def expert_combine_backward(grad, y, position, offsets, weights):
    """The gradients of ``expert_combine`` for the gradient ``grad`` [tokens,
    width] of its result: (that of ``y``, that of ``weights``)."""
    tokens, top_k, experts = _route(position, offsets)
    ldy = _sorted(y, "y", tokens, top_k)
    width = y.shape[1]
    ldo = _matrix(grad, "grad", y.dtype)
    if grad.shape != (tokens, width):
        raise ValueError("grad must be [%d, %d]" % (tokens, width))
    _vector(weights, torch.float32, position.shape, "weights")
    index = _same_device(y, grad, position, offsets, weights)
    y_grad = torch.empty((tokens * top_k, width), dtype=y.dtype, device=y.device)
    weights_grad = torch.empty((tokens, top_k), dtype=torch.float32, device=y.device)
    code = iq.load().iq_expert_combine_backward(
        _DTYPES[y.dtype], grad.data_ptr(), ldo, y.data_ptr(), ldy, tokens, width,
        position.data_ptr(), top_k, offsets.data_ptr(), experts, weights.data_ptr(),
        y_grad.data_ptr(), width, weights_grad.data_ptr(), _stream(index))
    iq._check(code, "iq_expert_combine_backward")
    return y_grad, weights_grad
