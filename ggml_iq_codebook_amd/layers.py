"""Python binding of the layer operators of libiqcodec.so (``include/iq_layers.h``):
products in 8-bit integers with a scale per token and per channel, dense and
with a weight per expert, and the routing of tokens to experts and back with
its gradients.

Like the rest of the binding it only marshals: tensors are checked, results
that were not given are allocated, and the library is called on the current HIP
stream.  That part is compiled (``csrc/binding.cpp``): the small calls of these
operators are bound by the host.  Matrices are two-dimensional with consecutive
values in a row; rows may have a stride of their own (slices of larger tensors
are taken as they are).  All tensors are on the current device.

Calls that may find a data error wait for the GPU and raise it (``check=True``).
With a status word of the caller's and ``check=False`` nothing waits, and the word
can be read later; without a word ``check=False`` clears one that nobody reads.

Autograd: ``expert_dispatch``, its gradient and ``expert_combine`` are functions
of the graph like torch's own.  The 8-bit products and ``expert_combine_backward``
have no gradient: a backward pass that reaches their results raises.
``quantize_rows`` and ``expert_sort`` answer with integers and scales of them,
which are constants.  ``out`` cannot be given where gradients are recorded.
"""

from __future__ import annotations

import ctypes
import importlib
import os
import sys

import torch
from torch.autograd import Function

# The package, whose helpers and loaded library the calls below use (it imports
# this module before it defines them).
iq = sys.modules[__package__]

_binding = None


def _native():
    """The compiled part (built first only if it does not exist)."""
    global _binding
    if _binding is None:
        iq.load()
        if not os.path.exists(os.path.join(os.path.dirname(__file__), "_layers.so")):
            from . import build
            build.build_binding()
        module = importlib.import_module("._layers", __package__)
        module.set_error(iq.IQError)
        _binding = module
    return _binding


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
    for name, args in {"iq_int8_linear_workspace": [i64, i64, i64],
                       "iq_expert_sort_workspace": [i64, i32]}.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, i64


def _word(status, check, like):
    """The status word of a call: the caller's; None with ``check``, so that the
    library waits and returns the data error; or a fresh one nobody reads."""
    if status is None and not check and isinstance(like, torch.Tensor):
        return torch.zeros(1, dtype=torch.int32, device=like.device)
    return status


# --- autograd: what the calls below turn to when the binding answers
# NotImplemented, because gradients are being recorded for one of the arguments

def _rows(grad):
    """A gradient as the kernels take it: consecutive values in a row."""
    return grad if grad.stride(1) == 1 else grad.contiguous()


class _Dispatch(Function):
    @staticmethod
    def forward(ctx, x, position, offsets):
        ctx.save_for_backward(position, offsets)
        return _binding.expert_dispatch(x, position, offsets, None)

    @staticmethod
    def backward(ctx, grad):
        return expert_dispatch_backward(_rows(grad), *ctx.saved_tensors), None, None


class _DispatchBackward(Function):
    @staticmethod
    def forward(ctx, grad, position, offsets):
        ctx.save_for_backward(position, offsets)
        return _binding.expert_dispatch_backward(grad, position, offsets, None)

    @staticmethod
    def backward(ctx, grad):
        return expert_dispatch(_rows(grad), *ctx.saved_tensors), None, None


class _Combine(Function):
    @staticmethod
    def forward(ctx, y, position, offsets, weights):
        ctx.save_for_backward(y, position, offsets, weights)
        return _binding.expert_combine(y, position, offsets, weights, None)

    @staticmethod
    def backward(ctx, grad):
        y_grad, weights_grad = expert_combine_backward(_rows(grad), *ctx.saved_tensors)
        return y_grad, None, None, weights_grad


class _NoGradient(Function):
    """A call whose results have a place in the graph, but no gradient beyond."""

    @staticmethod
    def forward(ctx, name, *args):
        ctx.name = name
        return getattr(_binding, name)(*args)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("%s has no gradient; call it under torch.no_grad() or on detached tensors"
                           % ctx.name)


def _no_out(out):
    if out is not None:
        raise ValueError("out cannot be given where gradients are recorded")


def quantize_rows(x, *, status=None, check=True):
    """Rows of ``x`` [rows, cols] (fp32, bf16 or fp16) as 8-bit integers with a scale each.

    Returns (codes int8 [rows, cols], scale fp32 [rows]) with
    scale = max|row| * (1/127) and code = the integer nearest to value / scale
    (halves to even).  A weight's rows are its output channels, so this also
    makes the weight of the products below.  A row with a NaN or an infinity is
    reported (IQ_ERR_NONFINITE) and written as zeros.  Autograd takes both results
    as constants.
    """
    status = _word(status, check, x)
    result = (_binding or _native()).quantize_rows(x, status)
    iq._raise_on_status(status, check, "iq_quantize_rows")
    return result


def int8_matmul(x, x_scale, w, w_scale, *, dtype=torch.bfloat16, out=None):
    """``(x @ w.T) * x_scale[:, None] * w_scale`` in 8-bit integers.

    ``x`` int8 [tokens, depth] with ``x_scale`` fp32 [tokens], ``w`` int8
    [channels, depth] with ``w_scale`` fp32 [channels] (both as
    ``quantize_rows`` gives them).  The sums are exact.  Returns
    [tokens, channels] in ``dtype`` (or in the type of ``out``).
    """
    args = x, x_scale, w, w_scale, dtype, out
    result = (_binding or _native()).int8_matmul(*args)
    if result is NotImplemented:
        _no_out(out)
        result = _NoGradient.apply("int8_matmul", *args)
    return result


def int8_linear(x, w, w_scale, *, out=None, status=None, check=True):
    """A layer served in 8-bit integers: ``int8_matmul(*quantize_rows(x), w, w_scale)``.

    ``x`` [tokens, depth] in fp32, bf16 or fp16; the result [tokens, channels]
    has its type.  A token with a NaN or an infinity is reported
    (IQ_ERR_NONFINITE) and answered with zeros.
    """
    status = _word(status, check, x)
    args = x, w, w_scale, out, status
    result = (_binding or _native()).int8_linear(*args)
    if result is NotImplemented:
        _no_out(out)
        result = _NoGradient.apply("int8_linear", *args)
    iq._raise_on_status(status, check, "iq_int8_linear")
    return result


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
    args = x, x_scale, w, w_scale, offsets, order, top_k, dtype, out
    result = (_binding or _native()).int8_expert_matmul(*args)
    if result is NotImplemented:
        _no_out(out)
        result = _NoGradient.apply("int8_expert_matmul", *args)
    return result


def expert_sort(experts_of, num_experts, *, status=None, check=True):
    """Choices sorted by expert.

    ``experts_of`` [tokens, top_k] int32 or int64: each choice's expert, or -1
    where it was dropped.  Returns int32 tensors: ``order`` [tokens * top_k],
    the choice (token * top_k + slot) at each place; ``position`` [tokens,
    top_k], the place of each choice; ``offsets`` [num_experts + 1], each
    expert's first place.  Equal choices keep their order, dropped ones come
    last, from offsets[num_experts] on.
    """
    status = _word(status, check, experts_of)
    result = (_binding or _native()).expert_sort(experts_of, num_experts, status)
    iq._raise_on_status(status, check, "iq_expert_sort")
    return result


def expert_dispatch(x, position, offsets, *, out=None):
    """Tokens copied to the places of their choices: [tokens * top_k, width],
    row position[t, j] holding ``x[t]`` (zeros where the choice was dropped)."""
    result = (_binding or _native()).expert_dispatch(x, position, offsets, out)
    if result is NotImplemented:
        _no_out(out)
        result = _Dispatch.apply(x, position, offsets)
    return result


def expert_dispatch_backward(grad, position, offsets, *, out=None):
    """The gradient of ``expert_dispatch``: for the gradient of its result, that
    of ``x``, the sum over each token's kept choices."""
    result = (_binding or _native()).expert_dispatch_backward(grad, position, offsets, out)
    if result is NotImplemented:
        _no_out(out)
        result = _DispatchBackward.apply(grad, position, offsets)
    return result


def expert_combine(y, position, offsets, weights, *, out=None):
    """Rows brought back to their tokens: out[t] = the sum over the kept choices
    j of weights[t, j] * y[position[t, j]] (``weights`` fp32 [tokens, top_k])."""
    result = (_binding or _native()).expert_combine(y, position, offsets, weights, out)
    if result is NotImplemented:
        _no_out(out)
        result = _Combine.apply(y, position, offsets, weights)
    return result


def expert_combine_backward(grad, y, position, offsets, weights):
    """The gradients of ``expert_combine`` for the gradient ``grad`` [tokens,
    width] of its result: (that of ``y``, that of ``weights``)."""
    args = grad, y, position, offsets, weights
    result = (_binding or _native()).expert_combine_backward(*args)
    if result is NotImplemented:
        result = _NoGradient.apply("expert_combine_backward", *args)
    return result
