"""Python binding of the layer operators of libiqcodec.so (``include/iq_layers.h``,
``iq_fp4.h``, ``iq_router.h``):
products in 8-bit integers with a scale per token and per channel and products
with 4-bit weights, dense and with a weight per expert, the router with its
balance loss, and the routing of tokens to experts and back, with gradients.

Like the rest of the binding it only marshals: tensors are checked, results
that were not given are allocated, and the library is called on the current HIP
stream.  That part is compiled (``csrc/binding.cpp``): the small calls of these
operators are bound by the host.  Matrices are two-dimensional with consecutive
values in a row; rows may have a stride of their own (slices of larger tensors
are taken as they are).  All tensors are on the current device.

Calls that may find a data error wait for the GPU and raise it (``check=True``).
With a status word of the caller's and ``check=False`` nothing waits, and the word
can be read later; without a word ``check=False`` clears one that nobody reads.

Autograd: ``expert_gate``, ``expert_balance``, ``expert_dispatch``, its gradient and
``expert_combine`` are functions of the graph like torch's own.  The products and
the other gradients have no gradient: a backward pass that reaches their results
raises.  ``quantize_rows``, ``quantize_groups`` and ``expert_sort`` answer with
integers and scales of them, which are constants.  ``out`` cannot be given where
gradients are recorded.  No operator has a rule for forward mode: a tensor with a
tangent is refused.
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
    """Argument types of the entry points of ``include/iq_layers.h``, ``iq_fp4.h`` and
    ``iq_router.h``."""
    P, i64, i32, c = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    for name, args in {
        "iq_quantize_rows": [c, P, i64, i64, i64, P, i64, P, P, P],
        "iq_int8_matmul": [P, i64, P, P, i64, P, i64, i64, i64, c, P, i64, P],
        "iq_int8_linear": [c, P, i64, P, i64, P, i64, i64, i64, P, i64, P, i64, P, P],
        "iq_int8_expert_matmul": [P, i64, P, i64, P, i32, P, i32, i64, P, i64, i64, P, i64, i64,
                                  c, P, i64, P],
        "iq_quantize_groups": [c, P, i64, i64, i64, P, i64, P, i64, P, P],
        "iq_dequantize_groups": [P, i64, P, i64, i64, i64, c, P, i64, P],
        "iq_fp4_linear": [c, P, i64, P, i64, P, i64, i64, i64, i64, P, i64, P, i64, P],
        "iq_fp4_expert_linear": [c, P, i64, i64, P, i32, P, i32, i64, P, i64, i64, P, i64, i64, i64,
                                 i64, P, i64, P, i64, P],
        "iq_expert_gate": [c, P, i64, i64, i32, i32, i32, P, P, P, P],
        "iq_expert_gate_backward": [c, P, P, i64, i64, i32, P, P, i32, i32, P, i64, P],
        "iq_expert_balance": [c, P, i64, i64, i32, P, i32, i32, P, P, P, P, i64, P, P],
        "iq_expert_balance_backward": [c, P, P, i64, i64, i32, P, P, P, i64, P],
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
                       "iq_fp4_linear_workspace": [c, P, i64, i64, i64, i64],
                       "iq_fp4_expert_linear_workspace": [c, P, i64, i64, i32, i64, i64, i64],
                       "iq_expert_balance_workspace": [i64, i32],
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
# (or one has a tangent, which makes a Function raise)

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


class _Gate(Function):
    # The gradient of renormalized weights does not read the logits: they are not kept.
    @staticmethod
    def forward(ctx, logits, top_k, renormalize, status):
        choice, weights = _binding.expert_gate(logits, top_k, renormalize, status)
        ctx.mark_non_differentiable(choice)
        ctx.save_for_backward(choice, weights, *(() if renormalize else (logits,)))
        ctx.like = logits.shape[1], logits.dtype
        return choice, weights

    @staticmethod
    def backward(ctx, _, grad):
        choice, weights, *kept = ctx.saved_tensors
        experts, dtype = ctx.like
        # (the type and shape alone: one row for all tokens)
        logits = kept[0] if kept else weights.new_empty((1, experts), dtype=dtype).expand(len(weights), experts)
        return expert_gate_backward(grad.contiguous(), logits, choice, weights,
                                    renormalize=not kept), None, None, None


class _Balance(Function):
    @staticmethod
    def forward(ctx, logits, choice, status):
        loss, counts, live = _binding.expert_balance(logits, choice, status)
        ctx.mark_non_differentiable(counts, live)
        ctx.save_for_backward(logits, counts, live)
        return loss, counts, live

    @staticmethod
    def backward(ctx, grad, *_):
        return expert_balance_backward(grad, *ctx.saved_tensors), None, None


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


def quantize_groups(w, *, status=None, check=True):
    """Rows of ``w`` [rows, cols] (fp32, bf16 or fp16, cols a multiple of 32) as 4-bit
    floats, 32 of which share a power of two (the MXFP4 format).

    Returns (codes uint8 [rows, cols / 2], scale uint8 [rows, cols / 32]): the
    scale byte s of a group stands for 2^(s - 127), a quarter of the power of two
    at or below the group's largest magnitude, and a code for a sign and one of 0, 1/2,
    1, 3/2, 2, 3, 4, 6, the nearest to value / scale (halves to the even code, 6
    beyond 6); a byte has two codes, the first one in its low bits.  A group with a
    NaN or an infinity is reported (IQ_ERR_NONFINITE) and written as zeros.
    Autograd takes both results as constants.
    """
    status = _word(status, check, w)
    result = (_binding or _native()).quantize_groups(w, status)
    iq._raise_on_status(status, check, "iq_quantize_groups")
    return result


def dequantize_groups(codes, scale, *, dtype=torch.float32, out=None):
    """What ``quantize_groups`` wrote, as values in ``dtype`` (or in the type of ``out``):
    [rows, cols].  They are exact in fp32 and bf16, rounded in fp16."""
    result = (_binding or _native()).dequantize_groups(codes, scale, dtype, out)
    if result is NotImplemented:
        _no_out(out)                  # codes and scales have no gradient
    return result


def fp4_linear(x, w, w_scale, *, out=None):
    """``x @ values(w, w_scale).T`` with a 4-bit weight as ``quantize_groups`` gives it.

    ``x`` [tokens, depth] in fp32, bf16 or fp16; ``w`` uint8 [channels, depth / 2] and
    ``w_scale`` uint8 [channels, depth / 32].  The products are exact, the sums in
    fp32; the result [tokens, channels] has the type of ``x``.  A NaN or an
    infinity in ``x`` passes to its token's results.
    """
    args = x, w, w_scale, out
    result = (_binding or _native()).fp4_linear(*args)
    if result is NotImplemented:
        _no_out(out)
        result = _NoGradient.apply("fp4_linear", *args)
    return result


def fp4_expert_linear(x, w, w_scale, offsets, order=None, *, top_k=1, out=None):
    """``fp4_linear`` with a weight per expert, on rows in the order of their experts.

    ``w`` uint8 [experts, channels, depth / 2] and ``w_scale`` uint8 [experts, channels,
    depth / 32]; ``offsets`` and ``order`` as for ``int8_expert_matmul``.
    """
    args = x, w, w_scale, offsets, order, top_k, out
    result = (_binding or _native()).fp4_expert_linear(*args)
    if result is NotImplemented:
        _no_out(out)
        result = _NoGradient.apply("fp4_expert_linear", *args)
    return result


def expert_gate(logits, top_k, *, renormalize=True, status=None, check=True):
    """The router's choice: each token's ``top_k`` experts and their weights.

    ``logits`` [tokens, experts] in fp32, bf16 or fp16.  Returns (choice int32 [tokens,
    top_k], weights fp32 [tokens, top_k]): the largest logits' experts, the largest
    first and the lowest expert first among equal ones, with their probabilities
    (softmax over all experts), which ``renormalize`` divides by their sum.  A logit
    of -inf is an expert that is never chosen; where fewer than ``top_k`` are left,
    as for a padded token with nothing but -inf, the last choices are -1 with weight
    0 (``expert_sort`` takes them as dropped).  A token with a NaN or +inf is reported
    (IQ_ERR_NONFINITE) and has no choices.  The weights have a gradient.
    """
    status = _word(status, check, logits)
    args = logits, top_k, renormalize, status
    result = (_binding or _native()).expert_gate(*args)
    if result is NotImplemented:
        result = _Gate.apply(*args)
    iq._raise_on_status(status, check, "iq_expert_gate")
    return result


def expert_gate_backward(grad, logits, choice, weights, *, renormalize=True):
    """The gradient of ``expert_gate``: of ``logits``, for the gradient ``grad`` fp32
    [tokens, top_k] of its weights."""
    args = grad, logits, choice, weights, renormalize
    result = (_binding or _native()).expert_gate_backward(*args)
    if result is NotImplemented:
        result = _NoGradient.apply("expert_gate_backward", *args)
    return result


def expert_balance(logits, choice, *, status=None, check=True):
    """How evenly the experts are used: (loss, counts, live).

    ``logits`` [tokens, experts], ``choice`` [tokens, top_k] int32 or int64, -1 where a
    choice was dropped.  ``counts`` int32 [experts] are the choices of each expert,
    ``live`` the number of tokens with a finite logit (padded tokens have none), and
    the loss, a scalar, experts * sum_e (counts[e] / sum(counts)) * (mean over the live
    tokens of expert e's probability): 1 where either is even.  It has a gradient;
    the counts are constants.  A token with a NaN or +inf is reported
    (IQ_ERR_NONFINITE) and does not count, nor does a choice out of range
    (IQ_ERR_INDEX).
    """
    status = _word(status, check, logits)
    args = logits, choice, status
    result = (_binding or _native()).expert_balance(*args)
    if result is NotImplemented:
        result = _Balance.apply(*args)
    iq._raise_on_status(status, check, "iq_expert_balance")
    return result


def expert_balance_backward(grad, logits, counts, live):
    """The gradient of ``expert_balance``: of ``logits``, for the gradient ``grad`` (fp32,
    one value) of its loss."""
    args = grad, logits, counts, live
    result = (_binding or _native()).expert_balance_backward(*args)
    if result is NotImplemented:
        result = _NoGradient.apply("expert_balance_backward", *args)
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
