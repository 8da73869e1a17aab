"""Plain implementations of the layer operators in 64 bits (numpy), and the
rounding bounds that the kernels' answers are held to."""

import numpy as np
import torch

# Unit roundoff of each storage type, and half its smallest subnormal.
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def to64(t):
    return t.detach().double().cpu().numpy()


def quantize(x):
    """Codes and scales with every step in numpy's (IEEE) fp32."""
    x = np.asarray(x, np.float32)
    top = np.abs(x).max(axis=1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        scale = (top * (np.float32(1.0) / np.float32(127.0))).astype(np.float32)
        q = np.rint((x / scale[:, None]).astype(np.float32))
    q = np.where(scale[:, None] > 0, q, 0.0)
    bad = ~np.isfinite(x).all(axis=1)
    scale[bad] = 0.0
    q[bad] = 0.0
    return np.clip(q, -127, 127).astype(np.int8), scale


def product(x, x_scale, w, w_scale):
    """Exact integer sums (int64), scaled in fp64."""
    s = x.astype(np.int64) @ w.astype(np.int64).T
    return s.astype(np.float64) * x_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)


def product_bound(y, dtype):
    """The sum's conversion and two products in fp32, then one rounding to dtype."""
    return np.abs(y) * (ROUND[dtype] + 3.5 * 2.0 ** -24) + 2 * TINY[dtype]


def sort(choice, experts):
    flat = choice.reshape(-1)
    key = np.where((flat < 0) | (flat >= experts), experts, flat)
    order = np.argsort(key, kind="stable")
    position = np.empty_like(order)
    position[order] = np.arange(order.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=experts + 1)[:experts])])
    return order.astype(np.int32), position.reshape(choice.shape).astype(np.int32), offsets.astype(np.int32)


def expert_product(x, x_scale, w, w_scale, order, offsets, top_k):
    y = np.zeros((len(order), w.shape[1]))
    for e in range(w.shape[0]):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        tok = order[rows] // top_k
        y[rows] = product(x[tok], x_scale[tok], w[e], w_scale[e])
    return y


def dispatch(x, position, offsets):
    t, k = position.shape
    out = np.zeros((t * k, x.shape[1]))
    for i in range(t):
        for j in range(k):
            if position[i, j] < offsets[-1]:
                out[position[i, j]] = x[i]
    return out


def combine(y, position, offsets, weights):
    """The sum and, for the bound, the sum of its terms' magnitudes."""
    t, k = position.shape
    out, size = np.zeros((t, y.shape[1])), np.zeros((t, y.shape[1]))
    for i in range(t):
        for j in range(k):
            if position[i, j] < offsets[-1]:
                term = weights[i, j] * y[position[i, j]]
                out[i] += term
                size[i] += np.abs(term)
    return out, size


def combine_bound(out, size, top_k, dtype):
    """Each product rounded, then top_k - 1 additions, in fp32; one rounding to dtype."""
    return np.abs(out) * ROUND[dtype] + size * (top_k + 1) * 2.0 ** -24 * (1 + 2.0 ** -7) + 2 * TINY[dtype]


def combine_backward(grad, y, position, offsets, weights):
    """(gradient of y, of the weights, sums of the magnitudes of the latter's terms)."""
    t, k = position.shape
    gy, gw, size = np.zeros(y.shape), np.zeros((t, k)), np.zeros((t, k))
    for i in range(t):
        for j in range(k):
            p = position[i, j]
            if p < offsets[-1]:
                gy[p] = weights[i, j] * grad[i]
                gw[i, j] = np.dot(grad[i], y[p])
                size[i, j] = np.dot(np.abs(grad[i]), np.abs(y[p]))
    return gy, gw, size


def dot_bound(size, n):
    """Any order of n products and n - 1 additions in fp32."""
    return size * (n + 1) * 2.0 ** -24 * (1 + 2.0 ** -7) + 2.0 ** -140
