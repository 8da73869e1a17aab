"""Plain implementations of the 4-bit weights and the router in 64 bits (numpy),
and the rounding bounds that the kernels' answers are held to."""

import numpy as np
import torch

from tests.layers_ref import ROUND, TINY

U = 2.0 ** -24                        # half a step of fp32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EVEN = np.array([0, 2, 4, 6])


def quantize(x):
    """(codes of each value, scale byte of each group): every code tried, the nearest
    taken, the even one of two equally near."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    g = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(g).all(axis=2)
    g = np.where(bad[:, :, None], 0.0, g)
    top = np.abs(g).max(axis=2)
    _, e = np.frexp(top)                                  # top = m 2^e, 1/2 <= m < 1
    s = np.where(top > 0, np.clip(e - 1 - 2, -127, 127), -127)
    v = np.abs(g) / np.ldexp(1.0, s)[:, :, None]
    # ties to the even code: its distance counts as a little less
    away = np.abs(v[..., None] - MAGNITUDES)
    least = away.min(axis=3, keepdims=True)
    near = away == least
    pick = np.where(near[..., EVEN].any(axis=3), EVEN[near[..., EVEN].argmax(axis=3)], near.argmax(axis=3))
    code = pick + 8 * (np.signbit(g) & ~bad[:, :, None])
    return code.reshape(rows, cols).astype(np.uint8), (s + 127).astype(np.uint8)


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)


def values(packed, scale):
    """In fp32's range: infinite from 2^128 on, NaN for the scale byte 255."""
    code = unpack(np.asarray(packed)).astype(np.int64)
    v = MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.repeat(np.asarray(scale).astype(np.int64), 32, axis=-1)
    with np.errstate(over="ignore", invalid="ignore"):
        v = v * np.ldexp(1.0, s - 127)
        v = np.where(np.abs(v) >= 2.0 ** 128, np.sign(v) * np.inf, v)
    return np.where(s == 255, np.nan, v)


def product(x, w):
    """The product and the sum of its terms' magnitudes."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def product_bound(y, size, depth, dtype):
    """Exact products of at most three parts whose magnitudes add up to at most
    (1 + 2^-6) of the term's (each part is below 2^-7 of the one before); any order of
    their additions in fp32, each within one step (the rounding inside the matrix
    instructions is not specified); one rounding to dtype."""
    parts = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}[dtype]
    return np.abs(y) * ROUND[dtype] + size * (parts * depth + 8) * 2 * U * (1 + 2.0 ** -6) + 2 * TINY[dtype]


def softmax(l):
    """Rows of probabilities, zeros where no logit is finite; whether a row is live."""
    l = np.asarray(l, np.float64)
    bad = np.isnan(l).any(axis=1) | (l == np.inf).any(axis=1)
    l = np.where(bad[:, None], -np.inf, l)
    top = l.max(axis=1, keepdims=True)
    live = top[:, 0] > -np.inf
    with np.errstate(invalid="ignore"):
        e = np.where(live[:, None], np.exp(l - top), 0.0)
    return e / np.where(live, e.sum(axis=1), 1.0)[:, None], live


def gate(l, top_k, renormalize):
    p, live = softmax(l)
    l = np.where(live[:, None], np.asarray(l, np.float64), -np.inf) + 0.0
    order = np.argsort(-l, axis=1, kind="stable")[:, :top_k]
    kept = np.take_along_axis(l, order, 1) > -np.inf
    w = np.where(kept, np.take_along_axis(p, order, 1), 0.0)
    if renormalize:
        w = w / np.where(kept.any(axis=1), w.sum(axis=1), 1.0)[:, None]
    return np.where(kept, order, -1).astype(np.int32), w


def softmax_error(l):
    """Relative error of a probability in fp32, for each row: l - top is rounded once, so its
    exponential is off by up to |l - top| U, plus two steps for the exponential itself (the
    device library's bound), both in the numerator and in the sum; the sum of n terms in
    any order (n - 1) U; the quotient, or a reciprocal and a product, 2 U.  Terms below
    2^-126 are covered by the absolute part of the bounds."""
    l = np.asarray(l, np.float64)
    fin = np.isfinite(l)
    top = np.where(fin, l, -np.inf).max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        far = np.where(fin, np.minimum(top - l, 104.0), 0.0).max(axis=1)
    return (2 * (far + 4) + l.shape[1] + 3) * U * (1 + 2.0 ** -7)


def gate_backward(grad, l, choice, weights, renormalize):
    """(gradient, bound without the final rounding)."""
    t, k = choice.shape
    g, w = np.asarray(grad, np.float64), np.asarray(weights, np.float64)
    kept = (choice >= 0) & (choice < l.shape[1])
    gw = np.where(kept, g * w, 0.0)
    s, size = gw.sum(axis=1, keepdims=True), np.abs(gw).sum(axis=1, keepdims=True)
    part = np.where(kept, w * (g - s) if renormalize else gw, 0.0)
    # g - s: s is off by (k + 1) U size, the difference by one rounding, the product by one
    off = np.where(kept, np.abs(w) * (size * (k + 2) + 2 * np.abs(g - s)) if renormalize else np.abs(gw), 0.0) * U
    out, bound, many = np.zeros(l.shape), np.zeros(l.shape), np.zeros(l.shape)
    for i in range(t):
        for j in range(k):
            if kept[i, j]:
                out[i, choice[i, j]] += part[i, j]
                bound[i, choice[i, j]] += off[i, j]
                many[i, choice[i, j]] += np.abs(part[i, j])
    if not renormalize:
        p, _ = softmax(l)
        out -= p * s
        bound += p * size * (softmax_error(l)[:, None] + (k + 3) * U)
        many += p * np.abs(s)
    # sums of up to k + 1 terms
    return out, (bound + many * (k + 1) * U) * (1 + 2.0 ** -7) + 2.0 ** -120


def balance(l, choice):
    """(loss, counts, live tokens)."""
    p, live = softmax(l)
    e = l.shape[1]
    counts = np.array([(choice == i).sum() for i in range(e)])
    n, c = int(live.sum()), int(counts.sum())
    loss = e * (counts / c * p.sum(axis=0) / n).sum() if n and c else 0.0
    return loss, counts, n


def balance_bound(loss, l):
    """Positive terms only, so relative errors carry over: the probabilities', up to 32
    additions and a rounding in fp32, the rest in 64 bits, one rounding at the end."""
    return loss * (softmax_error(l).max(initial=0.0) + 35 * U) + 2.0 ** -120


def balance_backward(grad, l, counts, n):
    """(gradient, bound without the final rounding)."""
    p, live = softmax(l)
    e, c = l.shape[1], counts.sum()
    share = counts / c if c else counts * 0.0
    factor = float(grad) * e / n if n else 0.0
    mean = (p * share).sum(axis=1, keepdims=True)
    out = p * (share - mean) * factor
    rel = softmax_error(l)[:, None]
    # share: a reciprocal and a product; mean: the probabilities', the products and e terms
    off = (share + mean) * (e + 6) * U + mean * rel
    return out, (p * np.abs(factor) * off + np.abs(out) * (rel + 8 * U)) * (1 + 2.0 ** -7) + 2.0 ** -120
