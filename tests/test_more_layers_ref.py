"""CPU checks of the references themselves: the gradients against differences, the
rounding against its definition's own properties."""

import numpy as np
import pytest

from tests import more_layers_ref as ref


def logits(t, e, seed, masked=True):
    rng = np.random.default_rng(seed)
    l = 1.5 * rng.standard_normal((t, e))
    if masked:
        l[1, :] = -np.inf                  # a padded token
        l[:, 2] = -np.inf                  # an expert that is switched off
        l[3, 1:] = -np.inf                 # a token with one expert left
    return l


@pytest.mark.parametrize("renormalize", [True, False])
def test_gate_gradient_against_differences(renormalize):
    l, h = logits(6, 7, 1), 1e-5
    c, w = ref.gate(l, 3, renormalize)
    g = np.random.default_rng(2).standard_normal(w.shape)
    got, _ = ref.gate_backward(g, l, c, w, renormalize)
    for i, e in np.ndindex(l.shape):
        if not np.isfinite(l[i, e]):
            assert got[i, e] == 0
            continue
        side = []
        for d in (h, -h):
            m = l.copy()
            m[i, e] += d
            c2, w2 = ref.gate(m, 3, renormalize)
            assert np.array_equal(c2, c)
            side.append((g * w2).sum())
        assert abs((side[0] - side[1]) / (2 * h) - got[i, e]) < 1e-8


def test_balance_gradient_against_differences():
    l, h = logits(6, 7, 3), 1e-5
    c, _ = ref.gate(l, 3, True)
    _, counts, n = ref.balance(l, c)
    got, _ = ref.balance_backward(0.7, l, counts, n)
    assert n == 5 and counts.sum() == (c >= 0).sum()
    for i, e in np.ndindex(l.shape):
        if not np.isfinite(l[i, e]):
            assert got[i, e] == 0
            continue
        side = []
        for d in (h, -h):
            m = l.copy()
            m[i, e] += d
            side.append(0.7 * ref.balance(m, c)[0])
        assert abs((side[0] - side[1]) / (2 * h) - got[i, e]) < 1e-8


def test_even_use_has_a_loss_of_one():
    l = np.zeros((8, 4))
    c = np.arange(16).reshape(8, 2) % 4
    assert ref.balance(l, c)[0] == 1.0
    l = logits(8, 4, 5, masked=False)
    assert abs(ref.balance(l, c)[0] - 1.0) < 1e-12          # either is enough


def test_rounding_to_groups():
    rng = np.random.default_rng(4)
    x = (0.02 * rng.standard_normal((5, 96))).astype(np.float32)
    x[1, :32] = 0.0
    code, scale = ref.quantize(x)
    v = ref.values(ref.pack(code), scale)
    assert (v[1, :32] == 0).all() and scale[1, 0] == 0
    top = np.abs(x.reshape(5, 3, 32)).max(axis=2)
    s = np.ldexp(1.0, scale.astype(int) - 127)
    live = top > 0
    assert (top[live] >= 4 * s[live]).all() and (top[live] < 8 * s[live]).all()
    # within half a step of the grid, or at its end
    err = np.abs(v - x).reshape(5, 3, 32) / s[:, :, None]
    assert (err <= 2.0).all() and (err[np.abs(x.reshape(5, 3, 32)) <= 6 * s[:, :, None]] <= 1.0).all()
    # what a code stands for is rounded to itself
    again = ref.quantize(v)
    assert np.array_equal(ref.values(ref.pack(again[0]), again[1]), v)


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 32))
    x[0, :8] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    x[0, 8:14] = [-0.25, -0.75, -5.0, 7.0, 7.9, -0.0]
    code, scale = ref.quantize(x)
    assert scale[0, 0] == 127
    assert code[0, :14].tolist() == [6, 0, 2, 2, 4, 4, 6, 6, 8, 10, 14, 7, 7, 8]
