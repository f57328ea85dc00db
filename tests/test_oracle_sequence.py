"""Pins of the float64 definitions of the decayed linear attention, the rotary
positions and the layer norm (CPU)."""

import math

import numpy as np
import pytest

from oracle import sequence_oracle as sq


def _inputs(n=11, dk=5, dv=3, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((n, dk)), r.standard_normal((n, dk)), r.standard_normal((n, dv)), \
        r.standard_normal((n, dv)), r.standard_normal((dk, dv)), r.standard_normal((dk, dv))


@pytest.mark.parametrize("g", [0.0, -0.05, -2.0, -math.inf])
def test_decay_recurrence_is_the_masked_matrix(g):
    q, k, v, _, s0, _ = _inputs()
    n = len(q)
    out, states = sq.decay64(q, k, v, g, s0, scale=0.3)
    w = np.array([[math.exp(g) ** (t - j) if t >= j else 0.0 for j in range(n)] for t in range(n)])
    lam = np.array([math.exp(g) ** (t + 1) for t in range(n)])
    np.testing.assert_allclose(out, 0.3 * ((w * (q @ k.T)) @ v + lam[:, None] * (q @ s0)), atol=1e-12)
    np.testing.assert_allclose(states[n], math.exp(g) ** n * s0 + (w[-1][:, None] * k).T @ v, atol=1e-12)


def test_decay_by_hand():
    # S_0 = 0.5 * 2 + 1 * 3 = 4, o_0 = 4 * 1; S_1 = 0.5 * 4 + 2 * 1 = 4, o_1 = 4 * 3
    out, states = sq.decay64([[1.0], [3.0]], [[1.0], [2.0]], [[3.0], [1.0]], math.log(0.5), [[2.0]])
    np.testing.assert_allclose(out[:, 0], [4.0, 12.0])
    assert states[2][0, 0] == pytest.approx(4.0)


@pytest.mark.parametrize("length", [None, 0, 1, 7])
def test_decay_gradients_are_differences(length):
    q, k, v, do, s0, ds = _inputs(seed=1)
    g, scale, h = -0.3, 0.7, 1e-6

    def loss(q, k, v, s0):
        out, states = sq.decay64(q, k, v, g, s0, length, scale)
        return (out * do).sum() + (states[-1] * ds).sum()

    grads = sq.decay_backward64(q, k, v, g, do, s0, ds, length, scale)
    args = [q, k, v, s0]
    for i, got in enumerate(grads):
        want = np.zeros_like(args[i])
        for at in np.ndindex(want.shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[i][at] += h
            down[i][at] -= h
            want[at] = (loss(*up) - loss(*down)) / (2 * h)
        np.testing.assert_allclose(got, want, atol=1e-7)


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_rotary_keeps_relative_positions_and_norms(style):
    r = np.random.default_rng(2)
    x, y = r.standard_normal((1, 12)), r.standard_normal((1, 12))
    freq, amp = sq.rotary_frequencies64(8)
    rot = lambda a, p: sq.rotary64(a, [p], freq, amp, style)  # noqa: E731
    assert (rot(x, 9) * rot(y, 4)).sum() == pytest.approx((rot(x, 105) * rot(y, 100)).sum())
    assert np.linalg.norm(rot(x, 1234)) == pytest.approx(np.linalg.norm(x))
    np.testing.assert_array_equal(rot(x, 5)[:, 8:], x[:, 8:])
    back = sq.rotary64(rot(x, 77), [77], freq, amp, style, transpose=True)
    np.testing.assert_allclose(back, x, atol=1e-12)


def test_rotary_by_hand():
    # one pair, a quarter turn: (1, 0) -> (0, 1)
    y = sq.rotary64([[1.0, 0.0, 5.0]], [1], np.array([math.pi / 2]))
    np.testing.assert_allclose(y, [[0.0, 1.0, 5.0]], atol=1e-15)


def test_rotary_scalings():
    plain, one = sq.rotary_frequencies64(16)
    assert one == 1.0 and plain[0] == 1.0
    np.testing.assert_allclose(sq.rotary_frequencies64(16, scaling="linear", factor=4.0)[0], plain / 4)
    # a larger base keeps the fastest pair and divides the slowest by the factor
    wide = sq.rotary_frequencies64(16, scaling="base", factor=4.0)[0]
    assert wide[0] == plain[0] and wide[-1] == pytest.approx(plain[-1] / 4)
    parts, amp = sq.rotary_frequencies64(16, scaling="parts", factor=4.0, original_length=2048)
    assert parts[0] == plain[0] and parts[-1] == pytest.approx(plain[-1] / 4)
    assert amp == pytest.approx(1 + 0.1 * math.log(4.0))


def test_layernorm_gradients_are_differences():
    r = np.random.default_rng(3)
    x, w, b, dy = r.standard_normal((4, 6)), r.standard_normal(6), r.standard_normal(6), r.standard_normal((4, 6))
    y, mean, rstd = sq.layernorm64(x, w, b)
    np.testing.assert_allclose(((y - b) / w).mean(1), 0, atol=1e-12)
    grads = sq.layernorm_backward64(dy, x, mean, rstd, w)
    h = 1e-6
    for i, got in enumerate(grads):
        want = np.zeros_like(got)
        for at in np.ndindex(want.shape):
            d = [0.0, 0.0]
            for side, sign in enumerate((h, -h)):
                args = [x.copy(), w.copy(), b.copy()]
                args[i][at] += sign
                d[side] = (sq.layernorm64(*args)[0] * dy).sum()
            want[at] = (d[0] - d[1]) / (2 * h)
        np.testing.assert_allclose(got, want, atol=1e-7)
