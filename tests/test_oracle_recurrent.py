"""The float64 oracles of the recurrent layer and of the normalised queries and
keys: hand values, gradients against differences, and pieces against wholes."""

import numpy as np
import pytest

from oracle import recurrent_oracle as ro
from oracle import sequence_oracle as sq


def differences(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        g[i] = (f(hi) - f(lo)) / (2 * step)
    return g


def draw(seed, *shapes):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(s) for s in shapes]


def test_gated_by_hand():
    # sigma(0) = 1/2: a = exp(-1), c = sqrt(1 - exp(-2)), u = x / 2
    out, states = ro.gated64([[4.0], [0.0]], np.zeros((2, 1)), [-2.0], np.zeros((2, 1)), [1.0])
    h0 = np.exp(-1) + 2 * np.sqrt(1 - np.exp(-2))
    np.testing.assert_allclose(out[:, 0], [h0, np.exp(-1) * h0], rtol=1e-15)
    assert states[0, 0] == 1.0
    out, _ = ro.gated64([[4.0], [8.0]], np.zeros((2, 1)), scale="mean")
    np.testing.assert_allclose(out[:, 0], [2.0, 5.0])
    out, _ = ro.gated64([[4.0], [8.0]], np.zeros((2, 1)), scale="none", length=1)
    np.testing.assert_allclose(out[:, 0], [4.0, 0.0])


@pytest.mark.parametrize("decay", [True, False])
@pytest.mark.parametrize("scale", ["norm", "mean", "none"])
@pytest.mark.parametrize("length", [None, 3, 0])
def test_gated_gradients(decay, scale, length):
    n, d = 5, 3
    x, r, i, do, h, dh = draw(1, (n, d), (n, d), (n, d), (n, d), (d,), (d,))
    g = -np.array([0.05, 0.7, 3.0]) if decay else None

    def loss(x=x, r=r, i=i, h=h, g=g):
        out, states = ro.gated64(x, r, g, i, h, length, scale)
        return (out * do).sum() + (states[-1] * dh).sum()

    got = ro.gated_backward64(x, r, do, g, i, h, dh, length, scale)
    want = {"dx": differences(lambda v: loss(x=v), x), "dgate": differences(lambda v: loss(r=v), r),
            "dinput_gate": differences(lambda v: loss(i=v), i), "dstate": differences(lambda v: loss(h=v), h)}
    if decay:
        want["dlog_decay"] = differences(lambda v: loss(g=v), g)
    for name, w in want.items():
        np.testing.assert_allclose(got[name], w, rtol=1e-6, atol=1e-8, err_msg=name)


def test_gated_in_pieces():
    x, r, h = draw(2, (9, 4), (9, 4), (4,))
    whole, states = ro.gated64(x, r, state=h)
    a, s = ro.gated64(x[:4], r[:4], state=h)
    b, _ = ro.gated64(x[4:], r[4:], state=s[-1])
    np.testing.assert_array_equal(np.concatenate([a, b]), whole)
    np.testing.assert_array_equal(states[1:], whole)


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_qknorm(style):
    n, d = 4, 8
    x, dy, w = draw(3, (n, d), (n, d), (d,))
    freq, _ = sq.rotary_frequencies64(6)
    pos = np.array([0, 3, 17, 1000])
    y = ro.qknorm64(x, pos, freq, w, 1e-3, 1.5, style)
    np.testing.assert_allclose(y[0, 6:], (x[0] / np.sqrt((x[0] ** 2).mean() + 1e-3) * w)[6:])  # not rotated
    np.testing.assert_allclose((y[:, :6] ** 2).sum(1),
                               (1.5 * x / np.sqrt((x ** 2).mean(1) + 1e-3)[:, None] * w)[:, :6].__pow__(2).sum(1))
    loss = lambda x=x, w=w: (ro.qknorm64(x, pos, freq, w, 1e-3, 1.5, style) * dy).sum()  # noqa: E731
    dx, dw = ro.qknorm_backward64(dy, x, pos, freq, w, 1e-3, 1.5, style)
    np.testing.assert_allclose(dx, differences(lambda v: loss(x=v), x), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dw, differences(lambda v: loss(w=v), w), rtol=1e-6, atol=1e-8)


def test_shortconv_by_hand():
    x = np.array([[1.0], [2.0], [3.0]])
    out, state, _ = ro.shortconv64(x, [[10.0, 1.0]], [0.5], [[7.0]])
    np.testing.assert_allclose(out[:, 0], [71.5, 12.5, 23.5])
    assert state[0, 0] == 3.0
    out, state, _ = ro.shortconv64(x, [[10.0, 1.0]], None, [[7.0]], 0)
    assert (out == 0).all() and state[0, 0] == 7.0


@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("activation", ["none", "silu"])
@pytest.mark.parametrize("length", [None, 3, 1, 0])
def test_shortconv_gradients(taps, activation, length):
    n, d = 5, 2
    x, w, b, do, s, ds = draw(4, (n, d), (d, taps), (d,), (n, d), (taps - 1, d), (taps - 1, d))

    def loss(x=x, w=w, b=b, s=s):
        out, state, _ = ro.shortconv64(x, w, b, s, length, activation)
        return (out * do).sum() + (state * ds).sum()

    got = ro.shortconv_backward64(x, w, do, b, s, ds, length, activation)
    for name, want in (("dx", differences(lambda v: loss(x=v), x)), ("dweight", differences(lambda v: loss(w=v), w)),
                       ("dbias", differences(lambda v: loss(b=v), b)), ("dstate", differences(lambda v: loss(s=v), s))):
        np.testing.assert_allclose(got[name], want, rtol=1e-6, atol=1e-8, err_msg=name)
