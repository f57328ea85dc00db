"""Channels that forget fast and gates that are nearly closed or open: every result
relative to its own size, as float32 holds it.

With S = 2^-24 and |gate| below 43, errors relative to the value are:
sigma and 1 - sigma  k = (1.25 |gate| + 16) S: the argument times log2 e (1.22 S of
                     it), an approximate power (4), sum, reciprocal (2), products;
a                    ra = |log a| (k + 3 S) + 5 S of decays (the exponent's error and
                     the power's), k + S of sigmoids;
1 - a                rm = k + 44 S: where it is small, it is formed by itself, and
                     from a below 0.883, whose 5 S weigh 7.5 times as much there;
c                    rc = rm + 4 S;     u = x sigma(i):  ru = k of i + S;
1 / c                6 S more.
A step of the recurrence and the maps that it goes through round each term six
times at most.  A result is rounded once, half a step, 2^-8 for bf16."""

import numpy as np
import pytest
import torch

from oracle import recurrent_oracle as ro
from test_gpu_gated import COMBOS, STEP, f64, make, near
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu


def spread(shape, low, high, seed, dtype="f32"):
    gen = torch.Generator().manual_seed(seed)
    return (low + (high - low) * torch.rand(*shape, generator=gen)).to(
        torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()


def bounds(x, gate, log_decay, input_gate, state, dout, dstate_out, scale):
    a, c, log_a = ro.gated_factors64(gate, log_decay, scale)
    k = (1.25 * np.abs(gate) + 16) * STEP
    q, rest_i = (1.0, 1.0) if input_gate is None else (ro.sigmoid64(input_gate), ro.sigmoid64(-input_gate))
    ki = 0.0 if input_gate is None else (1.25 * np.abs(input_gate) + 16) * STEP
    ru, u = ki + STEP, np.abs(x) * q
    with np.errstate(invalid="ignore"):
        ra = np.abs(log_a) * (k + 3 * STEP) + 5 * STEP if log_decay is not None else k + STEP
    rc = {"norm": k + 48 * STEP, "mean": k + 48 * STEP, "none": 0 * k}[scale]
    n = len(x)
    eh, mh = np.zeros((n + 1, x.shape[1])), np.zeros((n + 1, x.shape[1]))
    mh[0] = np.abs(state)
    for t in range(n):
        keep, add = a[t] * mh[t], c[t] * u[t]
        eh[t + 1] = a[t] * eh[t] + (ra[t] + 6 * STEP) * keep + (rc[t] + (ru + 0 * u)[t] + 7 * STEP) * add
        mh[t + 1] = keep + add
    res = {name: np.zeros_like(x) for name in ("dx", "dgate", "dinput_gate")}
    res["dlog_decay"] = np.zeros(x.shape[1])
    g, e = np.abs(dstate_out), np.zeros(x.shape[1])
    s, rest = ro.sigmoid64(gate), ro.sigmoid64(-gate)
    for t in reversed(range(n)):
        g, e = g + np.abs(dout[t]), e + STEP * (g + np.abs(dout[t]))
        with np.errstate(divide="ignore", invalid="ignore"):
            dc = {"norm": np.where(c[t] > 0, a[t] ** 2 / c[t], 0.0), "mean": a[t], "none": 0 * a[t]}[scale]
        first, second = a[t] * mh[t], u[t] * dc
        both = first + second
        dlog = e * both + g * (a[t] * eh[t] + ra[t] * first
                               + (2 * ra[t] + rc[t] + (ru + 0 * u)[t] + 8 * STEP) * second + 6 * STEP * both)
        slope = rest[t] * (np.abs(log_decay) * s[t] if log_decay is not None else 1.0)
        res["dgate"][t] = slope * (dlog + (2 * k[t] + 4 * STEP) * g * both)
        gc = c[t] * (e + g * (rc[t] + 5 * STEP))
        res["dx"][t] = (q + 0 * u)[t] * (gc + (ki + 0 * u)[t] * c[t] * g)
        res["dinput_gate"][t] = (u * rest_i)[t] * (gc + 2 * (ki + 0 * u)[t] * c[t] * g)
        res["dlog_decay"] += s[t] * (dlog + (k[t] + (12 + n / 64) * STEP) * g * both)
        e = a[t] * e + (ra[t] + 6 * STEP) * a[t] * g
        g = a[t] * g
    res["dstate"] = e
    return eh, res


def check(p, dtype, scale):
    b, n, d = p["x"].shape
    dout, ds = make((b, n, d), 50, dtype), make((b, d), 51)
    out, state, marks = mb.mhla_gated_forward(**p, scale=scale, keep=True)
    grads = mb.mhla_gated_backward(p["x"], p["gate"], dout, p["log_decay"], p["input_gate"], p["state"], ds, marks,
                                   scale=scale)
    got = dict(zip(("dx", "dgate", "dinput_gate", "dlog_decay", "dstate"), grads))
    one = lambda t, i: None if t is None else f64(t[i])  # noqa: E731
    dlog, slack = np.zeros(d), np.zeros(d)
    for i in range(b):
        args = (f64(p["x"][i]), f64(p["gate"][i]), f64(p["log_decay"]), one(p["input_gate"], i), f64(p["state"][i]))
        want, states = ro.gated64(*args, None, scale)
        eh, err = bounds(*args, f64(dout[i]), f64(ds[i]), scale)
        near(f64(out[i]), want, eh[1:], dtype, "out")
        near(f64(state[i]), states[-1], eh[-1], "f32", "state")
        ref = ro.gated_backward64(args[0], args[1], f64(dout[i]), *args[2:], f64(ds[i]), None, scale)
        for name in ("dx", "dgate") + (("dinput_gate",) if args[3] is not None else ()):
            near(f64(got[name][i]), ref[name], err[name], dtype, name)
        near(f64(got["dstate"][i]), ref["dstate"], err["dstate"], "f32", "dstate")
        dlog += ref["dlog_decay"]
        slack += err["dlog_decay"]
    if got["dlog_decay"] is not None:
        near(f64(got["dlog_decay"]), dlog, slack + b * STEP * np.abs(dlog), "f32", "dlog_decay")


def strong(b, n, d, dtype, kind, in_gate, seed=1):
    """Decays of up to e^-20 a token; gates within 30 of sigmoids, input gates within 25."""
    return dict(x=make((b, n, d), seed, dtype),
                gate=make((b, n, d), seed + 1, dtype, 2.0, 0.5) if kind == "decay" else
                spread((b, n, d), -30.0, 30.0, seed + 1, dtype),
                log_decay=spread((d,), -20.0, -4.0, seed + 2) if kind == "decay" else None,
                input_gate=spread((b, n, d), -25.0, 25.0, seed + 3, dtype) if in_gate else None,
                state=make((b, d), seed + 4))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,scale,in_gate", COMBOS)
@pytest.mark.parametrize("b,n,d", [(1, 1, 8), (2, 40, 65), (3, 200, 130), (1, 600, 64)])
def test_fast_channels(b, n, d, kind, scale, in_gate, dtype):
    check(strong(b, n, d, dtype, kind, in_gate), dtype, scale)


@pytest.mark.parametrize("kind", ["decay", "sigmoid"])
@pytest.mark.parametrize("n", [1, 2, 3])
def test_states_alone(kind, n):
    """Without inputs the state is the product of the decays."""
    p = strong(4, n, 200, "f32", kind, False)
    p["x"].zero_()
    if kind == "sigmoid":
        p["gate"] = spread((4, n, 200), -20.0, 3.0, 8)
    check(p, "f32", "none")


def test_single_tokens():
    p = strong(5, 1, 300, "f32", "decay", True)
    p["x"].zero_()
    out = mb.mhla_gated_step(p["x"][:, 0], p["gate"][:, 0], p["state"].clone(), p["log_decay"], p["input_gate"][:, 0])
    for i in range(5):
        a, _, log_a = ro.gated_factors64(f64(p["gate"][i, 0]), f64(p["log_decay"]))
        k = (1.25 * np.abs(f64(p["gate"][i, 0])) + 16) * STEP
        want = a * f64(p["state"][i])
        near(f64(out[i]), want, (np.abs(log_a) * (k + 3 * STEP) + 7 * STEP) * np.abs(want), "f32", i)


@pytest.mark.parametrize("scale", ["norm", "mean", "none"])
def test_saturated(scale):
    """Open and closed gates, and channels that keep or forget everything."""
    p = strong(2, 130, 64, "f32", "decay", True)
    p["gate"][:, ::3] = 30.0
    p["gate"][:, 1::3] = -30.0
    p["input_gate"][:, ::2] = 40.0
    p["input_gate"][:, 1::4] = -40.0
    p["log_decay"][:8] = torch.tensor([0.0, -1e-6, -1e-8, -50.0, -500.0, -1e30, -0.125, -0.1250001])
    check(p, "f32", scale)
