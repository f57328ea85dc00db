"""Float64 definitions of a recurrent layer's operators and of the norm of
queries and keys with its rotation: gated linear recurrence, short causal
convolution, and their backward passes.  Plain NumPy, written from the
formulas, token by token; shares no code with the CUDA path.  Sequences are
[N, D] of one batch entry, rows of queries [N, d] of one head."""

from __future__ import annotations

import numpy as np

from oracle.sequence_oracle import rotary64


def sigmoid64(x):
    x = np.asarray(x, np.float64)
    return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def gated_factors64(gate, log_decay=None, scale="norm"):
    """(a, c, log a) of every token and channel."""
    s = sigmoid64(gate)
    log_a = s * np.asarray(log_decay, np.float64) if log_decay is not None else np.log(s)
    less = -np.expm1(log_a) if log_decay is not None else sigmoid64(-np.asarray(gate, np.float64))
    a = np.exp(log_a)
    c = {"norm": np.sqrt(np.maximum(less * (1.0 + a), 0.0)), "mean": less, "none": np.ones_like(a)}[scale]
    return a, c, log_a


def gated64(x, gate, log_decay=None, input_gate=None, state=None, length=None, scale="norm"):
    """(out [N, D], states [length + 1, D]) of h_t = a_t h_{t-1} + c_t u_t."""
    x = np.asarray(x, np.float64)
    n = len(x)
    length = n if length is None else min(max(int(length), 0), n)
    a, c, _ = gated_factors64(gate, log_decay, scale)
    u = x if input_gate is None else x * sigmoid64(input_gate)
    h = np.zeros(x.shape[1]) if state is None else np.asarray(state, np.float64)
    out, states = np.zeros_like(x), np.zeros((length + 1, x.shape[1]))
    states[0] = h
    for t in range(length):
        h = a[t] * h + c[t] * u[t]
        out[t] = states[t + 1] = h
    return out, states


def gated_backward64(x, gate, dout, log_decay=None, input_gate=None, state=None, dstate_out=None, length=None,
                     scale="norm"):
    """Gradients {dx, dgate, dinput_gate, dlog_decay, dstate} of L = sum(dout out) + sum(dstate_out state_out)."""
    x = np.asarray(x, np.float64)
    _, states = gated64(x, gate, log_decay, input_gate, state, length, scale)
    n, (a, c, _) = len(states) - 1, gated_factors64(gate, log_decay, scale)
    s, q = sigmoid64(gate), sigmoid64(input_gate) if input_gate is not None else np.ones_like(x)
    rest = sigmoid64(-np.asarray(input_gate, np.float64)) if input_gate is not None else np.zeros_like(x)
    res = {k: np.zeros_like(x) for k in ("dx", "dgate", "dinput_gate")}
    res["dlog_decay"] = np.zeros(x.shape[1])
    g = np.zeros(x.shape[1]) if dstate_out is None else np.asarray(dstate_out, np.float64)
    for t in reversed(range(n)):
        g = g + np.asarray(dout[t], np.float64)  # dL/dh_t
        if scale == "norm":
            with np.errstate(divide="ignore", invalid="ignore"):
                dc = np.where(c[t] > 0, -a[t] ** 2 / c[t], 0.0)
        else:
            dc = -a[t] if scale == "mean" else 0.0
        dlog = g * (a[t] * states[t] + x[t] * q[t] * dc)
        if log_decay is not None:
            res["dgate"][t] = dlog * np.asarray(log_decay, np.float64) * s[t] * sigmoid64(-np.asarray(gate[t], np.float64))
            res["dlog_decay"] += dlog * s[t]
        else:
            res["dgate"][t] = dlog * sigmoid64(-np.asarray(gate[t], np.float64))
        res["dx"][t] = g * c[t] * q[t]
        res["dinput_gate"][t] = g * c[t] * x[t] * q[t] * rest[t]
        g = a[t] * g
    res["dstate"] = g
    return res


def qknorm64(x, positions, freq, weight=None, eps=1e-6, amplitude=1.0, style="half"):
    """Rows [N, d]: the root-mean-square norm, the weight, the rotation."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    return rotary64(y, positions, freq, amplitude, style)


def qknorm_backward64(dy, x, positions, freq, weight=None, eps=1e-6, amplitude=1.0, style="half"):
    """(dx [N, d], dweight [d])."""
    x = np.asarray(x, np.float64)
    t = rotary64(dy, positions, freq, amplitude, style, transpose=True)
    size = np.sqrt((x * x).mean(1, keepdims=True) + eps)
    g = t if weight is None else t * np.asarray(weight, np.float64)
    dx = g / size - x * (g * x).mean(1, keepdims=True) / size ** 3
    return dx, (t * x / size).sum(0)


def shortconv64(x, weight, bias=None, state=None, length=None, activation="none"):
    """(out [N, D], state_out [K - 1, D], z [length, D])."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    n, taps = len(x), weight.shape[1]
    length = n if length is None else min(max(int(length), 0), n)
    before = np.zeros((taps - 1, x.shape[1])) if state is None else np.asarray(state, np.float64)
    rows = np.concatenate([before, x[:length]])
    z = np.zeros((length, x.shape[1]))
    for t in range(length):
        for j in range(taps):
            z[t] += weight[:, j] * rows[t + j]
        if bias is not None:
            z[t] += np.asarray(bias, np.float64)
    out = np.zeros_like(x)
    out[:length] = z * sigmoid64(z) if activation == "silu" else z
    return out, rows[length:], z


def shortconv_backward64(x, weight, dout, bias=None, state=None, dstate_out=None, length=None, activation="none"):
    """Gradients {dx, dweight, dbias, dstate}."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    _, _, z = shortconv64(x, weight, bias, state, length, activation)
    n, taps = len(z), weight.shape[1]
    before = np.zeros((taps - 1, x.shape[1])) if state is None else np.asarray(state, np.float64)
    rows = np.concatenate([before, x[:n]])
    dz = np.asarray(dout, np.float64)[:n]
    if activation == "silu":
        s = sigmoid64(z)
        dz = dz * (s + z * s * (1.0 - s))
    drows, dweight = np.zeros_like(rows), np.zeros_like(weight)
    for t in range(n):
        for j in range(taps):
            drows[t + j] += dz[t] * weight[:, j]
            dweight[:, j] += dz[t] * rows[t + j]
    if dstate_out is not None:
        drows[n:] += np.asarray(dstate_out, np.float64)
    dx = np.zeros_like(x)
    dx[:n] = drows[taps - 1:]
    return {"dx": dx, "dweight": dweight, "dbias": dz.sum(0), "dstate": drows[: taps - 1]}
