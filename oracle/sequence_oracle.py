"""Float64 definitions of the operators around the attention: linear attention
with a decay for each head, rotary positions and layer norm, with their
backward passes.  Plain NumPy, written from the formulas; shares no code with
the CUDA path.  Sequences are [N, d] of one head."""

from __future__ import annotations

import math

import numpy as np


def decay64(q, k, v, g, state=None, length=None, scale=1.0):
    """(out [N, dv], states [N + 1, dk, dv]): the recurrence
    S_t = e^g S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, token by token.
    states[0] is the incoming state, states[length] the outgoing one."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    n = len(q)
    length = n if length is None else min(max(int(length), 0), n)
    fade = math.exp(g)
    s = np.zeros((k.shape[1], v.shape[1])) if state is None else np.asarray(state, np.float64).copy()
    out = np.zeros((n, v.shape[1]))
    states = np.zeros((length + 1,) + s.shape)
    states[0] = s
    for t in range(length):
        s = fade * s + np.outer(k[t], v[t])
        states[t + 1] = s
        out[t] = scale * (q[t] @ s)
    return out, states


def decay_backward64(q, k, v, g, dout, state=None, dstate_out=None, length=None, scale=1.0):
    """(dq, dk, dv, dstate) of L = sum(dout out) + sum(dstate_out state_out)."""
    q, k, v, dout = (np.asarray(a, np.float64) for a in (q, k, v, dout))
    _, states = decay64(q, k, v, g, state, length, scale)
    n = len(states) - 1
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    r = np.zeros_like(states[0]) if dstate_out is None else np.asarray(dstate_out, np.float64).copy()
    for t in reversed(range(n)):
        dq[t] = scale * (states[t + 1] @ dout[t])
        r = r + scale * np.outer(q[t], dout[t])  # now dL/dS_t
        dk[t] = r @ v[t]
        dv[t] = k[t] @ r
        r = math.exp(g) * r
    return dq, dk, dv, r


def rotary_frequencies64(rot_dim, base=10000.0, scaling="none", factor=1.0, original_length=0.0):
    """(radians per position of each pair, amplitude)."""
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq, amplitude = [], 1.0
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "parts":
            turns = original_length * f / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            f = keep * f + (1.0 - keep) * f / factor
        freq.append(f)
    if scaling == "parts":
        amplitude = 0.1 * math.log(factor) + 1.0
    return np.array(freq), amplitude


def rotary64(x, positions, freq, amplitude=1.0, style="half", transpose=False):
    """x [N, d]: each pair (a, b) times amplitude e^{i position f}, entries
    from 2 len(freq) on copied."""
    x = np.asarray(x, np.float64)
    half = len(freq)
    angle = np.asarray(positions, np.float64)[:, None] * freq
    if transpose:
        angle = -angle
    turn = amplitude * np.exp(1j * angle)
    a, b = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    z = (x[:, a] + 1j * x[:, b]) * turn
    y = x.copy()
    y[:, a], y[:, b] = z.real, z.imag
    return y


def layernorm64(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis of [rows, cols]."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layernorm_backward64(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias) with the given statistics."""
    dy, x, mean, rstd = (np.asarray(a, np.float64) for a in (dy, x, mean, rstd))
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
