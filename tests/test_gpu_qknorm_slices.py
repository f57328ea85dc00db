"""Normalised queries and keys as slices of one fused projection, in place, at every
alignment of their rows, against float64 with the bounds of the operator's own tests."""

import numpy as np
import pytest
import torch

from oracle import recurrent_oracle as ro
from oracle import sequence_oracle as sq
from test_gpu_qknorm import STEP, f64, make, near, pairs
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("h,d,rot", [(3, 64, 32), (5, 48, 48)])
def test_slices(h, d, rot, dtype, offset, style):
    b, n, first = 2, 33, 100
    fused, dfused = (make((b, n, 3 * h * d + 8), dtype, i) for i in (1, 2))
    view = lambda t, i: t[:, :, offset + i * h * d: offset + (i + 1) * h * d].unflatten(2, (h, d))  # noqa: E731
    w = make((d,), "f32", 3, 0.3, 1.0)
    plan = mb.mhla_rotary_plan(rot)
    freq, amp = sq.rotary_frequencies64(rot)
    at, wide, mag = first + np.arange(n), f64(w), np.abs(f64(w))
    x, dy = [f64(view(fused, i)) for i in (0, 1)], [f64(view(dfused, i)) for i in (0, 1)]
    kw = dict(q_weight=w, k_weight=w, offset=first, style=style, layout="bnhd")
    (q, k), (dq, dk) = [view(fused, i) for i in (0, 1)], [view(dfused, i) for i in (0, 1)]
    grads = mb.mhla_qknorm_backward(dq, dk, q, k, plan, **kw, dq=dq, dk=dk)
    out = mb.mhla_qknorm_forward(q, k, plan, **kw, q_out=q, k_out=k)
    for i in (0, 1):
        dw, dw_size = np.zeros(d), np.zeros(d)
        for s in range(b):
            for j in range(h):
                xr, dr = x[i][s, :, j], dy[i][s, :, j]
                norm = 1 / np.sqrt((xr ** 2).mean(1, keepdims=True) + 1e-6)
                size = pairs(np.abs(xr) * norm * mag, rot // 2, amp, style)
                near(f64(out[i][s, :, j]), ro.qknorm64(xr, at, freq, wide, 1e-6, amp, style), 80 * STEP * size, dtype)
                dx, one = ro.qknorm_backward64(dr, xr, at, freq, wide, 1e-6, amp, style)
                t = pairs(np.abs(dr), rot // 2, amp, style)
                along = (t * mag * np.abs(xr) * norm).mean(1, keepdims=True)
                near(f64(grads[i][s, :, j]), dx, 80 * STEP * norm * (t * mag + 2 * np.abs(xr) * norm * along), dtype)
                dw += one
                dw_size += (t * np.abs(xr) * norm).sum(0)
        near(f64(grads[2 + i]), dw, (80 + b * n * h / 8 + 64) * STEP * dw_size, "f32")
