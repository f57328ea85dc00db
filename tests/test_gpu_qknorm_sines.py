"""Sines and cosines of bfloat16 rows where they are nearly zero, so that their own
error shows beside the result's rounding.

A row of size sqrt(d) with one entry meets one sine or cosine.  S = 2^-24: the angle
in half turns below 1 is rounded to S / 2 of a half turn, so pi / 2 S of the angle; the
sine itself, rstd and the products add 8 S of their value.  The result is rounded
once, half a step of bf16 being 2^-8 of it."""

import numpy as np
import pytest
import torch

from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24


def positions():
    """Where sin(p) or cos(p) is below 1 / 500 in size."""
    p = np.arange(1 << 20)
    return p[(np.abs(np.sin(p.astype(np.float64))) < 2e-3) | (np.abs(np.cos(p.astype(np.float64))) < 2e-3)]


@pytest.mark.parametrize("style,d,rot", [("half", 64, 64), ("half", 2, 2), ("half", 96, 2), ("interleaved", 64, 64),
                                         ("interleaved", 128, 34)])
@pytest.mark.parametrize("backward", [False, True])
def test_small_sines(style, d, rot, backward):
    p = positions()
    one, other = (0, rot // 2) if style == "half" else (0, 1)  # of the first pair, which turns by 1 a token
    plan = mb.mhla_rotary_plan(rot)
    row = torch.zeros(1, 1, len(p), d, dtype=torch.bfloat16, device="cuda")
    row[..., other] = 1.0
    kw = dict(eps=0.0, positions=torch.from_numpy(p).cuda(), style=style)
    if not backward:
        got, _ = mb.mhla_qknorm_forward(row, None, plan, **kw)
        sign, size = -1.0, np.sqrt(d)
    else:
        x = torch.zeros_like(row)
        x[..., d - 1] = 1.0
        if d == 2:  # mean(g xh) is not zero there
            pytest.skip("no entry beside the pair")
        got = mb.mhla_qknorm_backward(row, None, x, None, plan, **kw)[0]
        sign, size = 1.0, np.sqrt(d)
    got = got[0, 0].double().cpu().numpy()
    angle = p.astype(np.float64)
    for at, want in ((one, sign * size * np.sin(angle)), (other, size * np.cos(angle))):
        slack = np.pi / 2 * STEP * size + (2.0 ** -8 + 8 * STEP) * np.abs(want)
        bad = np.abs(got[:, at] - want) > slack
        assert not bad.any(), (int(bad.sum()), len(p), (np.abs(got[:, at] - want)[bad] / size).max() / STEP)
