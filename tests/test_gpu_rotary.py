"""Rotary positions on the GPU against complex multiplication in float64.

An entry is a product sum of two terms with sines off by 4 * 2^-24 (float32
sincospif and the 32-bit phase) and two roundings in float32, then one rounding
to the output's type: half a step relative, 2^-8 for bf16."""

import numpy as np
import pytest
import torch

from oracle import sequence_oracle as sq
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).cuda()


def f64(t):
    return t.cpu().double().numpy()


def check(got, x, positions, freq, amp, style, transpose, dtype):
    want = sq.rotary64(x, positions, freq, amp, style, transpose)
    half = len(freq)
    size = np.abs(x).copy()  # magnitude of the pair an entry belongs to
    a, b = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    size[:, a] = size[:, b] = amp * (np.abs(x[:, a]) + np.abs(x[:, b]))
    # the oracle's own angle: float64 products of positions below 2^40
    slack = 8 * 2.0 ** -24 * size + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(want) + 1e-30
    assert np.all(np.abs(got - want) <= slack), np.abs(got - want).max()
    np.testing.assert_array_equal(got[:, 2 * half:], x[:, 2 * half:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("b,n,h,hk,d,rot", [
    (1, 1, 1, 1, 64, 64), (2, 3, 4, 2, 64, 64), (3, 17, 5, 1, 128, 64), (1, 9, 2, 2, 16, 2), (2, 5, 3, 3, 48, 22),
    (1, 1031, 2, 1, 32, 32), (2, 4, 1, 2, 80, 80), (1, 3, 1, 1, 256, 256), (5, 2, 7, 7, 96, 40), (1, 2, 2, 1, 20, 12)])
def test_rotary(b, n, h, hk, d, rot, layout, style, dtype):
    shape = lambda heads: (b, heads, n, d) if layout == "bhnd" else (b, n, heads, d)  # noqa: E731
    q, k = make(shape(h), dtype, 1), make(shape(hk), dtype, 2)
    plan = mb.mhla_rotary_plan(rot)
    freq, amp = sq.rotary_frequencies64(rot)
    pos = torch.randint(-1000, 1 << 20, (b, n), generator=torch.Generator().manual_seed(3))
    for transpose, call in ((False, mb.mhla_rotary_forward), (True, mb.mhla_rotary_backward)):
        got = call(q, k, plan, positions=pos.cuda(), style=style, layout=layout)
        for x, y, heads in ((q, got[0], h), (k, got[1], hk)):
            for i in range(b):
                for j in range(heads):
                    at = (i, j) if layout == "bhnd" else (i, slice(None), j)
                    check(f64(y)[at], f64(x)[at], pos[i].numpy(), freq, amp, style, transpose, dtype)


@pytest.mark.parametrize("scaling", ["linear", "base", "parts"])
def test_scalings(scaling):
    x = make((1, 2, 40, 64), "f32", 1)
    plan = mb.mhla_rotary_plan(64, base=500000.0, scaling=scaling, factor=8.0, original_length=8192)
    freq, amp = sq.rotary_frequencies64(64, 500000.0, scaling, 8.0, 8192)
    got, none = mb.mhla_rotary_forward(x, None, plan, offset=65000)
    assert none is None and plan.amplitude == pytest.approx(amp)
    for j in range(2):
        check(f64(got)[0, j], f64(x)[0, j], 65000 + np.arange(40), freq, amp, "half", False, "f32")


def test_far_positions():
    """Positions up to 2^40: the angle keeps float64's accuracy (2^40 2^-53 = 2^-13 of the oracle's own angle)."""
    x = make((1, 1, 64, 32), "f32", 1)
    pos = torch.randint(1 << 39, 1 << 40, (64,), generator=torch.Generator().manual_seed(1))
    got, _ = mb.mhla_rotary_forward(x, None, mb.mhla_rotary_plan(32), positions=pos.cuda())
    want = sq.rotary64(f64(x)[0, 0], pos.numpy(), sq.rotary_frequencies64(32)[0])
    assert np.abs(f64(got)[0, 0] - want).max() <= 2 * 2.0 ** -13 * 2 * np.abs(f64(x)).max()


def test_positions_forms_agree():
    x = make((3, 4, 50, 32), "bf16", 1)
    plan = mb.mhla_rotary_plan(32)
    want, _ = mb.mhla_rotary_forward(x, None, plan, offset=7)
    for pos in (torch.arange(7, 57), torch.arange(7, 57, dtype=torch.int32), torch.arange(7, 57).expand(3, 50),
                torch.arange(7, 57)[None], torch.arange(7, 107)[::1][:50].repeat(3, 1)):
        got, _ = mb.mhla_rotary_forward(x, None, plan, positions=pos.cuda())
        assert torch.equal(got, want)
    wide = torch.arange(7, 107).cuda().repeat_interleave(2)[::2]  # a stride of two
    assert wide.stride(0) == 2
    assert torch.equal(mb.mhla_rotary_forward(x, None, plan, positions=wide[:50])[0], want)


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_in_place_and_streams(dtype, offset, style):
    b, n, h, d = 2, 33, 3, 64
    width = 3 * h * d + 8
    fused = make((b, n, width), dtype, 1)
    q = fused[:, :, offset: offset + h * d].unflatten(2, (h, d))
    k = fused[:, :, offset + h * d: offset + 2 * h * d].unflatten(2, (h, d))
    plan = mb.mhla_rotary_plan(32)
    want = mb.mhla_rotary_forward(q.contiguous(), k.contiguous(), plan, offset=100, style=style, layout="bnhd")
    keep = fused.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mb.mhla_rotary_forward(q, k, plan, offset=100, style=style, layout="bnhd", q_out=q, k_out=k, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and got[0] is q
    keep[:, :, offset: offset + 2 * h * d] = fused[:, :, offset: offset + 2 * h * d]
    assert torch.equal(keep, fused)


def test_empty():
    plan = mb.mhla_rotary_plan(32)
    x = torch.empty(2, 3, 0, 32, device="cuda")
    assert mb.mhla_rotary_forward(x, x, plan)[0].shape == x.shape
    x = torch.empty(2, 0, 4, 32, device="cuda")
    k = make((2, 1, 4, 32), "f32", 1)
    assert mb.mhla_rotary_forward(x, k, plan)[1].shape == k.shape
