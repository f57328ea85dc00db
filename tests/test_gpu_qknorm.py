"""Normalised and rotated queries and keys on the GPU against float64.

An entry of y is a sum of two products with sines off by 4 * 2^-24, rstd (the
sum of d squares in a tree over lanes: at most d / 4 + 8 roundings of its
terms, an approximate root of 2^-22), the weight and a few roundings: with
d <= 256, 80 * 2^-24 of the pair's magnitude.  A gradient adds the sum of g xh,
as many roundings of the sum of magnitudes.  A result is rounded once, 2^-8 for
bf16."""

import numpy as np
import pytest
import torch

from oracle import recurrent_oracle as ro
from oracle import sequence_oracle as sq
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = 2.0 ** -24


def make(shape, dtype, seed, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale + shift).to(DT[dtype]).cuda()


def f64(t):
    return t.cpu().double().numpy()


def pairs(size, half, amp, style):
    """Magnitudes of the pairs that entries belong to."""
    out = size.copy()
    a, b = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    out[:, a] = out[:, b] = amp * (size[:, a] + size[:, b])
    return out


def near(got, want, slack, dtype):
    bad = np.abs(got - want) > slack + (2.0 ** -8 if dtype == "bf16" else STEP) * np.abs(want) + 1e-30
    assert not bad.any(), (np.abs(got - want)[bad].max(), np.argwhere(bad)[:4].tolist())


def rows(t, i, j, layout):
    return f64(t[i, j] if layout == "bhnd" else t[i, :, j])


SHAPES = [(1, 1, 1, 1, 64, 64), (2, 3, 4, 2, 64, 64), (3, 17, 5, 1, 128, 64), (1, 9, 2, 2, 16, 2), (2, 5, 3, 3, 48, 22),
          (1, 1031, 2, 1, 32, 32), (2, 4, 1, 2, 80, 80), (1, 3, 1, 1, 256, 256), (5, 2, 7, 7, 96, 40), (1, 2, 2, 1, 20, 12),
          (2, 130, 9, 3, 128, 128), (1, 2, 1, 1, 2, 2), (1, 5, 2, 3, 254, 252)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("weight", ["own", "f32", None])
@pytest.mark.parametrize("b,n,h,hk,d,rot", SHAPES)
def test_qknorm(b, n, h, hk, d, rot, weight, layout, style, dtype):
    shape = lambda heads: (b, heads, n, d) if layout == "bhnd" else (b, n, heads, d)  # noqa: E731
    x = [make(shape(h), dtype, 1, 1.5), make(shape(hk), dtype, 2, 0.1)]
    dy = [make(shape(h), dtype, 3), make(shape(hk), dtype, 4)]
    w = [None, None] if weight is None else [make((d,), dtype if weight == "own" else "f32", 5 + i, 0.3, 1.0) for i in (0, 1)]
    plan = mb.mhla_rotary_plan(rot)
    freq, amp = sq.rotary_frequencies64(rot)
    pos = torch.randint(-1000, 1 << 20, (b, n), generator=torch.Generator().manual_seed(3))
    kw = dict(q_weight=w[0], k_weight=w[1], eps=1e-5, positions=pos.cuda(), style=style, layout=layout)
    y = mb.mhla_qknorm_forward(*x, plan, **kw)
    grads = mb.mhla_qknorm_backward(*dy, *x, plan, **kw)
    assert grads[2].dtype == grads[3].dtype == torch.float32
    for k, heads in ((0, h), (1, hk)):
        wk = None if w[k] is None else f64(w[k])
        size_w = np.ones(d) if wk is None else np.abs(wk)
        dw, dw_size = np.zeros(d), np.zeros(d)
        for i in range(b):
            for j in range(heads):
                xr, dr, at = rows(x[k], i, j, layout), rows(dy[k], i, j, layout), pos[i].numpy()
                norm = 1 / np.sqrt((xr ** 2).mean(1, keepdims=True) + 1e-5)
                size = pairs(np.abs(xr) * norm * size_w, rot // 2, amp, style)
                near(rows(y[k], i, j, layout), ro.qknorm64(xr, at, freq, wk, 1e-5, amp, style), 80 * STEP * size, dtype)
                dx, one = ro.qknorm_backward64(dr, xr, at, freq, wk, 1e-5, amp, style)
                t = pairs(np.abs(dr), rot // 2, amp, style)
                along = (t * size_w * np.abs(xr) * norm).mean(1, keepdims=True)
                near(rows(grads[k], i, j, layout), dx,
                     80 * STEP * norm * (t * size_w + 2 * np.abs(xr) * norm * along), dtype)
                dw += one
                dw_size += (t * np.abs(xr) * norm).sum(0)
        # terms off by 80 steps, at most b n h / 8 + 64 of them added in a row
        near(f64(grads[2 + k]), dw, (80 + b * n * heads / 8 + 64) * STEP * dw_size, "f32")


def test_without_rotation():
    x, k, w = make((2, 3, 40, 64), "bf16", 1), make((2, 1, 40, 64), "bf16", 2), make((64,), "f32", 3)
    y, ky = mb.mhla_qknorm_forward(x, k, None, q_weight=w)
    z = x.double() * torch.rsqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6) * w.double()
    assert ((y.double() - z).abs() <= (2.0 ** -8 + 80 * STEP) * z.abs()).all()
    same = mb.mhla_qknorm_forward(x, k, mb.mhla_rotary_plan(64), q_weight=w, positions=torch.zeros(40, dtype=torch.int32).cuda())
    # the lanes hold other columns, so the squares add in another order: each is within
    # 80 steps of the exact value before it is rounded, which then differs by a bf16 step at most
    for got, want in ((same[0], y), (same[1], ky)):
        assert ((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs()).all()
    y, none = mb.mhla_qknorm_forward(x, None, None)
    assert none is None
    dq, dk, dw, dkw = mb.mhla_qknorm_backward(y, None, x, None, None)
    assert dk is None and dkw is None and dw.shape == (64,)
    odd = make((1, 2, 3, 33), "f32", 4)  # rows of an odd length, no pairs
    z = odd.double() * torch.rsqrt((odd.double() ** 2).mean(-1, keepdim=True) + 1e-6)
    assert ((mb.mhla_qknorm_forward(odd, None, None)[0].double() - z).abs() <= 80 * STEP * z.abs()).all()


def test_rotation_is_the_rotary_operators():
    """With rows of norm sqrt(d) the two operators agree but for rstd's rounding; offsets and scalings carry over."""
    x = make((2, 4, 33, 64), "f32", 1)
    plan = mb.mhla_rotary_plan(32, base=500000.0, scaling="parts", factor=8.0, original_length=8192)
    normed, _ = mb.mhla_qknorm_forward(x, None, None, eps=0.0)
    want, _ = mb.mhla_rotary_forward(normed, None, plan, offset=70000)
    got, _ = mb.mhla_qknorm_forward(x, None, plan, eps=0.0, offset=70000)
    big = normed.abs() + 1.3 * normed.abs().roll(16, -1) + 1.3 * normed.abs().roll(-16, -1)
    assert ((got - want).abs() <= 8 * STEP * big).all()


def test_zero_rows_and_sizes():
    x = make((1, 2, 4, 64), "f32", 1)
    x[:, :, 1] = 0
    x[:, :, 2] *= 1e-18
    x[:, :, 3] *= 1e15
    y, _ = mb.mhla_qknorm_forward(x, None, None, eps=1e-6)
    z = x.double() * torch.rsqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6)
    assert ((y.double() - z).abs() <= 80 * STEP * z.abs() + 1e-30).all() and (y[:, :, 1] == 0).all()
    dq, _, dw, _ = mb.mhla_qknorm_backward(torch.ones_like(x), None, x, None, None)
    assert torch.isfinite(dq).all() and torch.isfinite(dw).all()


def test_rows_stay_apart():
    """A NaN or an infinity stays in its row, also next to rows that are not there."""
    x = make((1, 3, 5, 64), "bf16", 1)
    want = mb.mhla_qknorm_forward(x, None, None)[0]
    bad = x.clone()
    bad[0, 1, 2, 5], bad[0, 2, 4, 0] = float("nan"), float("inf")
    got = mb.mhla_qknorm_forward(bad, None, None)[0]
    ok = torch.ones(1, 3, 5, dtype=torch.bool)
    ok[0, 1, 2] = ok[0, 2, 4] = False
    assert torch.equal(got[ok.cuda()], want[ok.cuda()])
    assert torch.isnan(got[0, 1, 2]).all()


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("offset", [0, 1, 2, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_in_place(dtype, offset, style):
    b, n, h, d = 2, 33, 3, 64
    fused = make((b, n, 3 * h * d + 8), dtype, 1)
    dfused = make((b, n, 3 * h * d + 8), dtype, 2)
    view = lambda t, i: t[:, :, offset + i * h * d: offset + (i + 1) * h * d].unflatten(2, (h, d))  # noqa: E731
    q, k = view(fused, 0), view(fused, 1)
    dq, dk = view(dfused, 0), view(dfused, 1)
    plan, w = mb.mhla_rotary_plan(32), make((d,), "f32", 3)
    kw = dict(q_weight=w, k_weight=w, offset=100, style=style, layout="bnhd")
    c = lambda t: t.contiguous()  # noqa: E731
    want = mb.mhla_qknorm_forward(c(q), c(k), plan, **kw)
    grads = mb.mhla_qknorm_backward(c(dq), c(dk), c(q), c(k), plan, **kw)
    keep, dkeep = fused.clone(), dfused.clone()
    got = mb.mhla_qknorm_backward(dq, dk, q, k, plan, **kw, dq=dq, dk=dk)
    for a, w_ in zip(got, grads):  # another alignment adds in another order
        assert ((a.float() - w_.float()).abs() <= 2.0 ** -7 * w_.float().abs() + 1e-3).all()
    got = mb.mhla_qknorm_forward(q, k, plan, **kw, q_out=q, k_out=k)
    for a, w_ in zip(got, want):
        assert ((a.float() - w_.float()).abs() <= (2.0 ** -7 if dtype == "bf16" else 2.0 ** -19) * w_.float().abs() + 1e-6).all()
    for t, old in ((fused, keep), (dfused, dkeep)):
        old[:, :, offset: offset + 2 * h * d] = t[:, :, offset: offset + 2 * h * d]
        assert torch.equal(t, old)


def test_gradients_in_place_of_the_inputs():
    q, k, dq, dk = (make((2, 3, 50, 64), "bf16", i) for i in range(4))
    plan = mb.mhla_rotary_plan(64)
    want = mb.mhla_qknorm_backward(dq, dk, q, k, plan)
    got = mb.mhla_qknorm_backward(dq, dk, q, k, plan, dq=q, dk=k)
    assert got[0] is q and all(torch.equal(a, b) for a, b in zip(got, want))


def test_without_the_weights_gradients():
    q, k, dq, dk = (make((2, 3, 50, 64), "bf16", i) for i in range(4))
    want = mb.mhla_qknorm_backward(dq, dk, q, k, None)
    got = mb.mhla_qknorm_backward(dq, dk, q, k, None, params=False)
    assert got[2] is None and got[3] is None and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_empty():
    plan = mb.mhla_rotary_plan(32)
    x = torch.empty(2, 3, 0, 32, device="cuda")
    assert mb.mhla_qknorm_forward(x, x, plan)[0].shape == x.shape
    g = mb.mhla_qknorm_backward(x, x, x, x, plan)
    assert (g[2] == 0).all() and (g[3] == 0).all()
    x, k = torch.empty(2, 0, 4, 32, device="cuda"), make((2, 1, 4, 32), "f32", 1)
    assert mb.mhla_qknorm_forward(x, k, plan)[1].shape == k.shape
    g = mb.mhla_qknorm_backward(x, k, x, k, plan)
    assert (g[2] == 0).all() and not (g[3] == 0).all()


def test_results_do_not_change():
    q, k, dq, dk = (make((3, 5, 3000, 64), "bf16", i) for i in range(4))
    runs = [mb.mhla_qknorm_backward(dq, dk, q, k, mb.mhla_rotary_plan(64)) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_no_device_error_was_reported():
    assert mb.mhla_device_status() == (0, 0)
