"""Layer norm on the GPU against float64, forward and backward.

Bounds: a row's sums of c terms are off by at most (c + 4) 2^-24 of the sum of
magnitudes; every result is then a few products in float32 and one rounding to
its type (half a step: 2^-8 for bf16)."""

import numpy as np
import pytest
import torch

from oracle import sequence_oracle as sq
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(shape, dtype, seed, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale + shift).to(DT[dtype]).cuda()


def f64(t):
    return t.cpu().double().numpy()


def check(got, want, slack, what):
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - want) - slack
    assert over.max(initial=-1.0) <= 0, f"{what}: {np.abs(got - want).max():.3e} off, {over.max():.3e} over its bound"


SIZES = [(1, 1), (3, 2), (5, 7), (1, 8), (70, 16), (33, 31), (9, 32), (300, 64), (7, 100), (129, 129), (2, 256),
         (41, 500), (50, 512), (3, 513), (64, 1024), (5, 1151), (2, 2049), (3, 4096), (2, 6000), (3, 8192), (2, 9001),
         (2, 16384), (3, 20000), (1, 32776)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_layernorm(rows, cols, dtype, wdtype):
    x, dy = make((rows, cols), dtype, 1, 2.0, 1.5), make((rows, cols), dtype, 2)
    w, b = make((cols,), wdtype, 3, 0.3, 1.0), make((cols,), wdtype, 4)
    eps = 1e-5
    y, mean, rstd = mb.mhla_layernorm_forward(x, w, b, eps=eps)
    X, W, B = f64(x), f64(w), f64(b)
    want, m, r = sq.layernorm64(X, W, B, eps)
    half = 2.0 ** -8 if dtype == "bf16" else EPS
    e_mean = (cols + 4) * EPS * np.abs(X).mean(1)
    check(f64(mean), m, e_mean, "mean")
    # relative error of the variance: its own sum, and the mean's error twice
    var = ((X - m[:, None]) ** 2).mean(1) + eps
    dev = np.abs(X - m[:, None]).mean(1) + EPS * np.abs(X).max(1)
    e_r = r * ((cols + 8) * EPS + (2 * dev * e_mean + e_mean ** 2) / var)
    check(f64(rstd), r, e_r, "rstd")
    wide = np.abs(W) * (e_mean[:, None] + 4 * EPS * np.abs(X)) * r[:, None] + np.abs(want - B) * (e_r / r + 8 * EPS)[:, None]
    check(f64(y), want, wide + (half + EPS) * np.abs(want) + 4 * EPS * np.abs(B), "y")

    dx, dw, db = mb.mhla_layernorm_backward(dy, x, mean, rstd, weight=w)
    D, M, R = f64(dy), f64(mean), f64(rstd)
    want = sq.layernorm_backward64(D, X, M, R, W)
    xh = (X - M[:, None]) * R[:, None]
    e_xh = 4 * EPS * (np.abs(X) + np.abs(M[:, None])) * R[:, None] + EPS * np.abs(xh)
    g = np.abs(D * W)
    c1, c2 = g.mean(1, keepdims=True), (g * np.abs(xh)).mean(1, keepdims=True)
    slack = R[:, None] * ((cols + 16) * EPS * (g + c1 + np.abs(xh) * c2) + e_xh * c2 + np.abs(xh) * (g * e_xh).mean(1, keepdims=True))
    check(f64(dx), want[0], slack + half * np.abs(want[0]) + 1e-30, "dx")
    check(f64(dw), want[1], (rows + 8) * EPS * np.abs(D * xh).sum(0) + (np.abs(D) * e_xh).sum(0) + 1e-30, "dweight")
    check(f64(db), want[2], (rows + 8) * EPS * np.abs(D).sum(0), "dbias")


@pytest.mark.parametrize("cols", [64, 65, 1024])
def test_many_rows(cols):
    """More rows than one wave of CTAs; the sums do not change from call to call."""
    rows = 20011
    x, dy, w = make((rows, cols), "bf16", 1), make((rows, cols), "bf16", 2), make((cols,), "f32", 3)
    y, mean, rstd = mb.mhla_layernorm_forward(x, w)
    a = mb.mhla_layernorm_backward(dy, x, mean, rstd, weight=w)
    b = mb.mhla_layernorm_backward(dy, x, mean, rstd, weight=w)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    X, D = f64(x), f64(dy)
    want = sq.layernorm_backward64(D, X, f64(mean), f64(rstd), f64(w))
    for got, ref in zip(a[1:], want[1:]):
        # no sum has more than (rows / 152 + 700) terms in a row
        check(f64(got), ref, (rows / 152 + 700) * EPS * (np.abs(D) * 6).sum(0), "sums")
    pick = np.arange(0, rows, 997)
    ref = sq.layernorm64(X[pick], f64(w))[0]
    check(f64(y)[pick], ref, 2.0 ** -8 * np.abs(ref) + (cols + 32) * EPS * 8 * np.abs(f64(w)), "y")


def test_no_affine_and_large_mean():
    x = make((40, 64), "f32", 1, 1.0, 4096.0)
    y, mean, rstd = mb.mhla_layernorm_forward(x)
    want, m, r = sq.layernorm64(f64(x))
    # deviations are exact up to the mean's rounding: 64 terms of 4096
    check(f64(y), want, 68 * EPS * 4097 * r[:, None] * (1 + np.abs(want)) + 80 * EPS * np.abs(want), "y")
    dx, dw, db = mb.mhla_layernorm_backward(x, x, mean, rstd, params=False)
    assert dw is None and db is None and torch.isfinite(dx).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols,pad,offset", [(64, 8, 0), (64, 3, 1), (1024, 64, 8), (20000, 8, 0), (9000, 1, 1)])
def test_strides_in_place(cols, pad, offset, dtype):
    rows = 37
    buf = make((rows, cols + pad), dtype, 1)
    x = buf[:, offset: offset + cols]
    w, b = make((cols,), dtype, 3), make((cols,), dtype, 4)
    dy = make((rows, cols), dtype, 5)
    want, mean, rstd = mb.mhla_layernorm_forward(x.contiguous(), w, b)
    grads = mb.mhla_layernorm_backward(dy, x.contiguous(), mean, rstd, weight=w)
    # another path (scalar loads, another split of the sums) may round otherwise
    near = lambda s, t: torch.testing.assert_close(s, t, rtol=2.0 ** -7 if dtype == "bf16" else 1e-4, atol=1e-4)  # noqa: E731
    got = mb.mhla_layernorm_backward(dy, x, mean, rstd, weight=w)
    for s, t in zip(got, grads):
        near(s, t)
    keep, keep_x = buf.clone(), x.contiguous()
    out, _, _ = mb.mhla_layernorm_forward(x, w, b, out=x)
    assert out is x
    near(x, want)
    keep[:, offset: offset + cols] = x
    assert torch.equal(keep, buf)
    d = dy.clone()
    got = mb.mhla_layernorm_backward(d, keep_x, mean, rstd, weight=w, dx=d)
    assert all(torch.equal(s, t) for s, t in zip(got, grads))


def test_leading_axes_empty_rows_and_streams():
    x = make((2, 3, 5, 64), "bf16", 1)
    y, mean, _ = mb.mhla_layernorm_forward(x)
    assert y.shape == x.shape and mean.shape == x.shape[:3]
    assert torch.equal(y.view(-1, 64), mb.mhla_layernorm_forward(x.view(-1, 64))[0])
    with pytest.raises(ValueError):
        mb.mhla_layernorm_forward(x.transpose(1, 2))
    e = torch.empty(0, 64, device="cuda")
    y, mean, rstd = mb.mhla_layernorm_forward(e)
    dx, dw, db = mb.mhla_layernorm_backward(e, e, mean, rstd, weight=torch.ones(64, device="cuda"))
    assert y.shape == e.shape and not dw.any() and not db.any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, _, _ = mb.mhla_layernorm_forward(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y2, mb.mhla_layernorm_forward(x)[0])
