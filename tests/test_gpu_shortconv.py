"""The short causal convolution on the GPU against float64.

A sum of at most five terms and a logistic function (two approximate functions
and three roundings, 2^-20 of it for |z| <= 16): 16 * 2^-24 of the terms'
magnitudes.  A result is rounded once, half a step."""

import numpy as np
import pytest
import torch

from oracle import recurrent_oracle as ro
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = 2.0 ** -24


def make(shape, seed, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(DT[dtype]).cuda()


def f64(t):
    return None if t is None else t.cpu().double().numpy()


def near(got, want, slack, dtype, what):
    bad = np.abs(got - want) > slack + (2.0 ** -8 if dtype == "bf16" else STEP) * np.abs(want) + 1e-30
    assert not bad.any(), (what, np.abs(got - want)[bad].max(), np.argwhere(bad)[:4].tolist())


def check(b, n, d, taps, dtype, wdtype="f32", bias=True, state=True, lengths=None, activation="silu"):
    x, dout, w = make((b, n, d), 1, dtype), make((b, n, d), 2, dtype), make((d, taps), 3, wdtype, 0.6)
    bs = make((d,), 4, wdtype, 0.3) if bias else None
    s = make((b, taps - 1, d), 5, dtype) if state else None
    ds = make((b, taps - 1, d), 6, dtype) if state else None
    out, last = mb.mhla_shortconv_forward(x, w, bs, s, lengths, activation)
    dx, dw, db, dstate = mb.mhla_shortconv_backward(x, w, dout, bs, s, ds, lengths, activation)
    assert (db is None) == (bs is None) and (dstate is None) == (s is None)
    wn, bn = f64(w), f64(bs)
    want_w, size_w, want_b, size_b = np.zeros((d, taps)), np.zeros((d, taps)), np.zeros(d), np.zeros(d)
    for i in range(b):
        length = n if lengths is None else min(max(int(lengths[i]), 0), n)
        xi, si = f64(x[i]), None if s is None else f64(s[i])
        want, want_last, z = ro.shortconv64(xi, wn, bn, si, length, activation)
        size, _, _ = ro.shortconv64(np.abs(xi), np.abs(wn), None if bn is None else np.abs(bn),
                                    None if si is None else np.abs(si), length)
        near(f64(out[i]), want, 16 * STEP * size, dtype, "out")
        assert (out[i, length:] == 0).all()
        np.testing.assert_array_equal(f64(last[i]), want_last)
        args = (xi, wn, f64(dout[i]), bn, si, None if ds is None else f64(ds[i]), length, activation)
        ref = ro.shortconv_backward64(*args)
        # |silu'| <= 1.1 and its own slope <= 0.5, so an error of z counts half
        mag = (np.abs(args[2][:length]) * (1.1 * 16 * STEP + 0.5 * 16 * STEP * size[:length]))
        big = np.zeros((length + taps - 1, d))
        dw_slack = np.zeros((d, taps))
        before = np.zeros((taps - 1, d)) if si is None else np.abs(si)
        rows = np.concatenate([before, np.abs(xi[:length])])
        for j in range(taps):
            big[j: j + length] += np.abs(wn[:, j]) * (mag + 8 * STEP * 1.1 * np.abs(args[2][:length]))
            dw_slack[:, j] = (rows[j: j + length] * (mag + (80 + n / 64) * STEP * 1.1 * np.abs(args[2][:length]))).sum(0)
        if ds is not None:
            big[length:] += 4 * STEP * np.abs(args[5])
        near(f64(dx[i, :length]), ref["dx"][:length], big[taps - 1:], dtype, "dx")
        assert (dx[i, length:] == 0).all()
        if dstate is not None:
            near(f64(dstate[i]), ref["dstate"], big[: taps - 1], dtype, "dstate")
        want_w += ref["dweight"]
        want_b += ref["dbias"]
        size_w += dw_slack
        size_b += (mag + (80 + n / 64) * STEP * 1.1 * np.abs(args[2][:length])).sum(0)
    near(f64(dw), want_w, size_w, "f32", "dweight")
    if db is not None:
        near(f64(db), want_b, size_b, "f32", "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("activation", ["none", "silu"])
@pytest.mark.parametrize("b,n,d", [(1, 1, 1), (2, 2, 5), (1, 3, 64), (3, 17, 66), (1, 200, 130), (2, 513, 32),
                                   (1, 1500, 12)])
def test_shortconv(b, n, d, taps, activation, dtype):
    check(b, n, d, taps, dtype, wdtype=dtype, state=False, activation=activation)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("bias", [True, False])
def test_states_and_lengths(taps, bias, dtype):
    """Lengths around the taps, below zero and beyond the tokens."""
    lengths = torch.tensor([0, 1, 2, 3, 4, 70, 69, 64, -3, 500], dtype=torch.int32).cuda()
    check(10, 70, 40, taps, dtype, "bf16", bias, True, lengths)


def test_large():
    check(4, 700, 1024, 4, "bf16", "bf16")
    check(33, 5, 257, 4, "f32")


def test_padding_is_not_used():
    lengths = torch.tensor([5, 0, 33], dtype=torch.int32).cuda()
    x, dout, w = make((3, 40, 24), 1), make((3, 40, 24), 2), make((24, 4), 3)
    s = make((3, 3, 24), 4)
    bad, dbad = x.clone(), dout.clone()
    for i, k in enumerate(lengths.tolist()):
        bad[i, k:], dbad[i, k:] = float("nan"), float("inf")
    for act in ("none", "silu"):
        for a, b in zip(mb.mhla_shortconv_forward(bad, w, None, s, lengths, act),
                        mb.mhla_shortconv_forward(x, w, None, s, lengths, act)):
            assert torch.equal(a, b)
        for a, b in zip(mb.mhla_shortconv_backward(bad, w, dbad, None, s, None, lengths, act),
                        mb.mhla_shortconv_backward(x, w, dout, None, s, None, lengths, act)):
            assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1, 2, 4])
def test_slices(dtype, offset):
    b, n, d = 2, 90, 40
    fused = make((b, n, 2 * d + 8), 1, dtype)
    x = fused[:, :, offset: offset + d]
    w = make((d, 4), 3)
    res = torch.full((b, n, 2 * d + 8), 7.0, dtype=DT[dtype], device="cuda")
    out = res[:, :, offset: offset + d]
    got = mb.mhla_shortconv_forward(x, w, activation="silu", out=out)
    want = mb.mhla_shortconv_forward(x.contiguous(), w, activation="silu")
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(got[1], want[1])
    assert (res[:, :, :offset] == 7).all() and (res[:, :, offset + d:] == 7).all()
    dout = make((b, n, d + 3), 5, dtype)[:, :, 3:]
    got = mb.mhla_shortconv_backward(x, w, dout, activation="silu", dx=out)
    want = mb.mhla_shortconv_backward(x.contiguous(), w, dout.contiguous(), activation="silu")
    for a, t in zip(got[:2], want[:2]):
        assert torch.equal(a, t)
    assert (res[:, :, :offset] == 7).all() and (res[:, :, offset + d:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("b,d", [(1, 1), (3, 70), (64, 1024), (5, 1001)])
def test_step(b, d, taps, dtype):
    x, w, bias, s = make((b, 1, d), 1, dtype), make((d, taps), 2, dtype), make((d,), 3, dtype), make((b, taps - 1, d), 4, dtype)
    want, last = mb.mhla_shortconv_forward(x, w, bias, s, activation="silu")
    keep, into = s.clone(), torch.empty_like(s)
    out = mb.mhla_shortconv_step(x[:, 0], w, s, bias, "silu", state_out=into)
    assert torch.equal(s, keep) and torch.equal(into, last)
    assert torch.equal(out, want[:, 0])
    assert torch.equal(mb.mhla_shortconv_step(x[:, 0], w, s, bias, "silu"), out) and torch.equal(s, last)


def test_tokens_one_by_one():
    x, w, s = make((2, 20, 30), 1, "bf16"), make((30, 4), 2), make((2, 3, 30), 3, "bf16")
    want, last = mb.mhla_shortconv_forward(x, w, None, s)
    got = [mb.mhla_shortconv_step(x[:, t], w, s) for t in range(20)]
    assert torch.equal(torch.stack(got, 1), want) and torch.equal(s, last)


def test_in_place_state():
    for n in (1, 2, 100):
        x, w, s = make((2, n, 30), 1, "bf16"), make((30, 4), 2), make((2, 3, 30), 3, "bf16")
        want, last = mb.mhla_shortconv_forward(x, w, None, s)
        out, same = mb.mhla_shortconv_forward(x, w, None, s, state_out=s)
        assert same is s and torch.equal(out, want) and torch.equal(s, last)


def test_empty():
    x, w, s = torch.empty(2, 0, 8, device="cuda"), make((8, 4), 1), make((2, 3, 8), 2)
    out, last = mb.mhla_shortconv_forward(x, w, None, s)
    assert out.shape == x.shape and torch.equal(last, s)
    dx, dw, db, ds = mb.mhla_shortconv_backward(x, w, x, None, s, s)
    assert (dw == 0).all() and db is None and torch.equal(ds, s)
    x = torch.empty(0, 5, 8, device="cuda")
    assert mb.mhla_shortconv_forward(x, w)[1].shape == (0, 3, 8)
    dx, dw, db, ds = mb.mhla_shortconv_backward(x, w, x, make((8,), 3))
    assert (dw == 0).all() and (db == 0).all()


def test_without_the_weights_gradients():
    x, w, dout = make((2, 90, 40), 1, "bf16"), make((40, 4), 2), make((2, 90, 40), 3, "bf16")
    want = mb.mhla_shortconv_backward(x, w, dout, activation="silu")
    got = mb.mhla_shortconv_backward(x, w, dout, activation="silu", params=False)
    assert got[1] is None and got[2] is None and torch.equal(got[0], want[0])


def test_results_do_not_change():
    x, w, dout = make((3, 900, 200), 1, "bf16"), make((200, 4), 2), make((3, 900, 200), 3, "bf16")
    runs = [mb.mhla_shortconv_backward(x, w, dout, make((200,), 4), activation="silu") for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r[:3], runs[0][:3]))


def test_no_device_error_was_reported():
    assert mb.mhla_device_status() == (0, 0)


@pytest.mark.parametrize("first", [0, 1, 2, 3])
@pytest.mark.parametrize("d", [1, 2, 3, 5, 129, 131])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_lies_around_single_elements_is_not_used(first, d, dtype):
    """Rows that start at any element, NaN before the first, behind the last, between them and past the lengths."""
    b, n, width = 3, 41, d + 3
    gen = torch.Generator().manual_seed(d)
    w, bias = torch.randn(d, 4, generator=gen).cuda(), torch.randn(d, generator=gen).cuda()
    lengths = torch.tensor([41, 17, 0], dtype=torch.int32).cuda()

    def place():
        t = torch.randn(b, n, d, generator=gen).to(dtype).cuda()
        for i, k in enumerate((41, 17, 0)):
            t[i, k:] = 0
        memory = torch.full((first + b * n * width,), float("nan"), dtype=dtype, device="cuda")
        view = memory.as_strided((b, n, d), (n * width, width, 1), first)
        view.copy_(t)
        for i, k in enumerate((41, 17, 0)):
            view[i, k:] = float("nan")
        return t, memory, view

    (x, _, xv), (do, _, dov) = place(), place()
    out, state = mb.mhla_shortconv_forward(x, w, bias, lengths=lengths, activation="silu")
    dx, dw, db, _ = mb.mhla_shortconv_backward(x, w, do, bias, lengths=lengths, activation="silu")
    _, memory, result = place()
    got = mb.mhla_shortconv_forward(xv, w, bias, lengths=lengths, activation="silu", out=result)
    assert torch.equal(result, out) and torch.equal(got[1], state)
    grads = mb.mhla_shortconv_backward(xv, w, dov, bias, lengths=lengths, activation="silu", dx=result)
    assert torch.equal(result, dx) and torch.equal(grads[1], dw) and torch.equal(grads[2], db)
    result.fill_(float("nan"))
    assert memory.isnan().all()  # nothing was written between the rows
