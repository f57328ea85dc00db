"""The gated recurrence on the GPU against the float64 recurrence.

Errors: sigma is off by kappa = 2^-18 of itself for |gate| <= 16 (its argument
16 * 2^-24, two approximate functions and three roundings of 2^-22 at most, so
2^-19, and as much again for what expm1 and the root make of it); a by
kappa |log a| a and a rounding next to 1, 2^-24; a step of the recurrence rounds
its two terms and a map of the scan its own, 4 * 2^-24 of their magnitude in
all.  What a token adds is carried on by a, so the bounds follow the same
recurrences.  A result is rounded once: half a step, 2^-8 for bf16."""

import numpy as np
import pytest
import torch

from oracle import recurrent_oracle as ro
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
KAPPA, STEP = 2.0 ** -18, 2.0 ** -24
COMBOS = [("decay", "norm", True), ("decay", "mean", False), ("decay", "none", True), ("sigmoid", "norm", False),
          ("sigmoid", "mean", True), ("sigmoid", "none", False)]


def make(shape, seed, dtype="f32", scale=1.0, shift=0.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale + shift).to(DT[dtype]).cuda()


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def decays(d, seed=9):
    rate = torch.rand(d, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    return -torch.exp(rate * np.log(4000.0) + np.log(0.001)).float().cuda()


def problem(b, n, d, dtype, kind, in_gate, state, seed=1):
    p = dict(x=make((b, n, d), seed, dtype), gate=make((b, n, d), seed + 1, dtype, 2.0, 0.5),
             log_decay=decays(d) if kind == "decay" else None,
             input_gate=make((b, n, d), seed + 2, dtype) if in_gate else None,
             state=make((b, d), seed + 3) if state else None)
    return p


def bounds(x, gate, log_decay, input_gate, state, length, scale, dout=None, dstate_out=None):
    """Errors that float32 may leave in out, the final state and the gradients."""
    n = len(x) if length is None else min(max(length, 0), len(x))
    a, c, log_a = ro.gated_factors64(gate, log_decay, scale)
    q = ro.sigmoid64(input_gate) if input_gate is not None else np.ones_like(x)
    u = np.abs(x) * q
    m = np.zeros(x.shape[1]) if state is None else np.abs(state)
    e = np.zeros_like(m)
    da = KAPPA * np.abs(log_a) * a + STEP
    eh, mh = np.zeros((n + 1, x.shape[1])), np.zeros((n + 1, x.shape[1]))
    mh[0] = m
    for t in range(n):
        e = a[t] * e + da[t] * m + (3 * KAPPA + 4 * STEP) * c[t] * u[t] + 4 * STEP * a[t] * m
        m = a[t] * m + c[t] * u[t]
        eh[t + 1], mh[t + 1] = e, m
    if dout is None:
        return eh, mh
    res = {k: np.zeros_like(x) for k in ("dx", "dgate", "dinput_gate")}
    res["dlog_decay"] = np.zeros(x.shape[1])
    g = np.zeros(x.shape[1]) if dstate_out is None else np.abs(dstate_out)
    e = np.zeros_like(g)
    s, rest = ro.sigmoid64(gate), ro.sigmoid64(-gate)
    for t in reversed(range(n)):
        g, e = g + np.abs(dout[t]), e + STEP * (g + np.abs(dout[t]))
        with np.errstate(divide="ignore", invalid="ignore"):
            dc = {"norm": np.where(c[t] > 0, a[t] ** 2 / c[t], 0.0), "mean": a[t], "none": 0 * a[t]}[scale]
        terms = a[t] * mh[t] + u[t] * dc
        dlog = e * terms + g * (a[t] * eh[t] + (5 * KAPPA + 8 * STEP) * terms)
        slope = rest[t] * (np.abs(log_decay) * s[t] if log_decay is not None else 1.0)
        res["dgate"][t] = slope * (dlog + 4 * KAPPA * g * terms)
        res["dx"][t] = c[t] * q[t] * (e + 4 * KAPPA * g)
        # 1 - sigma(i) is a difference of numbers up to 1
        res["dinput_gate"][t] = c[t] * u[t] * ((1 - q[t]) * (e + 4 * KAPPA * g) + (KAPPA + 2 * STEP) * g)
        # the term's error and the roundings of a sum of n terms
        res["dlog_decay"] += s[t] * (dlog + (KAPPA + (12 + n / 64) * STEP) * g * terms)
        e = a[t] * e + da[t] * g + 4 * STEP * a[t] * g
        g = a[t] * g
    res["dstate"] = e + STEP * g
    return eh, mh, res


def near(got, want, slack, dtype, what):
    half = 2.0 ** -8 if dtype == "bf16" else STEP
    bad = np.abs(got - want) > slack + half * np.abs(want) + 1e-30
    assert not bad.any(), (what, np.abs(got - want)[bad].max(), int(bad.sum()), np.argwhere(bad)[:4].tolist())


def check(p, dtype, scale, lengths=None, dstate=False, marks=True, seed=50):
    b, n, d = p["x"].shape
    dout = make((b, n, d), seed, dtype)
    ds = make((b, d), seed + 1) if dstate else None
    out, state, kept = mb.mhla_gated_forward(**p, lengths=lengths, scale=scale, keep=True)
    grads = mb.mhla_gated_backward(p["x"], p["gate"], dout, p["log_decay"], p["input_gate"], p["state"], ds,
                                   kept if marks else None, lengths, scale)
    got = dict(zip(("dx", "dgate", "dinput_gate", "dlog_decay", "dstate"), grads))
    assert (got["dinput_gate"] is None) == (p["input_gate"] is None)
    assert (got["dlog_decay"] is None) == (p["log_decay"] is None)
    dlog, dlog_slack = np.zeros(d), np.zeros(d)
    one = lambda t, i: None if t is None else f64(t[i])  # noqa: E731
    for i in range(b):
        length = None if lengths is None else int(lengths[i])
        args = (f64(p["x"][i]), f64(p["gate"][i]), f64(p["log_decay"]), one(p["input_gate"], i), one(p["state"], i))
        want, states = ro.gated64(*args, length, scale)
        eh, mh, slack = bounds(*args, length, scale, f64(dout[i]), one(ds, i))
        k = len(states) - 1
        near(f64(out[i, :k]), want[:k], eh[1:], dtype, "out")
        assert (out[i, k:] == 0).all()
        near(f64(state[i]), states[-1], eh[-1], "f32", "state")
        at = np.minimum(np.arange(kept.shape[1]) * mb.GATED_MARK, k)
        near(f64(kept[i]), states[at], eh[at], "f32", "marks")
        ref = ro.gated_backward64(args[0], args[1], f64(dout[i]), *args[2:], one(ds, i), length, scale)
        for name in ("dx", "dgate") + (("dinput_gate",) if args[3] is not None else ()):
            near(f64(got[name][i]), ref[name], slack[name], dtype, name)
            assert (got[name][i, k:] == 0).all()
        if got["dstate"] is not None:
            near(f64(got["dstate"][i]), ref["dstate"], slack["dstate"], "f32", "dstate")
        dlog += ref["dlog_decay"]
        dlog_slack += slack["dlog_decay"]
    if got["dlog_decay"] is not None:
        near(f64(got["dlog_decay"]), dlog, dlog_slack + b * STEP * np.abs(dlog), "f32", "dlog_decay")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,scale,in_gate", COMBOS)
@pytest.mark.parametrize("b,n,d", [(1, 1, 1), (2, 3, 5), (1, 8, 64), (2, 64, 66), (1, 65, 130), (3, 200, 33),
                                   (1, 777, 96), (2, 1100, 64)])
def test_gated(b, n, d, kind, scale, in_gate, dtype):
    check(problem(b, n, d, dtype, kind, in_gate, False), dtype, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,scale,in_gate", COMBOS)
@pytest.mark.parametrize("marks", [True, False])
def test_states_and_lengths(kind, scale, in_gate, dtype, marks):
    """Lengths below zero and beyond the tokens are clamped; what lies past them is not used."""
    lengths = torch.tensor([0, 1, 150, 64, 63, 7, -5, 1000, 149], dtype=torch.int32).cuda()
    p = problem(9, 150, 70, dtype, kind, in_gate, True)
    for t in (p["x"], p["gate"], p["input_gate"]):
        if t is not None:
            for i, k in enumerate(lengths.clamp(0, 150).tolist()):
                t[i, k:] = float("nan")
    clean = {k: v if v is None or k in ("log_decay", "state") else torch.nan_to_num(v) for k, v in p.items()}
    check(clean, dtype, scale, lengths, True, marks)
    for a, b in zip(mb.mhla_gated_forward(**p, lengths=lengths, scale=scale, keep=True),
                    mb.mhla_gated_forward(**clean, lengths=lengths, scale=scale, keep=True)):
        assert torch.equal(a, b)
    dout = make((9, 150, 70), 60, dtype)
    bad = dout.clone()
    for i, k in enumerate(lengths.clamp(0, 150).tolist()):
        bad[i, k:] = float("inf")
    grads = [mb.mhla_gated_backward(q["x"], q["gate"], d, q["log_decay"], q["input_gate"], q["state"], lengths=lengths,
                                    scale=scale) for q, d in ((p, bad), (clean, dout))]
    for a, b in zip(*grads):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("b,n,d", [(1, 4000, 64), (1, 3001, 10), (2, 2049, 200), (40, 70, 900)])
def test_many_tiles(b, n, d):
    check(problem(b, n, d, "bf16", "decay", True, True), "bf16", "norm", dstate=True)


def test_extreme_gates():
    """Saturated gates in both directions, a decay of zero, and channels that keep or forget everything."""
    p = problem(2, 130, 64, "f32", "decay", True, True)
    p["gate"][:, ::3] = 30.0
    p["gate"][:, 1::3] = -30.0
    p["input_gate"][:, ::2] = 80.0
    p["log_decay"][:8] = torch.tensor([0.0, -1e-30, -1e-8, -50.0, -500.0, -1e30, -0.25, -0.2500001])
    for scale in ("norm", "mean", "none"):
        out, state, kept = mb.mhla_gated_forward(**p, scale=scale, keep=True)
        grads = mb.mhla_gated_backward(p["x"], p["gate"], torch.ones_like(p["x"]), p["log_decay"], p["input_gate"],
                                       p["state"], marks=kept, scale=scale)
        for t in (out, state) + grads:
            assert torch.isfinite(t).all(), scale
        for i in range(2):
            args = [f64(v[i]) if v.dim() > 1 else f64(v) for v in (p["x"], p["gate"], p["log_decay"], p["input_gate"],
                                                                 p["state"])]
            want, states = ro.gated64(*args, None, scale)
            # |gate| = 30 where 16 was counted on: twice the slack
            eh, mh = bounds(*args, None, scale)
            near(f64(out[i]), want, 2 * eh[1:], "f32", scale)
    p = dict(x=make((1, 9, 2), 1), gate=torch.full((1, 9, 2), float("-inf"), device="cuda"), state=make((1, 2), 2))
    out, state, _ = mb.mhla_gated_forward(**p, scale="mean")
    assert torch.equal(out, p["x"])  # a = 0: each token replaces the state
    p["gate"] = -p["gate"]
    out, state, _ = mb.mhla_gated_forward(**p, scale="mean")
    assert torch.equal(state, p["state"]) and torch.equal(out, p["state"][:, None].expand(1, 9, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1, 2])
def test_slices_of_a_fused_projection(dtype, offset):
    b, n, d = 2, 100, 48
    fused = make((b, n, 3 * d + 8), 1, dtype)
    x, r, i = (fused[:, :, offset + j * d: offset + (j + 1) * d] for j in range(3))
    g = decays(d)
    res = torch.full((b, n, 3 * d + 8), 7.0, dtype=DT[dtype], device="cuda")
    out = res[:, :, offset: offset + d]
    got = mb.mhla_gated_forward(x, r, g, i, out=out, keep=True)
    assert got[0] is out
    want = mb.mhla_gated_forward(x.contiguous(), r.contiguous(), g, i.contiguous(), keep=True)
    for a, w in zip(got, want):
        assert torch.equal(a, w)
    assert (res[:, :, :offset] == 7).all() and (res[:, :, offset + d:] == 7).all()
    dout = make((b, n, d + 3), 5, dtype)[:, :, 3:]
    dx, dr, di = (res[:, :, offset + j * d: offset + (j + 1) * d] for j in range(3))
    got = mb.mhla_gated_backward(x, r, dout, g, i, marks=want[2], dx=dx, dgate=dr, dinput_gate=di)
    ref = mb.mhla_gated_backward(x.contiguous(), r.contiguous(), dout.contiguous(), g, i.contiguous(), marks=want[2])
    for a, w in zip(got[:4], ref[:4]):
        assert torch.equal(a, w)
    assert got[4] is None and (res[:, :, 3 * d + offset:] == 7).all()


def test_broadcast_inputs():
    """One gate for every sequence, one row for every token."""
    x, r = make((3, 90, 40), 1), make((1, 90, 40), 2)
    i = make((3, 1, 40), 3).expand(3, 90, 40)
    got = mb.mhla_gated_forward(x, r.expand(3, 90, 40), None, i)
    want = mb.mhla_gated_forward(x, r.repeat(3, 1, 1), None, i.contiguous())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,scale,in_gate", COMBOS)
@pytest.mark.parametrize("b,d", [(1, 1), (3, 70), (64, 1024), (5, 1001)])
def test_step(b, d, kind, scale, in_gate, dtype):
    p = problem(b, 1, d, dtype, kind, in_gate, True)
    want, last, _ = mb.mhla_gated_forward(**p, scale=scale)
    flat = {k: v[:, 0] if k in ("x", "gate", "input_gate") and v is not None else v for k, v in p.items()}
    keep = p["state"].clone()
    into = torch.empty_like(keep)
    out = mb.mhla_gated_step(**flat, scale=scale, state_out=into)
    assert torch.equal(out, want[:, 0]) and torch.equal(into, last) and torch.equal(keep, p["state"])
    out = mb.mhla_gated_step(**flat, scale=scale)
    assert torch.equal(out, want[:, 0]) and torch.equal(p["state"], last)


def test_tokens_one_by_one():
    p = problem(2, 40, 50, "f32", "decay", True, True)
    out, last, _ = mb.mhla_gated_forward(**p)
    state = p["state"].clone()
    steps = [mb.mhla_gated_step(p["x"][:, t], p["gate"][:, t], state, p["log_decay"], p["input_gate"][:, t])
             for t in range(40)]
    # both are within the float32 bounds of the recurrence
    for i in range(2):
        eh, _ = bounds(f64(p["x"][i]), f64(p["gate"][i]), f64(p["log_decay"]), f64(p["input_gate"][i]),
                       f64(p["state"][i]), None, "norm")
        for t in range(40):
            near(f64(steps[t][i]), f64(out[i, t]), 2 * eh[t + 1], "f32", t)
        near(f64(state[i]), f64(last[i]), 2 * eh[-1], "f32", "state")


def test_in_place_states():
    p = problem(3, 100, 64, "bf16", "decay", True, True)
    want = mb.mhla_gated_forward(**p)
    state = p.pop("state").clone()
    got = mb.mhla_gated_forward(**p, state=state, state_out=state)
    assert torch.equal(got[0], want[0]) and torch.equal(state, want[1])
    dout, ds = make((3, 100, 64), 7, "bf16"), make((3, 64), 8)
    args = (p["x"], p["gate"], dout, p["log_decay"], p["input_gate"])
    want = mb.mhla_gated_backward(*args, dstate_out=ds, dstate=torch.empty_like(ds))
    mb.mhla_gated_backward(*args, dstate_out=ds, dstate=ds)
    assert torch.equal(ds, want[4])


def test_empty():
    x = torch.empty(2, 0, 8, device="cuda")
    s = make((2, 8), 1)
    out, state, marks = mb.mhla_gated_forward(x, x, decays(8), state=s, keep=True)
    assert out.shape == x.shape and torch.equal(state, s) and marks.shape == (2, 0, 8)
    dx, dr, di, dg, ds = mb.mhla_gated_backward(x, x, x, decays(8), state=s, dstate_out=s, marks=marks)
    assert torch.equal(ds, s) and (dg == 0).all() and di is None
    x = torch.empty(0, 5, 8, device="cuda")
    out, state, _ = mb.mhla_gated_forward(x, x, decays(8))
    assert out.shape == x.shape and state.shape == (0, 8)
    assert (mb.mhla_gated_backward(x, x, x, decays(8))[3] == 0).all()
    x = torch.empty(2, 5, 0, device="cuda")
    assert mb.mhla_gated_forward(x, x)[0].shape == x.shape


def test_results_do_not_change():
    p = problem(3, 900, 200, "bf16", "decay", True, True)
    dout = make((3, 900, 200), 7, "bf16")
    runs = []
    for _ in range(3):
        f = mb.mhla_gated_forward(**p, keep=True)
        runs.append(f + mb.mhla_gated_backward(p["x"], p["gate"], dout, p["log_decay"], p["input_gate"], p["state"],
                                               marks=f[2]))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_slow_channels_do_not_drift():
    """32k tokens in channels that remember thousands: float32's own noise, not a bias."""
    n, d = 32768, 64
    p = problem(1, n, d, "bf16", "decay", False, False)
    p["log_decay"] = torch.full((d,), -0.0005).cuda()
    p["x"] = p["x"].abs()  # nothing cancels, so an error of a shows in full
    out, state, _ = mb.mhla_gated_forward(**p, scale="mean")
    want, states = ro.gated64(f64(p["x"][0]), f64(p["gate"][0]), f64(p["log_decay"]), None, None, None, "mean")
    # a rounding of 2^-25 in a, the sum and the product at each of the ~4000 tokens
    # that a channel remembers, of either sign: 4 deviations of their random sum
    assert (np.abs(f64(state[0]) - states[-1]) / np.abs(states[-1])).max() <= 4 * np.sqrt(3 * 4000) * 2.0 ** -25


def test_no_device_error_was_reported():
    assert mb.mhla_device_status() == (0, 0)
