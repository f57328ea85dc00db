"""Linear attention with a decay for each head on the GPU against the float64
recurrence: prompts, single tokens and gradients.

Bounds are sums of roundings, entry by entry.  With half = 2^-8 the largest
relative error of one rounding to bf16: the tensor-core path rounds the output,
the decayed scores (terms of |P| |Z|) and the operand copy of the state
(|X| |S|), and holds the state's addends as bf16 pairs (2^-16 a term); the
CUDA-core path rounds the output only.  Sums in float32 add (terms + 32)
2^-24 of the sum of magnitudes (32: the roundings of powers and products)."""

import math

import numpy as np
import pytest
import torch

from oracle import sequence_oracle as sq
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
EPS = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def make(shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(DT[dtype]).cuda()


def rows(layout, b, h, n, d):
    return (b, h, n, d) if layout == "bhnd" else (b, n, h, d)


def head(t, layout, b, h):
    a = f64(t)
    return a[b, h] if layout == "bhnd" else a[b, :, h]


def decays(h, kind="usual"):
    if kind == "usual":
        return torch.log1p(-torch.exp2(-torch.linspace(1, 9, h, dtype=torch.float64))).float().cuda()
    return torch.full((h,), kind, dtype=torch.float32).cuda()


def check(got, want, slack, what):
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - want) - slack
    assert over.max(initial=-1.0) <= 0, f"{what}: {np.abs(got - want).max():.3e} off, {over.max():.3e} over its bound"


def roundings(dtype, tensor, want, scores, copies, sums, n, d, total):
    r = (n + 2 * d + 32) * EPS * sums
    if dtype == "bf16":
        r = r + HALF * np.abs(want)
        if tensor:  # prompts of fewer than 128 tokens keep 16 bits of the operands
            r = r + (1 + HALF) * HALF * (scores + copies) * (1 if total >= 128 else HALF) + 2.0 ** -16 * sums
    return r + 1e-30


def weights(g, n):
    d = np.arange(n)[:, None] - np.arange(n)[None, :]
    lam = math.exp(g)
    return np.where(d >= 0, lam ** np.maximum(d, 0).astype(np.float64), 0.0)


def check_forward(q, k, v, g, out, state_out, state, length, scale, dtype, tensor):
    n = len(q) if length is None else min(max(length, 0), len(q))
    want, states = sq.decay64(q, k, v, g, state, length, scale)
    abs_out, abs_states = sq.decay64(abs(q), abs(k), abs(v), g, None if state is None else abs(state), length, abs(scale))
    scores = np.zeros_like(want)
    copies = np.zeros_like(want)
    scores[:n] = abs(scale) * (weights(g, n) * np.abs(q[:n] @ k[:n].T)) @ np.abs(v[:n])
    most = np.maximum.accumulate(np.abs(states), axis=0)
    copies[:n] = abs(scale) * np.einsum("ta,tac->tc", np.abs(q[:n]), most[:n])
    check(out, want, roundings(dtype, tensor, want, scores, copies, abs_out, n, q.shape[1], len(q)), "out")
    check(state_out, states[n], 2.0 ** -16 * tensor * abs_states[n] + (n + 32) * EPS * abs_states[n] + 1e-30, "state")


SHAPES = [  # batch, heads, tokens, dk, dv, layout
    (1, 1, 1, 64, 64, "bhnd"),
    (2, 3, 2, 16, 16, "bnhd"),
    (1, 2, 63, 64, 64, "bnhd"),
    (1, 2, 64, 64, 128, "bhnd"),
    (2, 2, 65, 32, 64, "bhnd"),
    (1, 2, 127, 128, 128, "bnhd"),
    (1, 1, 129, 128, 16, "bhnd"),
    (2, 1, 200, 16, 32, "bhnd"),
    (1, 2, 333, 64, 32, "bnhd"),
    (1, 1, 700, 64, 64, "bhnd"),    # two segments
    (1, 2, 1111, 128, 64, "bnhd"),  # four segments, a short last chunk
    (1, 1, 128, 128, 128, "bhnd"),
    (1, 2, 300, 128, 64, "bhnd"),
    (2, 3, 1111, 128, 128, "bnhd"),
    (1, 1, 900, 32, 128, "bhnd"),
    (1, 1, 1025, 16, 64, "bhnd"),   # a last segment of one token
]
VARIANTS = [("bf16", "tensor"), ("bf16", "simt"), ("f32", "simt")]


@pytest.mark.parametrize("dtype,variant", VARIANTS)
@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("b,h,n,dk,dv,layout", SHAPES)
def test_forward(b, h, n, dk, dv, layout, with_state, dtype, variant):
    q, k = (make(rows(layout, b, h, n, dk), dtype, i) for i in (1, 2))
    v = make(rows(layout, b, h, n, dv), dtype, 3)
    g = decays(h)
    state = make((b, h, dk, dv), "f32", 4, 3.0) if with_state else None
    scale = dk ** -0.5
    out, state_out = mb.mhla_decay_forward(q, k, v, g, state=state, scale=scale, layout=layout, variant=variant)
    scale = float(np.float32(scale))
    for i in range(b):
        for j in range(h):
            check_forward(head(q, layout, i, j), head(k, layout, i, j), head(v, layout, i, j), float(g[j]),
                          head(out, layout, i, j), f64(state_out)[i, j], None if state is None else f64(state)[i, j],
                          None, scale, dtype, variant == "tensor")


@pytest.mark.parametrize("dtype,variant", VARIANTS)
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("n,lengths", [(130, [0, 1, 64, 65, 130, 999, -3]), (1300, [0, 1, 255, 256, 257, 1299, 1300])])
def test_forward_lengths(n, lengths, dim, dtype, variant):
    b, h, dk, dv = len(lengths), 1, dim, dim
    q, k, v = (make((b, h, n, dk), dtype, i) for i in (1, 2, 3))
    state = make((b, h, dk, dv), "f32", 4)
    g = decays(h, -0.01)
    past = torch.arange(n, device="cuda")[None, :] >= torch.tensor(lengths, device="cuda").clamp(0, n)[:, None]
    for t in (q, k, v):  # what lies past a length is never used
        t.masked_fill_(past[:, None, :, None], float("nan"))
    lens = torch.tensor(lengths, dtype=torch.int32).cuda()
    out, state_out = mb.mhla_decay_forward(q, k, v, g, state=state, lengths=lens, variant=variant)
    assert torch.equal(out.masked_select(past[:, None, :, None]), torch.zeros_like(out.masked_select(past[:, None, :, None])))
    for i in range(b):
        m = min(max(lengths[i], 0), n)
        qq, kk, vv = (np.nan_to_num(f64(t)[i, 0]) for t in (q, k, v))
        check_forward(qq, kk, vv, float(g[0]), f64(out)[i, 0], f64(state_out)[i, 0], f64(state)[i, 0], m, 1.0, dtype,
                      variant == "tensor")
        if m == 0:
            assert torch.equal(state_out[i], state[i])


@pytest.mark.parametrize("dtype,variant", VARIANTS)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("g", [0.0, -math.inf, -40.0, -1e-7, 0.01])
def test_forward_extreme_decays(g, d, dtype, variant):
    n = 600
    q, k, v = (make((1, 1, n, d), dtype, i) for i in (1, 2, 3))
    state = make((1, 1, d, d), "f32", 4, 1e4)
    out, state_out = mb.mhla_decay_forward(q, k, v, decays(1, g), state=state, variant=variant)
    check_forward(f64(q)[0, 0], f64(k)[0, 0], f64(v)[0, 0], float(np.float32(g)), f64(out)[0, 0], f64(state_out)[0, 0],
                  f64(state)[0, 0], None, 1.0, dtype, variant == "tensor")


def check_backward(q, k, v, do, g, got, state, dstate_out, length, scale, dtype, tensor):
    n = len(q) if length is None else min(max(length, 0), len(q))
    want = sq.decay_backward64(q, k, v, g, do, state, dstate_out, length, scale)
    mag = lambda a: None if a is None else np.abs(a)  # noqa: E731
    sums = sq.decay_backward64(abs(q), abs(k), abs(v), g, abs(do), mag(state), mag(dstate_out), length, scale)
    _, states = sq.decay64(q, k, v, g, state, length, scale)
    most_s = np.maximum.accumulate(np.abs(states), axis=0)
    r = np.zeros_like(states[0]) if dstate_out is None else dstate_out.copy()
    most_r = np.zeros((n,) + r.shape)
    top = np.abs(r)
    for t in reversed(range(n)):
        r = r + scale * np.outer(q[t], do[t])
        top = np.maximum(top, np.abs(r))
        most_r[t] = top
        r = math.exp(g) * r
    w = scale * weights(g, n)
    part, score = w * np.abs(do[:n] @ v[:n].T), w * np.abs(q[:n] @ k[:n].T)
    terms = [part @ np.abs(k[:n]), part.T @ np.abs(q[:n]), score.T @ np.abs(do[:n])]
    copies = [scale * np.einsum("tc,tac->ta", np.abs(do[:n]), most_s[:n]), np.einsum("tc,tac->ta", np.abs(v[:n]), most_r),
              np.einsum("ta,tac->tc", np.abs(k[:n]), most_r)]
    for i, name in enumerate(("dq", "dk", "dv")):
        full = [np.zeros_like(want[i]), np.zeros_like(want[i])]
        full[0][:n], full[1][:n] = terms[i], copies[i]
        check(got[i], want[i], roundings(dtype, tensor, want[i], full[0], full[1], sums[i], n, 128, len(q)), name)
    check(got[3], want[3], (2.0 ** -16 * tensor + (n + 32) * EPS) * sums[3] + 1e-30, "dstate")


@pytest.mark.parametrize("dtype,variant", VARIANTS)
@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("b,h,n,dk,dv,layout", SHAPES)
def test_backward(b, h, n, dk, dv, layout, with_state, dtype, variant):
    q, k = (make(rows(layout, b, h, n, dk), dtype, i) for i in (1, 2))
    v, do = (make(rows(layout, b, h, n, dv), dtype, i) for i in (3, 5))
    g = decays(h)
    state = make((b, h, dk, dv), "f32", 4, 3.0) if with_state else None
    ds = make((b, h, dk, dv), "f32", 6) if with_state else None
    scale = dk ** -0.5
    into = None if with_state else torch.empty(b, h, dk, dv, device="cuda")  # asked for although there is no state
    got = mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds, scale=scale, layout=layout, variant=variant,
                                 dstate=into)
    if not with_state:
        fewer = mb.mhla_decay_backward(q, k, v, g, do, scale=scale, layout=layout, variant=variant)
        assert fewer[3] is None
        for x, y in zip(fewer[:3], got[:3]):  # states of 16 bits where none is asked for
            torch.testing.assert_close(x, y, rtol=2.0 ** -6, atol=2.0 ** -8 * y.abs().max().item())
    scale = float(np.float32(scale))
    for i in range(b):
        for j in range(h):
            check_backward(*(head(t, layout, i, j) for t in (q, k, v, do)), float(g[j]),
                           [head(t, layout, i, j) for t in got[:3]] + [f64(got[3])[i, j]],
                           None if state is None else f64(state)[i, j], None if ds is None else f64(ds)[i, j], None,
                           scale, dtype, variant == "tensor")


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("dtype,variant", VARIANTS)
def test_backward_lengths(d, dtype, variant):
    n, lengths = 600, [0, 1, 63, 300, 600]
    b = len(lengths)
    q, k, v, do = (make((b, 1, n, d), dtype, i) for i in (1, 2, 3, 4))
    state, ds = make((b, 1, d, d), "f32", 5), make((b, 1, d, d), "f32", 6)
    past = torch.arange(n, device="cuda")[None, :] >= torch.tensor(lengths, device="cuda")[:, None]
    for t in (q, k, v, do):
        t.masked_fill_(past[:, None, :, None], float("inf"))
    g = decays(1, -0.02)
    got = mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds, variant=variant,
                                 lengths=torch.tensor(lengths, dtype=torch.int32).cuda())
    for t in got[:3]:
        assert not t.masked_select(past[:, None, :, None]).any()
    for i in range(b):
        check_backward(*(np.nan_to_num(f64(t)[i, 0], posinf=0.0) for t in (q, k, v, do)), float(g[0]),
                       [f64(t)[i, 0] for t in got], f64(state)[i, 0], f64(ds)[i, 0], lengths[i], 1.0, dtype,
                       variant == "tensor")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (32, 64), (64, 64), (64, 16), (128, 32), (128, 128)])
def test_step(dk, dv, dtype):
    b, h = 3, 5
    g = decays(h)
    g[0] = -math.inf
    state = make((b, h, dk, dv), "f32", 9, 4.0)
    before = state.clone()
    q, k, v = make((b, h, dk), dtype, 1), make((b, h, dk), dtype, 2), make((b, h, dv), dtype, 3)
    other = torch.empty_like(state)
    apart = mb.mhla_decay_step(q, k, v, g, state, scale=0.25, state_out=other)
    assert torch.equal(state, before)
    out = mb.mhla_decay_step(q, k, v, g, state, scale=0.25)
    assert torch.equal(out, apart) and torch.equal(state, other)
    for i in range(b):
        for j in range(h):
            a = [f64(t)[i, j][None] for t in (q, k, v)]
            want, states = sq.decay64(*a, float(g[j]), f64(before)[i, j], None, 0.25)
            mag, abs_states = sq.decay64(*(np.abs(x) for x in a), float(g[j]), np.abs(f64(before)[i, j]), None, 0.25)
            check(f64(out)[i, j], want[0], roundings(dtype, False, want[0], 0, 0, mag[0], 1, dk, 1), "out")
            check(f64(state)[i, j], states[1], 32 * EPS * abs_states[1], "state")


def test_step_follows_prompt():
    """A prompt and then single tokens give what the whole prompt gives."""
    b, h, n, d, more = 2, 3, 137, 64, 5
    q, k, v = (make((b, h, n + more, d), "f32", i) for i in (1, 2, 3))
    g = decays(h)
    whole, last = mb.mhla_decay_forward(q, k, v, g)
    out, state = mb.mhla_decay_forward(q[:, :, :n], k[:, :, :n], v[:, :, :n], g)
    parts = [out]
    for t in range(n, n + more):
        parts.append(mb.mhla_decay_step(q[:, :, t], k[:, :, t], v[:, :, t], g, state)[:, :, None])
    mag, abs_last = mb.mhla_decay_forward(q.abs(), k.abs(), v.abs(), g)
    tol = 2 * (n + 2 * d + 64) * EPS  # both sides
    assert ((torch.cat(parts, 2) - whole).abs() <= tol * mag).all()
    assert ((state - last).abs() <= tol * abs_last).all()


@pytest.mark.parametrize("variant,dtype", [("tensor", "bf16"), ("simt", "f32")])
def test_later_tokens_leave_earlier_outputs(variant, dtype):
    n, d = 800, 64
    q, k, v = (make((1, 2, n, d), dtype, i) for i in (1, 2, 3))
    g = decays(2)
    a, _ = mb.mhla_decay_forward(q, k, v, g, variant=variant)
    cut = 415
    for t in (q, k, v):
        t[:, :, cut:] = make((1, 2, n - cut, d), dtype, 77)
    b, _ = mb.mhla_decay_forward(q, k, v, g, variant=variant)
    assert torch.equal(a[:, :, :cut], b[:, :, :cut]) and not torch.equal(a[:, :, cut:], b[:, :, cut:])


@pytest.mark.parametrize("dtype,d", [("bf16", 32), ("f32", 32)])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_strides_and_alignment(offset, dtype, d):
    """q, k, v, out as slices of one fused buffer, aligned or not; a broadcast k."""
    b, n, h = 2, 150, 3
    width = 4 * h * d + 5 + (3 if offset == 0 else 0)  # rows 16-byte aligned only for offset 0
    fused = make((b, n, width), dtype, 1)
    part = lambda i: fused[:, :, offset + i * h * d: offset + (i + 1) * h * d].unflatten(2, (h, d))  # noqa: E731
    q, k, v, out = (part(i) for i in range(4))
    g = decays(h)
    want, state = mb.mhla_decay_forward(q.contiguous(), k.contiguous(), v.contiguous(), g, layout="bnhd")
    keep = fused.clone()
    got, state2 = mb.mhla_decay_forward(q, k, v, g, layout="bnhd", out=out)
    assert torch.equal(got, want) and torch.equal(state, state2)
    keep[:, :, offset + 3 * h * d: offset + 4 * h * d] = fused[:, :, offset + 3 * h * d: offset + 4 * h * d]
    assert torch.equal(keep, fused)  # nothing else was written
    do = make((b, n, h, d), dtype, 8)
    want = mb.mhla_decay_backward(q.contiguous(), k.contiguous(), v.contiguous(), g, do, layout="bnhd")
    grads = torch.full_like(fused, 7)
    gpart = lambda i: grads[:, :, offset + i * h * d: offset + (i + 1) * h * d].unflatten(2, (h, d))  # noqa: E731
    got = mb.mhla_decay_backward(q, k, v, g, do, layout="bnhd", dq=gpart(0), dk=gpart(1), dv=gpart(2))
    for x, y in zip(got[:3], want[:3]):
        assert torch.equal(x, y)
    assert (grads[:, :, :offset] == 7).all() and (grads[:, :, offset + 3 * h * d:] == 7).all()
    one = k[:, :, :1].expand(b, n, h, d)  # one key head for all
    want, _ = mb.mhla_decay_forward(q.contiguous(), one.contiguous(), v.contiguous(), g, layout="bnhd")
    got, _ = mb.mhla_decay_forward(q, one, v, g, layout="bnhd")
    assert torch.equal(got, want)
    st1, st2 = state.clone(), state.clone()
    a = mb.mhla_decay_step(q[:, 3], one[:, 3], v[:, 3], g, st1)
    c = mb.mhla_decay_step(q[:, 3].contiguous(), one[:, 3].contiguous(), v[:, 3].contiguous(), g, st2)
    assert torch.equal(a, c) and torch.equal(st1, st2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [100, 1500])
def test_state_in_place_and_repeatable(n, dtype):
    """Also the 64-entry rows' own kernel; long enough for several segments in the second case."""
    q, k, v, do = (make((1, 2, n, 64), dtype, i) for i in (1, 2, 3, 4))
    g = decays(2)
    state, ds = make((1, 2, 64, 64), "f32", 5), make((1, 2, 64, 64), "f32", 6)
    out, want = mb.mhla_decay_forward(q, k, v, g, state=state)
    mine = state.clone()
    out2, same = mb.mhla_decay_forward(q, k, v, g, state=mine, state_out=mine)
    assert same is mine and torch.equal(mine, want) and torch.equal(out, out2)
    a = mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds)
    b = mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds, dstate=ds)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_empty_problems():
    g = decays(2)
    q = torch.empty(3, 2, 0, 32, device="cuda", dtype=torch.bfloat16)
    state = make((3, 2, 32, 32), "f32", 1)
    out, s = mb.mhla_decay_forward(q, q, q, g, state=state)
    assert out.shape == q.shape and torch.equal(s, state)
    _, s = mb.mhla_decay_forward(q, q, q, g)
    assert not s.any()
    _, _, _, ds = mb.mhla_decay_backward(q, q, q, g, q, state=state, dstate_out=state)
    assert torch.equal(ds, state)
    q = torch.empty(0, 2, 5, 32, device="cuda")
    out, s = mb.mhla_decay_forward(q, q, q, g)
    assert out.numel() == 0 and s.numel() == 0


def test_other_stream_and_graph():
    q, k, v = (make((2, 4, 700, 64), "bf16", i) for i in (1, 2, 3))
    g = decays(4)
    want, state = mb.mhla_decay_forward(q, k, v, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, s = mb.mhla_decay_forward(q, k, v, g, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(s, state)
    out, st = torch.empty_like(want), torch.zeros_like(state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mb.mhla_decay_forward(q, k, v, g, out=out, state_out=st)
        mb.mhla_decay_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, st)
    graph.replay()
    mb.mhla_decay_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, state)
    assert torch.equal(out, want) and torch.equal(st, state)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(60, 64), (256, 64), (900, 64), (1400, 128)])
def test_backward_in_place_streams_and_graph(n, d, dtype):
    """The gradients' passes run side by side: same bits in place, on another stream, and from a graph."""
    q, k, v, do = (make((2, 3, n, d), dtype, i) for i in (1, 2, 3, 4))
    g, state, ds = decays(3), make((2, 3, d, d), "f32", 5), make((2, 3, d, d), "f32", 6)
    want = mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds)
    inplace = ds.clone()
    for x, y in zip(mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=inplace, dstate=inplace), want):
        assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    first, second = ([torch.zeros_like(x) for x in want] for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for into in (first, second):  # the side streams join one capture twice
            mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds, dq=into[0], dk=into[1], dv=into[2],
                                   dstate=into[3])
    for _ in range(2):
        graph.replay()
    for into in (first, second):
        for x, y in zip(into, want):
            assert torch.equal(x, y)


def test_backward_beside_a_capture():
    """A call on a stream of its own while the same thread captures another one stays out of the capture."""
    n, d = 100, 64  # one segment: no workspace
    q, k, v, do = (make((1, 2, n, d), "bf16", i) for i in (1, 2, 3, 4))
    g = decays(2)
    want = mb.mhla_decay_backward(q, k, v, g, do)
    into, beside = ([torch.zeros_like(x) for x in want[:3]] for _ in range(2))
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mb.mhla_decay_backward(q, k, v, g, do, dq=into[0], dk=into[1], dv=into[2])
        mb.mhla_decay_backward(q, k, v, g, do, dq=beside[0], dk=beside[1], dv=beside[2], stream=other)
    torch.cuda.synchronize()
    for x, y in zip(beside, want):
        assert torch.equal(x, y)
    for x in into:
        assert not x.any()
    graph.replay()
    for x, y in zip(into, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [70, 1000])
def test_unaligned_rows(n, d):
    """Rows that are not 16-byte aligned take another kernel, with another order of sums and the same bounds."""
    h = 2
    fused = make((1, n, 4 * h * d + 1), "bf16", 1)
    q, k, v, out = (fused[:, :, 1 + i * h * d: 1 + (i + 1) * h * d].unflatten(2, (h, d)) for i in range(4))
    g = decays(h)
    got, state = mb.mhla_decay_forward(q, k, v, g, layout="bnhd", scale=0.125, out=out)
    for j in range(h):
        check_forward(head(q, "bnhd", 0, j), head(k, "bnhd", 0, j), head(v, "bnhd", 0, j), float(g[j]),
                      head(got, "bnhd", 0, j), f64(state)[0, j], None, None, 0.125, "bf16", True)


def test_no_device_error_was_reported():
    """None of the kernels' bounded waits ran out above."""
    assert mb.mhla_device_status() == (0, 0)
