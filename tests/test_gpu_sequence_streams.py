"""Calls on streams of their own, several at a time."""

import pytest
import torch

from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu


def make(shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


def decay_forward(seed):
    q, k, v = (make((1, 4, 2500, 64), seed + i) for i in range(3))
    g = torch.full((4,), -0.01, device="cuda")
    return lambda **kw: mb.mhla_decay_forward(q, k, v, g, **kw)


def decay_backward(seed):
    q, k, v, do = (make((1, 4, 2500, 64), seed + i) for i in range(4))
    g, s = torch.full((4,), -0.01, device="cuda"), make((1, 4, 64, 64), seed, torch.float32)
    return lambda **kw: mb.mhla_decay_backward(q, k, v, g, do, state=s, **kw)


def norm_backward(seed):
    x, dy = make((3000, 512), seed), make((3000, 512), seed + 1)
    _, mean, rstd = mb.mhla_layernorm_forward(x)
    return lambda **kw: mb.mhla_layernorm_backward(dy, x, mean, rstd, **kw)


def block_attention(seed):
    q, k, v, do = (make((1, 4, 1024, 64), seed + i) for i in range(4))
    mc = torch.softmax(make((16, 16), seed, torch.float32), 1)
    args = ((1, 32, 32), (1, 8, 8))
    return lambda **kw: (mb.mhla_forward(q, k, v, mc, *args, **kw),) + mb.mhla_backward(q, k, v, mc, do, *args, **kw)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("kind", [decay_forward, decay_backward, norm_backward, block_attention])
def test_calls_on_two_streams_at_once(kind, raw):
    """Each has a workspace of its own, although neither waits for the other, and nor does the current stream."""
    problems = [kind(10), kind(20)]
    want = [p() for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    got, filled = [], []
    for _ in range(10):
        for p, s in zip(problems, streams):
            got.append(p(stream=s.cuda_stream if raw else s))
        filled.append(torch.full((1 << 20,), 7.0, device="cuda"))  # on the current stream
    torch.cuda.synchronize()
    for i, results in enumerate(got):
        for x, y in zip(results, want[i % 2]):
            assert torch.equal(x, y)
    assert all((t == 7.0).all() for t in filled)


def test_results_may_be_dropped_on_the_current_stream():
    problem = norm_backward(30)
    want, side = problem(), torch.cuda.Stream()
    for _ in range(20):
        side.wait_stream(torch.cuda.current_stream())
        got = problem(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        del got, x


def test_gradients_on_one_stream_do_not_wait_for_another():
    """A stream that is held up holds up none of the others, whichever share its hardware queue."""
    problem = decay_backward(50)
    want, held = problem(), torch.cuda.Stream()
    others = [torch.cuda.Stream() for _ in range(6)]
    for s in [held] + others:
        problem(stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(held):
        torch.cuda._sleep(2_000_000_000)  # about a second
    first = problem(stream=held)
    done = torch.cuda.Event()
    done.record(held)
    got, ends = [], []
    for s in others:
        got.append(problem(stream=s))
        ends.append(torch.cuda.Event())
        ends[-1].record(s)
    early = False
    while not early and not done.query():
        early = any(e.query() for e in ends)
        early = early and not done.query()
    torch.cuda.synchronize()
    assert early
    for results in got + [first]:
        for x, y in zip(results, want):
            assert torch.equal(x, y)


def test_gradients_on_more_streams_than_have_side_streams():
    problem = decay_backward(60)
    want = problem()
    streams = [torch.cuda.Stream() for _ in range(24)]
    assert len({s.cuda_stream for s in streams}) > 16
    torch.cuda.synchronize()
    for _ in range(2):
        got = [problem(stream=s) for s in streams]
        torch.cuda.synchronize()
        for results in got:
            for x, y in zip(results, want):
                assert torch.equal(x, y)


def test_gradients_captured_on_two_streams_in_turn():
    problems = [decay_backward(70), decay_backward(80)]
    want = [p() for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    into = [tuple(torch.zeros_like(x) for x in w) for w in want]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in problems]
    for p, s, g, t in zip(problems, streams, graphs, into):
        with torch.cuda.graph(g, stream=s):
            p(dq=t[0], dk=t[1], dv=t[2], dstate=t[3])
    for g in graphs:
        g.replay()
    for p, s, w in zip(problems, streams, want):  # the side streams are free again
        for x, y in zip(p(stream=s), w):
            torch.cuda.current_stream().wait_stream(s)
            assert torch.equal(x, y)
    for t, w in zip(into, want):
        for x, y in zip(t, w):
            assert torch.equal(x, y)


def test_the_default_stream_by_handle():
    problem = norm_backward(40)
    want = problem()
    for handle in (0, 1):
        for x, y in zip(problem(stream=handle), want):
            assert torch.equal(x, y)


def test_no_device_error_was_reported():
    assert mb.mhla_device_status() == (0, 0)
