"""Where the C entries of the sequence operators keep their scratch: memory of
their own (a NULL workspace), or the caller's, whose bounds they keep."""

import pytest
import torch

from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

GUARD = 4096


def make(shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


class Guarded:
    """A workspace of exactly the bytes that are asked for, between bytes that nobody may write."""

    def __init__(self, need):
        self.need = need
        self.all = torch.full((need + 2 * GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
        self.view = self.all[GUARD: GUARD + need]

    def check(self):
        assert (self.all[:GUARD] == 0x5A).all() and (self.all[GUARD + self.need:] == 0x5A).all()
        assert not (self.view == 0x5A).all()  # it was used


SHAPES = [  # tokens, dk, dv, dtype, first element of q's and k's rows
    (2500, 64, 64, torch.bfloat16, 0), (2500, 128, 128, torch.bfloat16, 0), (2500, 128, 64, torch.bfloat16, 0),
    (2500, 64, 128, torch.bfloat16, 0), (2500, 32, 64, torch.bfloat16, 0), (2500, 64, 64, torch.bfloat16, 1),
    (1300, 64, 64, torch.float32, 0), (1300, 128, 32, torch.float32, 1)]


def problem(n, dk, dv, dtype, first):
    q, k = (make((2, 3, n, dk + first), i, dtype)[..., first:] for i in (1, 2))
    v, do = make((2, 3, n, dv), 3, dtype), make((2, 3, n, dv), 4, dtype)
    state, ds = make((2, 3, dk, dv), 5, torch.float32), make((2, 3, dk, dv), 6, torch.float32)
    return q, k, v, do, torch.full((3,), -0.01, device="cuda"), state, ds


def forward_entry(call, q, k, v, g, state, out, state_out):
    return call.call(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), None, state.data_ptr(), call.ref,
                     out.data_ptr(), mb._ptr(state_out), None, 0, call.stream())


@pytest.mark.parametrize("n,dk,dv,dtype,first", SHAPES)
def test_decay_forward(n, dk, dv, dtype, first):
    q, k, v, _, g, state, _ = problem(n, dk, dv, dtype, first)
    want = mb.mhla_decay_forward(q, k, v, g, state=state)
    call = mb._decay_forward_call(q, k, v, g, state, None, 1.0, "bhnd", "auto", None, None)
    assert call.need > 0
    ws = Guarded(call.need)
    got = mb.mhla_decay_forward(q, k, v, g, state=state, workspace=ws.view)
    ws.check()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    out, last = torch.empty_like(want[0]), torch.empty_like(want[1])
    assert forward_entry(call, q, k, v, g, state, out, last) == mb.MHLA_OK
    assert torch.equal(out, want[0]) and torch.equal(last, want[1])
    # No final state: pairs of bf16 hold the states' addends in between (off by
    # 2^-16), so the roundings of the state's copy and of the output may fall the
    # other way, a whole step of 2^-7 each.
    out.zero_()
    assert forward_entry(call, q, k, v, g, state, out, None) == mb.MHLA_OK
    if dtype == torch.float32:
        assert torch.equal(out, want[0])
    else:
        sums, _ = mb.mhla_decay_forward(*(t.abs().float() for t in (q, k, v)), g, state=state.abs())
        assert ((out.float() - want[0].float()).abs() <= 2.0 ** -7 * (want[0].float().abs() + sums)).all()


@pytest.mark.parametrize("n,dk,dv,dtype,first", SHAPES)
def test_decay_backward(n, dk, dv, dtype, first):
    q, k, v, do, g, state, ds = problem(n, dk, dv, dtype, first)
    want = mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds)
    call = mb._decay_backward_call(q, k, v, g, do, state, ds, None, 1.0, "bhnd", "auto", None, None, None, None)
    assert call.need > 0
    ws = Guarded(call.need)
    got = mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds, workspace=ws.view)
    ws.check()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    into = [torch.empty_like(x) for x in want]
    args = (q, k, v, g, None, state, do, ds)
    status = call.call(*(mb._ptr(t) for t in args), call.ref, *(t.data_ptr() for t in into), None, 0, call.stream())
    assert status == mb.MHLA_OK
    assert all(torch.equal(x, y) for x, y in zip(into, want))


@pytest.mark.parametrize("rows,cols,dtype,first", [
    (3000, 512, torch.bfloat16, 0), (700, 1000, torch.bfloat16, 1), (5, 64, torch.float32, 0), (300, 20000, torch.bfloat16, 0),
    (300, 9000, torch.float32, 1)])
def test_layernorm_backward(rows, cols, dtype, first):
    x, dy = make((rows, cols + first), 1, dtype)[:, first:], make((rows, cols), 2, dtype)
    _, mean, rstd = mb.mhla_layernorm_forward(x)
    want = mb.mhla_layernorm_backward(dy, x, mean, rstd)
    call = mb._norm_backward_call(dy, x, mean, rstd, None, None, None, None, True)
    ws = Guarded(call.need)
    got = mb.mhla_layernorm_backward(dy, x, mean, rstd, workspace=ws.view)
    ws.check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    into = [torch.empty_like(t) for t in want]
    status = call.call(dy.data_ptr(), x.data_ptr(), None, mean.data_ptr(), rstd.data_ptr(), call.ref,
                       *(t.data_ptr() for t in into), None, 0, call.stream())
    assert status == mb.MHLA_OK
    assert all(torch.equal(a, b) for a, b in zip(into, want))


def test_scratch_of_the_entries_inside_a_graph():
    q, k, v, _, g, state, _ = problem(2500, 64, 64, torch.bfloat16, 0)
    want = mb.mhla_decay_forward(q, k, v, g, state=state)
    call = mb._decay_forward_call(q, k, v, g, state, None, 1.0, "bhnd", "auto", None, None)
    out, last = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert forward_entry(call, q, k, v, g, state, out, last) == mb.MHLA_OK
    for _ in range(2):
        graph.replay()
    assert torch.equal(out, want[0]) and torch.equal(last, want[1])


def test_no_device_error_was_reported():
    assert mb.mhla_device_status() == (0, 0)
