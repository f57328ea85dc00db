"""Workspaces, streams and graphs of the recurrent layer's operators and of the
normalised queries and keys."""

import pytest
import torch

from test_gpu_sequence_workspaces import Guarded
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu


def make(shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def gated(seed, dtype=torch.bfloat16):
    """Clusters (few channels) forward and backward, the marks formed by the backward call."""
    x, r, i, do = (make((1, 3000, 200), seed + j, dtype) for j in range(4))
    g, s, ds = -make((200,), seed, torch.float32).abs(), make((1, 200), 5, torch.float32), make((1, 200), 6, torch.float32)
    return lambda **k: mb.mhla_gated_backward(x, r, do, g, i, state=s, dstate_out=ds, **k)


def gated_wide(seed):
    """CTAs that run alone."""
    x, r, do = (make((40, 300, 520), seed + j) for j in range(3))
    _, _, marks = mb.mhla_gated_forward(x, r, keep=True)
    g = -make((520,), seed, torch.float32).abs()
    return lambda **k: mb.mhla_gated_backward(x, r, do, g, marks=marks, **k)


def qknorm(seed):
    q, k, dq, dk = (make((2, 700, h, 64), seed + h) for h in (8, 2, 8, 2))
    w, plan = make((64,), seed), mb.mhla_rotary_plan(64)
    return lambda **a: mb.mhla_qknorm_backward(dq, dk, q, k, plan, q_weight=w, k_weight=w, layout="bnhd", **a)


def conv(seed):
    x, do, w, b = make((3, 900, 200), seed), make((3, 900, 200), seed + 1), make((200, 4), seed + 2), make((200,), seed + 3)
    return lambda **k: mb.mhla_shortconv_backward(x, w, do, b, activation="silu", **k)


KINDS = [gated, gated_wide, qknorm, conv]


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", KINDS)
def test_workspace_bounds(kind, monkeypatch):
    """Exactly the bytes that are asked for, between bytes that nobody may write, and memory of the entry's own."""
    needs = []
    real = mb._Call.workspace
    monkeypatch.setattr(mb._Call, "workspace", lambda self, given: (needs.append(self.need), real(self, given))[1])
    call = kind(10)
    want = call()
    assert needs[-1] > 0
    ws = Guarded(needs[-1])
    assert same(call(workspace=ws.view), want)
    ws.check()
    short = torch.empty(needs[-1] - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(mb.MhlaError) as e:
        call(workspace=short)
    assert e.value.status == mb.MHLA_ERR_WORKSPACE
    monkeypatch.setattr(mb._Call, "workspace", lambda self, given: (None, 0))
    assert same(call(), want)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_calls_on_two_streams_at_once(kind, raw):
    problems = [kind(10), kind(20)]
    want = [p() for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for p, s in zip(problems, streams):
            got.append(p(stream=s.cuda_stream if raw else s))
    torch.cuda.synchronize()
    for i, results in enumerate(got):
        assert same(results, want[i % 2])


@pytest.mark.parametrize("kind", KINDS)
def test_two_graphs_share_a_workspace_in_turn(kind, monkeypatch):
    """Graphs captured with one workspace, replayed one after the other, on new inputs."""
    needs = []
    real = mb._Call.workspace
    monkeypatch.setattr(mb._Call, "workspace", lambda self, given: (needs.append(self.need), real(self, given))[1])
    problems = [kind(10), kind(20)]
    want = [p() for p in problems]
    ws = torch.empty(max(needs), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs, into = [torch.cuda.CUDAGraph() for _ in problems], []
    for p, g in zip(problems, graphs):
        with torch.cuda.graph(g):
            into.append(p(workspace=ws))
    for _ in range(2):
        for g, r, w in zip(graphs, into, want):
            for t in r:
                if t is not None:
                    t.zero_()
            g.replay()
            assert same(r, w)


def test_a_token_loop_in_a_graph():
    """Steps of the convolution, the recurrence and the rotation captured once and replayed for every token."""
    b, d, h, n = 3, 128, 2, 6
    x, r = make((b, n, d), 1), make((b, n, d), 2)
    w, g, plan = make((d, 4), 3), -make((d,), 4, torch.float32).abs(), mb.mhla_rotary_plan(64)
    conv, conv_state = mb.mhla_shortconv_forward(x, w, activation="silu")
    want, last, _ = mb.mhla_gated_forward(conv, r, g)
    rotated, _ = mb.mhla_qknorm_forward(want.unflatten(2, (h, 64)), None, plan, layout="bnhd")

    xt, rt, pos = x[:, 0].clone(), r[:, 0].clone(), torch.zeros(b, 1, dtype=torch.int64, device="cuda")
    rows, state = torch.zeros(b, 3, d, dtype=x.dtype, device="cuda"), torch.zeros(b, d, device="cuda")

    def token():
        y = mb.mhla_gated_step(mb.mhla_shortconv_step(xt, w, rows, activation="silu"), rt, state, g)
        return y, mb.mhla_qknorm_forward(y.unflatten(1, (h, 64))[:, None], None, plan, positions=pos, layout="bnhd")[0]

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = token()
    rows.zero_()
    state.zero_()
    for t in range(n):
        xt.copy_(x[:, t])
        rt.copy_(r[:, t])
        pos.fill_(t)
        graph.replay()
        # the states' float32 sums in another order, then one bf16 step
        assert ((y.float() - want[:, t].float()).abs() <= 2.0 ** -7 * want[:, t].float().abs() + 1e-6).all()
        # a step of y's, and one of the result
        close = (z[:, 0].float() - rotated[:, t].float()).abs()
        size = rotated[:, t].float().abs()
        assert (close <= 2.0 ** -6 * (size + size.roll(32, -1))).all()
    assert torch.equal(rows, conv_state)
    assert ((state - last).abs() <= 1e-5 * last.abs() + 1e-6).all()


def test_no_device_error_was_reported():
    assert mb.mhla_device_status() == (0, 0)
