"""Decayed linear attention at the sizes where its plans use many CTAs, long
segments and several waves: every head against the recurrence in float64, and
the kernels that the sizes are meant for (read from a captured graph).

Bounds are those of the small shapes, entry by entry: with half = 2^-8 for one
rounding to bf16, the output's (half |o|), the decayed scores' and the operand
copy of the state's (half (1 + half) of |P| |Z| and |X| |S|), pairs of bf16 for
the state's addends (2^-16 a term), and (terms + 32) 2^-24 of the sum of
magnitudes for float32 sums."""

import re

import pytest
import torch

from token_level_head_phi_gb300 import binding as mb

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:DEBUG")]

HALF, EPS = 2.0 ** -8, 2.0 ** -24


def make(shape, seed, dtype=torch.bfloat16, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def decays(h):
    return torch.log1p(-torch.exp2(-torch.linspace(1, 9, h, dtype=torch.float64))).float().cuda()


def kernels(call, tmp_path):
    """Names of the attention's kernels that the call launches."""
    path = tmp_path / "graph.dot"
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    graph.debug_dump(str(path))
    return set(re.findall(r"decay_[a-z_]*kernel(?:I(?:L[bi]\d+E|f|13__nv_bfloat16)+E)?", path.read_text()))


# ------------------------------------------------------- float64, all heads


def one_pass(x, y, z, lam, state, last_first, read, update):
    """The recurrence over [units, tokens, .]: (o, final state, |x| times the largest states so far).

    First token first, a token reads the state with itself in it; last token
    first, the state is a gradient that decays behind the token."""
    s = state.clone()
    top = s.abs()
    o, copies = (x.new_zeros(x.shape[0], x.shape[1], z.shape[2]) for _ in range(2))
    for i in reversed(range(x.shape[1])) if last_first else range(x.shape[1]):
        xi = x[:, i, None]
        if not last_first:
            copies[:, i] = (xi.abs() @ top)[:, 0]
            s = lam * s
        s = s + update * y[:, i, :, None] * z[:, i, None]
        top = torch.maximum(top, s.abs())
        o[:, i] = (xi @ s)[:, 0]
        if last_first:
            copies[:, i] = (xi.abs() @ top)[:, 0]
            s = lam * s
    return o * read, s, copies * read


def bounded(x, y, z, lam, state, last_first, read, update, score):
    """(o, bound of o, state, its bound)."""
    n, d = x.shape[1], max(x.shape[2], z.shape[2])
    o, s, copies = one_pass(x, y, z, lam, state, last_first, read, update)
    sums, abs_s, _ = one_pass(x.abs(), y.abs(), z.abs(), lam, state.abs(), last_first, read, update)
    t = torch.arange(n, device="cuda", dtype=torch.float64)
    dist = t[:, None] - t[None] if not last_first else t[None] - t[:, None]
    p = (x @ y.transpose(1, 2)).abs_()
    p *= torch.where(dist >= 0, lam ** dist.clamp(min=0), 0.0)
    scores = score * (p @ z.abs())
    sum_bound = (n + 2 * d + 32) * EPS
    bound = (sum_bound + 2.0 ** -16) * sums + HALF * o.abs() + (1 + HALF) * HALF * (scores + copies) + 1e-30
    return o, bound, s, (2.0 ** -16 + sum_bound) * abs_s + 1e-30


def near(got, want, bound, what):
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if not got.numel():
        return
    over = ((got.double() - want).abs() - bound).max().item()
    assert over <= 0, f"{what}: {over:.3e} over its bound"


def ragged(b, n):
    """Whole, a part, none, one token, and the ends of chunks."""
    return [n, n - n // 6 + 3, 0, 1, n // 2, 128, n - 1, 127][:b] + [(n - 37 * i) % n for i in range(8, b)]


def both(cases):
    """With and without lengths; the long ones, whose references take seconds, with lengths only (the first is whole)."""
    return [c + (w,) for c in cases for w in ((True,) if c[2] >= 3000 else (False, True))]


FORWARD = [  # batch, heads, tokens, dk, dv, kernels
    (3, 17, 2048, 64, 128, ["decay_tc_state_kernelILb0ELi1ELi1EE", "decay_tc_kernelILb1ELb0EE"]),  # 714 CTAs of states
    (20, 20, 300, 64, 64, ["decay_tc_kernelILb1ELb0EE"]),                 # two waves of one segment
    (2, 76, 600, 128, 128, ["decay_tc_wide_kernelILb0ELi2EE"]),           # 128 columns, five chunks
    (3, 10, 4000, 128, 128, ["decay_tc_wide_kernelILb0ELi2EE", "decay_tc_state_kernelILb0ELi2ELi2EE"]),  # four chunks
    (4, 19, 2000, 128, 128, ["decay_tc_wide_kernelILb0ELi1EE"]),          # 64 columns, sixteen chunks
    (3, 4, 4000, 128, 64, ["decay_tc_wide_kernelILb0ELi1EE", "decay_tc_state_kernelILb0ELi2ELi1EE"]),
    (8, 64, 300, 32, 64, ["decay_mma_kernelILi32ELi64ELb1ELb0EE"]),       # two waves
]


@pytest.mark.parametrize("b,h,n,dk,dv,want,with_lengths", both(FORWARD))
def test_forward(b, h, n, dk, dv, want, with_lengths, tmp_path):
    q, k, v = make((b, n, h, dk), 1), make((b, n, h, dk), 2), make((b, n, h, dv), 3)
    g, state, scale = decays(h), make((b, h, dk, dv), 4, torch.float32, 3.0), 0.125
    lengths = ragged(b, n) if with_lengths else [n] * b
    for i, m in enumerate(lengths):
        for t in (q, k, v):
            t[i, m:] = float("nan")  # never used
    lens = torch.tensor(lengths, dtype=torch.int32).cuda() if with_lengths else None
    call = lambda: mb.mhla_decay_forward(q, k, v, g, state=state, lengths=lens, scale=scale, layout="bnhd")  # noqa: E731
    assert set(want) <= kernels(call, tmp_path)
    out, last = call()
    lam = g.double().exp()[:, None, None]
    for i, m in enumerate(lengths):
        assert not out[i, m:].any()
        x, y, z = (t[i, :m].transpose(0, 1).double() for t in (q, k, v))
        o, o_bound, s, s_bound = bounded(x, y, z, lam, state[i].double(), False, scale, 1.0, scale)
        near(out[i, :m].transpose(0, 1), o, o_bound, f"out of sequence {i}")
        near(last[i], s, s_bound, f"state of sequence {i}")


BACKWARD = [
    (3, 17, 3584, 64, 128, ["decay_tc_state_kernelILb1ELi1ELi1EE", "decay_tc_kernelILb1ELb1EE"]),  # 612 CTAs of states
    (2, 64, 700, 64, 64, ["decay_tc_kernelILb1ELb1EE", "decay_tc_kernelILb1ELb0EE"]),
    (2, 76, 600, 128, 128, ["decay_tc_wide_kernelILb1ELi2EE", "decay_tc_wide_kernelILb0ELi2EE"]),
    (3, 10, 4000, 128, 128, ["decay_tc_wide_kernelILb1ELi2EE", "decay_tc_state_kernelILb1ELi2ELi2EE",
                             "decay_tc_wide_kernelILb0ELi2EE", "decay_tc_state_kernelILb0ELi2ELi2EE"]),
    (4, 32, 300, 32, 64, ["decay_mma_kernelILi32ELi64ELb1ELb0EE", "decay_mma_kernelILi64ELi32ELb1ELb0EE"]),
]


@pytest.mark.parametrize("b,h,n,dk,dv,want,with_lengths", both(BACKWARD))
def test_backward(b, h, n, dk, dv, want, with_lengths, tmp_path):
    q, k, v, do = make((b, n, h, dk), 1), make((b, n, h, dk), 2), make((b, n, h, dv), 3), make((b, n, h, dv), 5)
    g, scale = decays(h), 0.125
    state, ds = make((b, h, dk, dv), 4, torch.float32, 3.0), make((b, h, dk, dv), 6, torch.float32)
    lengths = ragged(b, n) if with_lengths else [n] * b
    for i, m in enumerate(lengths):
        for t in (q, k, v, do):
            t[i, m:] = float("inf")
    lens = torch.tensor(lengths, dtype=torch.int32).cuda() if with_lengths else None
    call = lambda: mb.mhla_decay_backward(q, k, v, g, do, state=state, dstate_out=ds, lengths=lens,  # noqa: E731
                                          scale=scale, layout="bnhd")
    assert set(want) <= kernels(call, tmp_path)
    got = call()
    lam = g.double().exp()[:, None, None]
    for i, m in enumerate(lengths):
        for t in got[:3]:
            assert not t[i, m:].any()
        qq, kk, vv, dd = (t[i, :m].transpose(0, 1).double() for t in (q, k, v, do))
        s0, s1 = state[i].double(), ds[i].double()
        passes = {"dq": (dd, vv, kk, lam, s0.transpose(1, 2), False, scale, 1.0, scale),
                  "dk": (vv, dd, qq, lam, s1.transpose(1, 2), True, 1.0, scale, scale),
                  "dv": (kk, qq, dd, lam, s1, True, 1.0, scale, scale)}
        for t, (name, args) in zip(got, passes.items()):
            o, o_bound, s, s_bound = bounded(*args)
            near(t[i, :m].transpose(0, 1), o, o_bound, f"{name} of sequence {i}")
        near(got[3][i], s, s_bound, f"dstate of sequence {i}")  # of dv's pass


def test_no_device_error_was_reported():
    assert mb.mhla_device_status() == (0, 0)
