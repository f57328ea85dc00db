"""Offsets beyond 32 bits, many short sequences and very wide rows for the
recurrent layer's operators and the normalised queries and keys."""

import pytest
import torch

from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

TOKEN = 1 << 27  # elements from token to token: the 17th lies behind 2^31


@pytest.fixture(scope="module")
def far():
    """A view [1, 20, 64] of bf16 whose tokens are far apart, over 5 GB."""
    memory = torch.empty(20 * TOKEN, dtype=torch.bfloat16, device="cuda")
    yield memory.as_strided((1, 20, 64), (20 * TOKEN, TOKEN, 1))
    del memory
    torch.cuda.empty_cache()


def make(shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def test_far_tokens_of_the_recurrence(far):
    x, r, do = make((1, 20, 64), 1), make((1, 20, 64), 2), make((1, 20, 64), 3)
    want = mb.mhla_gated_forward(x, r, keep=True)
    grads = mb.mhla_gated_backward(x, r, do, marks=want[2])
    far.copy_(x)
    assert all(torch.equal(a, b) for a, b in zip(mb.mhla_gated_forward(far, r, keep=True), want))
    assert torch.equal(mb.mhla_gated_backward(far, r, do, marks=want[2])[1], grads[1])
    mb.mhla_gated_forward(x, r, out=far)
    assert torch.equal(far, want[0])
    mb.mhla_gated_backward(x, r, do, marks=want[2], dx=far)
    assert torch.equal(far, grads[0])


def test_far_tokens_of_the_convolution(far):
    x, do, w = make((1, 20, 64), 1), make((1, 20, 64), 2), make((64, 4), 3)
    want = mb.mhla_shortconv_forward(x, w, activation="silu")
    grads = mb.mhla_shortconv_backward(x, w, do, activation="silu")
    far.copy_(x)
    assert all(torch.equal(a, b) for a, b in zip(mb.mhla_shortconv_forward(far, w, activation="silu"), want))
    assert all(torch.equal(a, b) for a, b in zip(mb.mhla_shortconv_backward(far, w, do, activation="silu")[:2], grads))
    mb.mhla_shortconv_forward(x, w, activation="silu", out=far)
    assert torch.equal(far, want[0])
    mb.mhla_shortconv_backward(x, w, do, activation="silu", dx=far)
    assert torch.equal(far, grads[0])


def test_far_tokens_of_queries(far):
    q, dq, plan = make((1, 20, 1, 64), 1), make((1, 20, 1, 64), 2), mb.mhla_rotary_plan(64)
    want, _ = mb.mhla_qknorm_forward(q, None, plan, layout="bnhd")
    grads = mb.mhla_qknorm_backward(dq, None, q, None, plan, layout="bnhd")
    view = far[:, :, None]
    view.copy_(q)
    assert torch.equal(mb.mhla_qknorm_forward(view, None, plan, layout="bnhd")[0], want)
    got = mb.mhla_qknorm_backward(dq, None, view, None, plan, layout="bnhd", dq=view)
    assert torch.equal(view, grads[0]) and torch.equal(got[2], grads[2])


def test_many_sequences_of_a_few_tokens():
    b, n, d = 70001, 3, 8
    x, r, w = make((b, n, d), 1), make((b, n, d), 2), make((d, 4), 3)
    out, last = mb.mhla_shortconv_forward(x, w)
    y, state, marks = mb.mhla_gated_forward(out, r, keep=True)
    dx, dr, _, _, _ = mb.mhla_gated_backward(out, r, y, marks=marks)
    dc, dw, _, _ = mb.mhla_shortconv_backward(x, w, dx)
    q, _ = mb.mhla_qknorm_forward(y.view(b, n, 1, d), None, mb.mhla_rotary_plan(d), layout="bnhd")
    at = torch.tensor([0, 1, 33333, 65535, 65536, 70000]).cuda()
    few = lambda t: t[at].contiguous()  # noqa: E731
    o2, l2 = mb.mhla_shortconv_forward(few(x), w)
    y2, s2, m2 = mb.mhla_gated_forward(o2, few(r), keep=True)
    dx2, dr2, _, _, _ = mb.mhla_gated_backward(o2, few(r), y2, marks=m2)
    q2, _ = mb.mhla_qknorm_forward(y2.view(6, n, 1, d), None, mb.mhla_rotary_plan(d), layout="bnhd")
    for big, small in ((out, o2), (last, l2), (y, y2), (state, s2), (dx, dx2), (dr, dr2), (q, q2),
                       (dc, mb.mhla_shortconv_backward(few(x), w, dx2)[0])):
        assert torch.equal(big[at], small)
    want = torch.einsum("btd,btd->d", dx.double(), x.double())  # the last tap meets the token itself
    size = torch.einsum("btd,btd->d", dx.double().abs(), x.double().abs())
    assert ((dw[:, 3].double() - want).abs() <= 256 * 2.0 ** -24 * size).all()


def test_wide_rows():
    b, n, d = 1, 40, 70000
    x, r, w = make((b, n, d), 1), make((b, n, d), 2), make((d, 2), 3)
    g = -make((d,), 4, torch.float32).abs()
    part = slice(69888, 70000)  # starts at a multiple of 64
    y, state, marks = mb.mhla_gated_forward(x, r, g, keep=True)
    cut = lambda t: t[..., part].contiguous()  # noqa: E731
    y2, s2, m2 = mb.mhla_gated_forward(cut(x), cut(r), cut(g), keep=True)
    assert torch.equal(cut(marks), m2) and torch.equal(cut(y), y2) and torch.equal(cut(state), s2)
    full = mb.mhla_gated_backward(x, r, y, g, marks=marks)
    few = mb.mhla_gated_backward(cut(x), cut(r), y2, cut(g), marks=m2)
    assert all(torch.equal(cut(a), b) for a, b in zip(full[:2], few[:2]))
    out, _ = mb.mhla_shortconv_forward(x, w)
    assert torch.equal(cut(out), mb.mhla_shortconv_forward(cut(x), w[part].contiguous())[0])


def test_no_device_error_was_reported():
    assert mb.mhla_device_status() == (0, 0)


def test_more_sequences_than_a_grid_is_high():
    # above 8 x 65535 sequences of one segment, 8 of them a CTA; small whole numbers,
    # whose sums are exact
    B, D = 530_000, 128
    gen = torch.Generator().manual_seed(5)
    x = torch.randint(-2, 3, (B, 1, D), generator=gen).to(torch.bfloat16).cuda()
    do = torch.randint(-1, 2, (B, 1, D), generator=gen).to(torch.bfloat16).cuda()
    w = torch.randint(-2, 3, (D, 4), generator=gen).to(torch.bfloat16).cuda()
    out, _ = mb.mhla_shortconv_forward(x, w)
    assert torch.equal(out, x * w[:, 3])
    db = torch.empty(D, device="cuda")
    dx, dw, _, _ = mb.mhla_shortconv_backward(x, w, do, dbias=db)
    assert torch.equal(dx, do * w[:, 3])
    assert torch.equal(db, do.float().sum((0, 1)))
    assert torch.equal(dw[:, 3], (do.float() * x.float()).sum((0, 1))) and not dw[:, :3].any()
