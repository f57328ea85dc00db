"""The states that the backward call forms where it is given no marks: the same bits
as those of the forward call, for every way that rows are fetched, CTAs alone and
clusters, and lengths that leave warps without tokens."""

import pytest
import torch
from test_gpu_gated import COMBOS, make, problem

from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,n,d", [(40, 900, 520), (40, 900, 522), (40, 900, 521), (1, 5000, 200), (1, 5000, 130),
                                   (2, 3000, 65)])
@pytest.mark.parametrize("ragged", [False, True])
def test_formed_marks(b, n, d, ragged, dtype):
    p = problem(b, n, d, dtype, "decay", True, True)
    lengths = torch.tensor([(n - 37 * i) % (n + 1) for i in range(b)], dtype=torch.int32).cuda() if ragged else None
    dout = make((b, n, d), 60, dtype)
    _, _, marks = mb.mhla_gated_forward(**p, lengths=lengths, keep=True)
    args = (p["x"], p["gate"], dout, p["log_decay"], p["input_gate"], p["state"])
    want = mb.mhla_gated_backward(*args, marks=marks, lengths=lengths)
    for _ in range(4):
        assert all(torch.equal(a, w) for a, w in zip(mb.mhla_gated_backward(*args, lengths=lengths), want))


@pytest.mark.parametrize("kind,scale,in_gate", COMBOS)
def test_formed_marks_of_every_kind(kind, scale, in_gate):
    p = problem(3, 700, 70, "bf16", kind, in_gate, True)
    dout = make((3, 700, 70), 60, "bf16")
    marks = mb.mhla_gated_forward(**p, scale=scale, keep=True)[2]
    args = (p["x"], p["gate"], dout, p["log_decay"], p["input_gate"], p["state"])
    want = mb.mhla_gated_backward(*args, marks=marks, scale=scale)
    got = mb.mhla_gated_backward(*args, scale=scale)
    assert all((a is None and w is None) or torch.equal(a, w) for a, w in zip(got, want))
