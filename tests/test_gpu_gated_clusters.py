"""The gated recurrence in clusters of every size: three to seven CTAs, which do
not divide the tiles, rows in 16-byte, paired and single pieces, and lengths that
end before, inside and behind a cluster's round."""

import pytest
import torch
from test_gpu_gated import check, problem

from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,n,d,dtype", [
    (1, 1300, 64, "bf16"),   # 6 CTAs forward, 7 backward
    (5, 900, 1024, "bf16"),  # 3 and 3
    (3, 900, 1010, "bf16"),  # 4 and 5, pairs
    (1, 1300, 65, "bf16"),   # 6 and 7, single elements
    (3, 900, 321, "f32"),    # 5 and 5, single elements
    (3, 1300, 322, "f32"),   # 6 and 6, pairs
    (5, 500, 500, "f32"),    # 3 and 3
    (1, 1300, 128, "f32"),   # 7 and 7
])
@pytest.mark.parametrize("ragged", [False, True])
def test_sizes(b, n, d, dtype, ragged):
    lengths = torch.tensor([n // 3, n, 0, 65, n - 1][:b], dtype=torch.int32).cuda() if ragged else None
    check(problem(b, n, d, dtype, "decay", True, ragged), dtype, "norm", lengths, ragged)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,n,d", [(3, 333, 65), (2, 200, 130), (40, 70, 321), (1, 1300, 63)])
def test_row_starts_do_not_change_results(b, n, d, dtype):
    """The same rows at single elements, at pairs (with a lone last column where d is odd) and at 16
    bytes, each time with columns behind them that have to stay."""
    lengths = torch.tensor([n - i % 7 for i in range(b)], dtype=torch.int32).cuda()
    decay = -torch.rand(d, generator=torch.Generator().manual_seed(3)).cuda()
    values = [torch.randn(b, n, d, generator=torch.Generator().manual_seed(i)).to(dtype).cuda() for i in range(4)]
    want = None
    for width, first in ((d + 16 + d % 2, 1), (d + 18 + d % 2, 2), ((d + 15) // 8 * 8 + 8, 8)):
        def place(t=None):
            memory = torch.full((b, n, width + first), 7.0, dtype=dtype, device="cuda")[:, :, :width]
            view = memory[:, :, first:first + d]
            if t is not None:
                view.copy_(t)
            return memory, view

        x, r, i, do = (place(t)[1] for t in values)
        (mo, out), (mx, dx), (mr, dr), (mi, di) = (place() for _ in range(4))
        _, state, marks = mb.mhla_gated_forward(x, r, decay, i, lengths=lengths, out=out, keep=True)
        grads = mb.mhla_gated_backward(x, r, do, decay, i, marks=marks, lengths=lengths, dx=dx, dgate=dr, dinput_gate=di)
        got = [t.clone() for t in (out, state, marks, dx, dr, di, grads[3])]
        for memory, view in ((mo, out), (mx, dx), (mr, dr), (mi, di)):
            view.fill_(7.0)
            assert (memory == 7.0).all()
        if want is None:
            want = got
        assert all(torch.equal(a, t) for a, t in zip(got, want)), (width, first)
