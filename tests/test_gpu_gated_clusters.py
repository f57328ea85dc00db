"""The gated recurrence in clusters of every size: three to seven CTAs, which do
not divide the tiles, rows in 16-byte, paired and single pieces, and lengths that
end before, inside and behind a cluster's round."""

import pytest
import torch
from test_gpu_gated import check, problem

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
