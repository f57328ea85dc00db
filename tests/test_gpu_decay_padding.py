"""A short sequence on a large kept state, alone and padded to the length of a
longer neighbour: which roundings its outputs take (include/mhla.h)."""

import pytest
import torch

from test_gpu_decay import check_forward, decays, f64, make
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu

PADDED = [64, 127, 128, 300, 1300]


def padded(t, n):
    out = torch.full(t.shape[:2] + (n, t.shape[3]), float("nan"), dtype=t.dtype, device=t.device)
    out[:, :, : t.shape[2]] = t
    return out


@pytest.mark.parametrize("variant,dtype", [("tensor", "bf16"), ("simt", "bf16"), ("simt", "f32")])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 5, 64])
def test_padding(m, d, variant, dtype):
    q, k, v = (make((1, 2, m, d), dtype, i) for i in (1, 2, 3))
    state, g = make((1, 2, d, d), "f32", 4, 1000.0), decays(2)
    lens = torch.tensor([m], dtype=torch.int32).cuda()
    results = []
    for n in PADDED:
        out, last = mb.mhla_decay_forward(padded(q, n), padded(k, n), padded(v, n), g, state=state, lengths=lens,
                                          variant=variant)
        assert not out[:, :, m:].any()
        for j in range(2):
            check_forward(*(f64(padded(t, n).nan_to_num())[0, j] for t in (q, k, v)), float(g[j]), f64(out)[0, j],
                          f64(last)[0, j], f64(state)[0, j], m, 1.0, dtype, variant == "tensor")
        results.append((out[:, :, :m], last))
    for out, last in results[1:]:
        if variant == "simt":  # no rounding of an operand: the same at every padded length
            assert torch.equal(out, results[0][0]) and torch.equal(last, results[0][1])
            continue
        # sums of magnitudes of a state's entry: 16 bits or more of every addend, at every padded length
        size = (state.abs() + m * k.abs().amax().float() * v.abs().amax().float())
        assert ((last - results[0][1]).abs() <= 2 * 2.0 ** -16 * size).all()
    if variant == "tensor":  # below 128 tokens one chunk with operands of 16 bits, whatever the padding
        assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
