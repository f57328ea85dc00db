"""The hybrid example's gradients in bfloat16 against the same model in float64.

On its way through two layers and back a value is rounded to bfloat16 about 48 times
(weights, projections, norms, the operators' results, products, sums), each time by at
most 2^-8 of its size: 48 * 2^-8 of a gradient's size where no error grows.  A gradient
that is missing, of the wrong sign or off by a factor of two is off by 1 / 2 or more."""

import torch
import pytest

from test_gpu_hybrid_model import example, plain_loss  # noqa: F401

pytestmark = pytest.mark.gpu


def test_gradients(example):  # noqa: F811
    model = example.HybridModel(dtype=torch.bfloat16, layers=2)
    with torch.no_grad():  # weights that matter
        for name in list(model.params):
            if name.endswith((".q.w", ".k.w", "conv.b")):
                model.params[name] += 0.3 * torch.randn(model.params[name].shape, generator=torch.Generator().manual_seed(3)).cuda()
    tokens = example.motif_batch(4, 140, 64, torch.Generator().manual_seed(2))
    loss, grads = model.loss_and_grads(tokens)
    params = {k: v.double().requires_grad_() for k, v in model.params.items()}
    want = plain_loss(model, params, tokens)
    want.backward()
    assert set(grads) == set(params)
    off = {name: ((g.double() - params[name].grad).norm() / params[name].grad.norm()).item() for name, g in grads.items()}
    assert max(off.values()) <= 48 * 2.0 ** -8, off
    assert abs(loss.item() - want.item()) <= 48 * 2.0 ** -8 * want.item()
