"""The operators together, as the example model uses them: its gradients are
those of the same model written in plain float64 operations, it learns, and
generating token by token gives what the whole sequence gives."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("sequence_model", os.path.join(ROOT, "examples", "sequence_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_loss(model, params, tokens):
    """The model in float64 with automatic differentiation."""
    def norm(x, w=None, b=None):
        z = x - x.mean(-1, keepdim=True)
        z = z / ((z * z).mean(-1, keepdim=True) + 1e-5).sqrt()
        return z if w is None else z * w + b

    def rotate(x):  # [B, N, H, d]
        half = x.shape[-1] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
        a = torch.arange(x.shape[1], dtype=torch.float64, device=x.device)[:, None, None] * freq
        c, d = x[..., :half], x[..., half:]
        return torch.cat([c * a.cos() - d * a.sin(), c * a.sin() + d * a.cos()], -1)

    x = params["embed"][tokens[:, :-1]]
    n = x.shape[1]
    dist = torch.arange(n, device=x.device)[:, None] - torch.arange(n, device=x.device)
    w = torch.exp(model.decay.double()[:, None, None] * dist.clamp(min=0)) * (dist >= 0)
    for i in range(model.layers):
        h = norm(x, params[f"{i}.norm.w"], params[f"{i}.norm.b"])
        q, k, v = (h @ params[f"{i}.qkv"]).unflatten(-1, (3, model.heads, model.head_dim)).unbind(-3)
        score = torch.einsum("bthd,bjhd->bhtj", rotate(q), rotate(k)) * w * model.scale
        o = norm(torch.einsum("bhtj,bjhd->bthd", score, v))
        x = x + o.flatten(2) @ params[f"{i}.out"]
    logp = (x @ params["head"]).log_softmax(-1)
    return -logp.gather(-1, tokens[:, 1:, None]).mean()


def test_gradients(example):
    model = example.SequenceModel(dtype=torch.float32)
    tokens = example.motif_batch(3, 140, 64, torch.Generator().manual_seed(2))
    loss, grads = model.loss_and_grads(tokens)
    params = {k: v.double().requires_grad_() for k, v in model.params.items()}
    want = plain_loss(model, params, tokens)
    want.backward()
    assert abs(loss.item() - want.item()) <= 1e-5 * want.item()
    assert set(grads) == set(params)
    for name, g in grads.items():
        ref = params[name].grad
        # float32 throughout; sums of up to 417 rows through a few layers of products
        assert (g.double() - ref).norm() <= 1e-4 * ref.norm(), name


def test_learns_and_generates(example):
    model, moments = example.SequenceModel(), {}
    gen = torch.Generator().manual_seed(1)
    losses = [model.train_step(example.motif_batch(32, 97, 64, gen), moments).item() for _ in range(100)]
    assert losses[-1] < 0.5 * losses[0]
    prompt = example.motif_batch(4, 60, 64, gen)
    tokens, logits = model.generate(prompt, 12)
    whole, _ = model.forward(torch.cat([prompt, tokens[:, :-1]], 1))
    # bf16 layers: the two forms round differently, a few 2^-8 of the largest logit
    assert (whole[:, 59:] - logits).abs().max() <= 16 * 2.0 ** -8 * whole.abs().max()
