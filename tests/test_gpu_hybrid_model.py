"""The operators together, as the hybrid example uses them: its gradients are
those of the same model in plain float64 operations, and generating token by
token gives what the whole sequence gives."""

import torch
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from examples import hybrid_model
    return hybrid_model


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

    rms = lambda x, w: x * w / ((x * x).mean(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    silu = torch.nn.functional.silu
    x = params["embed"][tokens[:, :-1]]
    n = x.shape[1]
    dist = torch.arange(n, device=x.device)[:, None] - torch.arange(n, device=x.device)
    fade = torch.exp(model.decay.double()[:, None, None] * dist.clamp(min=0)) * (dist >= 0)
    for i in range(model.layers):
        h = norm(x, params[f"{i}.norm.w"], params[f"{i}.norm.b"])
        if i % 2:
            q, k, v = (h @ params[f"{i}.qkv"]).unflatten(-1, (3, model.heads, model.head_dim)).unbind(-3)
            q, k = rotate(rms(q, params[f"{i}.q.w"])), rotate(rms(k, params[f"{i}.k.w"]))
            score = torch.einsum("bthd,bjhd->bhtj", q, k) * fade * model.scale
            f = norm(torch.einsum("bhtj,bjhd->bthd", score, v)).flatten(2)
        else:
            u, r, g, o = (h @ params[f"{i}.in"]).chunk(4, -1)
            rows = torch.nn.functional.pad(u, (0, 0, model.TAPS - 1, 0)).unfold(1, model.TAPS, 1)  # [B, N, D, taps]
            c = silu((rows * params[f"{i}.conv.w"]).sum(-1) + params[f"{i}.conv.b"])
            a = torch.exp(params[f"{i}.decay"] * torch.sigmoid(r))
            add = torch.sqrt(1 - a * a) * c * torch.sigmoid(g)
            y, state = [], torch.zeros_like(add[:, 0])
            for t in range(n):
                state = a[:, t] * state + add[:, t]
                y.append(state)
            f = torch.stack(y, 1) * silu(o)
        x = x + f @ params[f"{i}.out"]
    logp = (x @ params["head"]).log_softmax(-1)
    return -logp.gather(-1, tokens[:, 1:, None]).mean()


def test_gradients(example):
    model = example.HybridModel(dtype=torch.float32, layers=3)
    with torch.no_grad():  # weights that matter
        for name in list(model.params):
            if name.endswith((".q.w", ".k.w", "conv.b")):
                model.params[name] += 0.3 * torch.randn(model.params[name].shape, generator=torch.Generator().manual_seed(3)).cuda()
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


def test_trains(example):
    """Steps run in bf16 and keep every weight finite and every decay a decay."""
    model, moments = example.HybridModel(), {}
    gen = torch.Generator().manual_seed(1)
    for _ in range(5):
        model.train_step(example.motif_batch(8, 97, 64, gen), moments)
    assert all(torch.isfinite(v).all() for v in model.params.values())
    assert (model.params["0.decay"] < 0).all()


def test_generates(example):
    model = example.HybridModel(dtype=torch.float32, layers=4)
    prompt = example.motif_batch(4, 60, 64, torch.Generator().manual_seed(1))
    tokens, logits = model.generate(prompt, 12)
    whole, _ = model.forward(torch.cat([prompt, tokens[:, :-1]], 1))
    # float32 either way; sums of 128 products through four layers, a few hundred roundings
    assert (whole[:, 59:] - logits).abs().max() <= 512 * 2.0 ** -24 * whole.abs().max()
