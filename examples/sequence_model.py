"""A small sequence model on the operators around the attention: layer norm,
rotary positions and linear attention with a decay for each head.

    python examples/sequence_model.py

trains two layers on a synthetic task (sequences that repeat a random motif)
with every gradient formed by this package's backward calls, then generates:
the prompt runs in chunks, each further token on the kept states, and the
tokens' logits are compared with those of the whole sequence at once.

A layer is  h = norm(x);  q, k, v = h W;  q, k = rotary(q, k);
o = decayed attention(q, k, v);  x + norm over each head(o) W_out.
"""

from __future__ import annotations

import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from token_level_head_phi_gb300 import binding as mb  # noqa: E402


class SequenceModel:
    """Weights are float32; the layers compute in ``dtype``."""

    def __init__(self, vocab=64, heads=4, head_dim=32, layers=2, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator().manual_seed(seed)
        width = heads * head_dim
        rand = lambda *s: (torch.randn(*s, generator=gen) * s[0] ** -0.5).cuda()  # noqa: E731
        self.heads, self.head_dim, self.dtype, self.scale = heads, head_dim, dtype, head_dim ** -0.5
        self.params = {"embed": rand(vocab, width) * vocab ** 0.5 * 0.5, "head": rand(width, vocab)}
        for i in range(layers):
            self.params |= {f"{i}.norm.w": torch.ones(width).cuda(), f"{i}.norm.b": torch.zeros(width).cuda(),
                            f"{i}.qkv": rand(width, 3 * width), f"{i}.out": rand(width, width)}
        self.layers = layers
        self.plan = mb.mhla_rotary_plan(head_dim)
        self.decay = torch.log1p(-torch.exp2(-torch.linspace(2, 6, heads))).cuda()

    def _split(self, x):
        """q, k, v of a fused projection: three strided views [B, N, H, d]."""
        return x.unflatten(-1, (3, self.heads, self.head_dim)).unbind(-3)

    def forward(self, tokens, states=None, keep=None, offset=0):
        """Logits [B, N, vocab] and the layers' states; ``keep`` collects what the backward pass needs."""
        p, dt = self.params, self.dtype
        x = p["embed"][tokens].to(dt)
        out_states = []
        for i in range(self.layers):
            h, mean, rstd = mb.mhla_layernorm_forward(x, p[f"{i}.norm.w"], p[f"{i}.norm.b"])
            q, k, v = self._split(h @ p[f"{i}.qkv"].to(dt))
            q, k = mb.mhla_rotary_forward(q, k, self.plan, offset=offset, layout="bnhd")
            state = states[i] if states else None
            if tokens.shape[1] == 1 and state is not None:  # one token: the recurrent form, in place
                o = mb.mhla_decay_step(q[:, 0], k[:, 0], v[:, 0], self.decay, state, scale=self.scale)[:, None]
            else:
                o, state = mb.mhla_decay_forward(q, k, v, self.decay, state=state, scale=self.scale, layout="bnhd")
            out_states.append(state)
            n, hmean, hrstd = mb.mhla_layernorm_forward(o)  # over each head: stands in for the normaliser
            x_next = x + n.flatten(2) @ p[f"{i}.out"].to(dt)
            if keep is not None:
                keep.append((x, h, mean, rstd, q, k, v, o, n, hmean, hrstd))
            x = x_next
        if keep is not None:
            keep.append(x)
        return x.float() @ p["head"], out_states

    def backward(self, tokens, keep, dlogits):
        """Gradients of every weight."""
        p, dt, grads = self.params, self.dtype, {}
        x = keep.pop()
        flat = lambda t: t.flatten(0, -2).float()  # noqa: E731
        grads["head"] = flat(x).T @ flat(dlogits)
        dx = (dlogits @ p["head"].T).to(dt)
        for i in reversed(range(self.layers)):
            x, h, mean, rstd, q, k, v, o, n, hmean, hrstd = keep.pop()
            grads[f"{i}.out"] = flat(n.flatten(2)).T @ flat(dx)
            dn = (dx @ p[f"{i}.out"].to(dt).T).unflatten(-1, (self.heads, self.head_dim))
            do, _, _ = mb.mhla_layernorm_backward(dn, o, hmean, hrstd, params=False)
            # the three gradients land in one buffer, as the projection's backward reads them
            dqkv = torch.empty(*h.shape[:2], 3 * h.shape[2], dtype=dt, device=h.device)
            dq, dk, dv = self._split(dqkv)
            mb.mhla_decay_backward(q, k, v, self.decay, do, scale=self.scale, layout="bnhd", dq=dq, dk=dk, dv=dv)
            mb.mhla_rotary_backward(dq, dk, self.plan, layout="bnhd", dq=dq, dk=dk)  # in place
            grads[f"{i}.qkv"] = flat(h).T @ flat(dqkv)
            dh = dqkv @ p[f"{i}.qkv"].to(dt).T
            dnorm, grads[f"{i}.norm.w"], grads[f"{i}.norm.b"] = mb.mhla_layernorm_backward(
                dh, x, mean, rstd, weight=p[f"{i}.norm.w"])
            dx = dx + dnorm
        grads["embed"] = torch.zeros_like(p["embed"]).index_add_(0, tokens.flatten(), flat(dx))
        return grads

    def loss_and_grads(self, tokens):
        """Mean next-token cross entropy and its gradients."""
        keep = []
        logits, _ = self.forward(tokens[:, :-1], keep=keep)
        target = tokens[:, 1:]
        logp = logits.log_softmax(-1)
        loss = -logp.gather(-1, target[..., None]).mean()
        dlogits = logp.exp()
        dlogits.scatter_add_(-1, target[..., None], torch.full_like(dlogits[..., :1], -1.0))
        return loss, self.backward(tokens[:, :-1], keep, dlogits / target.numel())

    def train_step(self, tokens, moments, lr=3e-3):
        """One step of Adam."""
        loss, grads = self.loss_and_grads(tokens)
        t = moments["t"] = moments.get("t", 0) + 1
        for name, g in grads.items():
            m, s = moments.setdefault(name, (torch.zeros_like(g), torch.zeros_like(g)))
            m.lerp_(g, 0.1)
            s.lerp_(g * g, 0.01)
            self.params[name] -= lr * (m / (1 - 0.9 ** t)) / ((s / (1 - 0.99 ** t)).sqrt() + 1e-8)
        return loss

    def generate(self, prompt, count):
        """``count`` greedy tokens after the prompt, and the logits that chose them."""
        logits, states = self.forward(prompt)
        tokens, chosen = [], []
        for i in range(count):
            chosen.append(logits[:, -1])
            tokens.append(logits[:, -1:].argmax(-1))
            logits, states = self.forward(tokens[-1], states, offset=prompt.shape[1] + i)
        return torch.cat(tokens, 1), torch.stack(chosen, 1)


def motif_batch(batch, length, vocab, gen, period=12):
    """Sequences that repeat a random motif."""
    motif = torch.randint(0, vocab, (batch, period), generator=gen)
    return motif.repeat(1, -(-length // period))[:, :length].cuda()


def main(steps=150):
    model, moments = SequenceModel(), {}
    gen = torch.Generator().manual_seed(1)
    for step in range(steps):
        loss = model.train_step(motif_batch(32, 97, 64, gen), moments)
        if step % 25 == 0 or step == steps - 1:
            print(f"step {step:4d}  loss {loss.item():.3f}")
    prompt = motif_batch(4, 60, 64, gen)
    tokens, logits = model.generate(prompt, 24)
    want = motif_batch_continuation(prompt, 24)
    print(f"generated tokens that continue the motif: {(tokens == want).float().mean().item():.2f}")
    whole, _ = model.forward(torch.cat([prompt, tokens[:, :-1]], 1))
    print(f"logits of single tokens against the whole sequence: {(whole[:, 59:] - logits).abs().max().item():.3f}")


def motif_batch_continuation(prompt, count, period=12):
    at = torch.arange(prompt.shape[1], prompt.shape[1] + count, device=prompt.device)
    return prompt[:, at % period]


if __name__ == "__main__":
    main()
