"""A small hybrid sequence model: layers of a gated recurrence and layers of
decayed linear attention with normalised, rotated queries and keys.

    python examples/hybrid_model.py

trains it on sequences that repeat a random motif, every gradient formed by this
package's backward calls, then generates: the prompt runs at once, each further
token on the kept states, and the tokens' logits are compared with those of the
whole sequence.

Both layers are  x + f(norm(x)) W_out  with
recurrent:  u, r, i, o = h W;  c = silu(conv(u));  y = recurrence(c, r, i);  f = y silu(o);
attention:  q, k, v = h W;  q, k = rotary(norm over each head(q, k));
            f = norm over each head(decayed attention(q, k, v)).
"""

from __future__ import annotations

import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from examples.sequence_model import SequenceModel, motif_batch  # noqa: E402
from token_level_head_phi_gb300 import binding as mb  # noqa: E402


class HybridModel(SequenceModel):
    """Odd layers attend, even ones recur.  Weights are float32; the layers compute in ``dtype``."""

    TAPS = 4

    def __init__(self, vocab=64, heads=4, head_dim=32, layers=2, dtype=torch.bfloat16, seed=0):
        super().__init__(vocab, heads, head_dim, layers, dtype, seed)
        gen = torch.Generator().manual_seed(seed + 1)
        width = heads * head_dim
        rand = lambda *s: (torch.randn(*s, generator=gen) * s[0] ** -0.5).cuda()  # noqa: E731
        for i in range(layers):
            if i % 2:
                self.params |= {f"{i}.q.w": torch.ones(head_dim).cuda(), f"{i}.k.w": torch.ones(head_dim).cuda()}
            else:
                del self.params[f"{i}.qkv"]
                self.params |= {f"{i}.in": rand(width, 4 * width),
                                f"{i}.conv.w": (torch.randn(width, self.TAPS, generator=gen) * 0.5).cuda(),
                                f"{i}.conv.b": torch.zeros(width).cuda(),
                                f"{i}.decay": -torch.exp(torch.linspace(-4, 1, width)).cuda()}
        self.scale = 1.0  # queries and keys have norm sqrt(head_dim) already

    def _recurrent(self, i, h, state, kept):
        """One recurrent layer on h [B, N, width]: its output before W_out and its states."""
        p, dt = self.params, self.dtype
        u, r, g, o = (h @ p[f"{i}.in"].to(dt)).chunk(4, -1)  # strided views of one projection
        cw, cb, decay = p[f"{i}.conv.w"], p[f"{i}.conv.b"], p[f"{i}.decay"]
        marks = None
        if h.shape[1] == 1 and state is not None:  # one token: states in place
            c = mb.mhla_shortconv_step(u[:, 0], cw, state[0], cb, "silu")
            y = mb.mhla_gated_step(c, r[:, 0], state[1], decay, g[:, 0])[:, None]
            c = c[:, None]
        else:
            first = state or (None, None)
            c, rows = mb.mhla_shortconv_forward(u, cw, cb, state=first[0], activation="silu")
            y, last, marks = mb.mhla_gated_forward(c, r, decay, g, state=first[1], keep=kept is not None)
            state = (rows, last)
        if kept is not None:
            kept += [u, r, g, o, c, y, marks]
        return y * torch.nn.functional.silu(o), state

    def _attend(self, i, h, state, offset, kept):
        p = self.params
        q0, k0, v = self._split(h @ p[f"{i}.qkv"].to(self.dtype))
        q, k = mb.mhla_qknorm_forward(q0, k0, self.plan, q_weight=p[f"{i}.q.w"], k_weight=p[f"{i}.k.w"], offset=offset,
                                      layout="bnhd")
        if h.shape[1] == 1 and state is not None:
            o = mb.mhla_decay_step(q[:, 0], k[:, 0], v[:, 0], self.decay, state, scale=self.scale)[:, None]
        else:
            o, state = mb.mhla_decay_forward(q, k, v, self.decay, state=state, scale=self.scale, layout="bnhd")
        n, mean, rstd = mb.mhla_layernorm_forward(o)  # over each head
        if kept is not None:
            kept += [q0, k0, v, q, k, o, mean, rstd]
        return n.flatten(2), state

    def forward(self, tokens, states=None, keep=None, offset=0):
        """Logits [B, N, vocab] and the layers' states; ``keep`` collects what the backward pass needs."""
        p, dt = self.params, self.dtype
        x = p["embed"][tokens].to(dt)
        out_states = []
        for i in range(self.layers):
            h, mean, rstd = mb.mhla_layernorm_forward(x, p[f"{i}.norm.w"], p[f"{i}.norm.b"])
            kept = None if keep is None else [x, h, mean, rstd]
            state = states[i] if states else None
            f, state = self._attend(i, h, state, offset, kept) if i % 2 else self._recurrent(i, h, state, kept)
            out_states.append(state)
            x = x + f @ p[f"{i}.out"].to(dt)
            if keep is not None:
                keep.append(kept + [f])
        if keep is not None:
            keep.append(x)
        return x.float() @ p["head"], out_states

    def _recurrent_backward(self, i, df, kept, grads):
        """Gradient of the layer's projection, [B, N, 4 width]."""
        p = self.params
        u, r, g, o, c, y, marks = kept
        s = torch.sigmoid(o.float())
        dproj = torch.empty(*u.shape[:2], 4 * u.shape[2], dtype=u.dtype, device=u.device)
        du, dr, dg, do = dproj.chunk(4, -1)
        do.copy_(df.float() * y.float() * s * (1 + o.float() * (1 - s)))
        dy = (df.float() * o.float() * s).to(self.dtype)
        dc, _, _, grads[f"{i}.decay"], _ = mb.mhla_gated_backward(c, r, dy, p[f"{i}.decay"], g, marks=marks, dgate=dr,
                                                                  dinput_gate=dg)
        _, grads[f"{i}.conv.w"], grads[f"{i}.conv.b"], _ = mb.mhla_shortconv_backward(
            u, p[f"{i}.conv.w"], dc, p[f"{i}.conv.b"], activation="silu", dx=du)
        return dproj

    def _attend_backward(self, i, df, kept, grads):
        p = self.params
        q0, k0, v, q, k, o, mean, rstd = kept
        do, _, _ = mb.mhla_layernorm_backward(df.unflatten(-1, (self.heads, self.head_dim)), o, mean, rstd, params=False)
        dproj = torch.empty(*df.shape[:2], 3 * df.shape[2], dtype=df.dtype, device=df.device)
        dq, dk, dv = self._split(dproj)
        mb.mhla_decay_backward(q, k, v, self.decay, do, scale=self.scale, layout="bnhd", dq=dq, dk=dk, dv=dv)
        _, _, grads[f"{i}.q.w"], grads[f"{i}.k.w"] = mb.mhla_qknorm_backward(
            dq, dk, q0, k0, self.plan, q_weight=p[f"{i}.q.w"], k_weight=p[f"{i}.k.w"], layout="bnhd", dq=dq, dk=dk)
        return dproj

    def backward(self, tokens, keep, dlogits):
        """Gradients of every weight."""
        p, dt, grads = self.params, self.dtype, {}
        flat = lambda t: t.flatten(0, -2).float()  # noqa: E731
        x = keep.pop()
        grads["head"] = flat(x).T @ flat(dlogits)
        dx = (dlogits @ p["head"].T).to(dt)
        for i in reversed(range(self.layers)):
            x, h, mean, rstd, *kept, f = keep.pop()
            grads[f"{i}.out"] = flat(f).T @ flat(dx)
            df = dx @ p[f"{i}.out"].to(dt).T
            back, name = (self._attend_backward, f"{i}.qkv") if i % 2 else (self._recurrent_backward, f"{i}.in")
            dproj = back(i, df, kept, grads)
            grads[name] = flat(h).T @ flat(dproj)
            dnorm, grads[f"{i}.norm.w"], grads[f"{i}.norm.b"] = mb.mhla_layernorm_backward(
                dproj @ p[name].to(dt).T, x, mean, rstd, weight=p[f"{i}.norm.w"])
            dx = dx + dnorm
        grads["embed"] = torch.zeros_like(p["embed"]).index_add_(0, tokens.flatten(), flat(dx))
        return grads

    def train_step(self, tokens, moments, lr=3e-3):
        loss = super().train_step(tokens, moments, lr)
        for i in range(0, self.layers, 2):
            self.params[f"{i}.decay"].clamp_(max=-1e-4)  # decays stay decays
        return loss


def main(steps=150):
    model, moments = HybridModel(), {}
    gen = torch.Generator().manual_seed(1)
    for step in range(steps):
        loss = model.train_step(motif_batch(32, 97, 64, gen), moments)
        if step % 25 == 0 or step == steps - 1:
            print(f"step {step:4d}  loss {loss.item():.3f}")
    prompt = motif_batch(4, 60, 64, gen)
    tokens, logits = model.generate(prompt, 24)
    whole, _ = model.forward(torch.cat([prompt, tokens[:, :-1]], 1))
    print(f"logits of single tokens against the whole sequence: {(whole[:, 59:] - logits).abs().max().item():.3f}")


if __name__ == "__main__":
    main()
