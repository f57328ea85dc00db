"""Cases that time and check the operators of a decayed linear-attention layer.

Three operators, each with its training and its serving form:

* ``decay_*``: linear attention with a decay for each head -- prompts in chunks
  (with or without an incoming state and ragged lengths), single tokens on a
  kept state, and the backward pass;
* ``rotary_*``: rotary positions on queries and keys, and their transpose;
* ``norm_*``: layer norm, forward and backward.

``run`` computes an operator in its plain form (elementary torch operations in
float32, angles in float64, rounded once at the end) or, with ``own`` set,
through this package's entry points.  ``exact`` computes the same outputs in
float64 straight from the definitions, token by token.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 128      # chunk of the plain decayed form
EPS = 1e-5       # of the layer norm
SIDE = 1 << 20   # positions start anywhere below this


def listed():
    return [
        # one new token of 16 sequences: the rotation between the projections and the state update (latency)
        {"name": "rotary_token", "op": "rotary", "batch": 16, "tokens": 1, "heads": 12, "kv_heads": 12, "dim": 64,
         "rot": 64, "style": "half", "layout": "bnhd", "scaling": "none", "factor": 1.0, "back": False, "dtype": "bf16"},
        # queries and keys of whole 32k-token prompts, head-major as the attention reads them
        {"name": "rotary_prompt", "op": "rotary", "batch": 4, "tokens": 32768, "heads": 16, "kv_heads": 16, "dim": 64,
         "rot": 64, "style": "interleaved", "layout": "bhnd", "scaling": "none", "factor": 1.0, "back": False,
         "dtype": "bf16"},
        # a training step's way back: part of each head, fewer key heads, frequencies stretched for a long context
        {"name": "rotary_back_part", "op": "rotary", "batch": 3, "tokens": 1531, "heads": 8, "kv_heads": 2, "dim": 128,
         "rot": 64, "style": "half", "layout": "bnhd", "scaling": "parts", "factor": 4.0, "back": True, "dtype": "f32"},
        # the block's first norm while one token of 64 sequences is generated (latency)
        {"name": "norm_token", "op": "norm", "rows": 64, "cols": 1024, "affine": True, "back": False, "dtype": "bf16"},
        # the norm over each head's output that stands in for the dropped normaliser, on 32k-token prompts
        {"name": "norm_heads", "op": "norm", "rows": 4 * 16 * 32768, "cols": 64, "affine": False, "back": False,
         "dtype": "bf16"},
        # a training step's way back through the block's norm, with the weight's and bias's gradients
        {"name": "norm_train", "op": "norm", "rows": 4 * 16384, "cols": 1024, "affine": True, "back": True,
         "dtype": "bf16"},
        # 32k-token prompts of 16 heads: the largest
        {"name": "decay_prompt", "op": "decay", "batch": 4, "heads": 16, "tokens": 32768, "dk": 64, "dv": 64,
         "layout": "bhnd", "state": False, "ragged": False, "dtype": "bf16"},
        # a padded batch of prompts that continue earlier ones, token-major, wider heads
        {"name": "decay_ragged", "op": "decay", "batch": 5, "heads": 12, "tokens": 1999, "dk": 128, "dv": 128,
         "layout": "bnhd", "state": True, "ragged": True, "dtype": "bf16"},
        # one new token of one sequence (latency) and of 64 sequences (the states' bandwidth)
        {"name": "decay_token_one", "op": "step", "batch": 1, "heads": 16, "dk": 64, "dv": 64, "dtype": "bf16"},
        {"name": "decay_token", "op": "step", "batch": 64, "heads": 16, "dk": 128, "dv": 128, "dtype": "bf16"},
        # training: the gradients of two 8k-token sequences, and of a small odd float32 problem with a carried state
        {"name": "decay_train", "op": "decay_back", "batch": 2, "heads": 16, "tokens": 8192, "dk": 64, "dv": 64,
         "layout": "bhnd", "state": False, "ragged": False, "dtype": "bf16"},
        {"name": "decay_train_f32", "op": "decay_back", "batch": 3, "heads": 5, "tokens": 777, "dk": 64, "dv": 32,
         "layout": "bnhd", "state": True, "ragged": True, "dtype": "f32"},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    kind = rng.choice(["rotary", "norm", "decay", "decay", "step", "decay_back"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "rotary":
        dim = rng.choice([16, 32, 48, 64, 80, 96, 128])
        heads = rng.randint(1, 16)
        batch = _log(rng, 1, 32)
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        return {"op": "rotary", "batch": batch, "tokens": _log(rng, 1, max(1, 32_000_000 // (heads * dim * batch))),
                "heads": heads, "kv_heads": rng.choice([heads, rng.randint(1, heads)]), "dim": dim, "rot": rot,
                "style": rng.choice(["half", "interleaved"]), "layout": rng.choice(["bhnd", "bnhd"]),
                "scaling": rng.choice(["none", "linear", "base", "parts"]), "factor": round(rng.uniform(1.0, 16.0), 2),
                "back": rng.random() < 0.4, "dtype": dtype}
    if kind == "norm":
        cols = _log(rng, 8, 16384)
        return {"op": "norm", "rows": _log(rng, 1, 64_000_000 // cols), "cols": cols, "affine": rng.random() < 0.7,
                "back": rng.random() < 0.5, "dtype": dtype}
    dk, dv = rng.choice([16, 32, 64, 64, 128]), rng.choice([16, 32, 64, 64, 128])
    if kind == "step":
        return {"op": "step", "batch": _log(rng, 1, 64), "heads": rng.randint(1, 24), "dk": dk, "dv": dv,
                "dtype": dtype}
    batch, heads = _log(rng, 1, 8), rng.randint(1, 16)
    most = (64_000_000 if kind == "decay" else 16_000_000) // (batch * heads * max(dk, dv))
    return {"op": kind, "batch": batch, "heads": heads, "tokens": _log(rng, 1, min(32768, most)), "dk": dk, "dv": dv,
            "layout": rng.choice(["bhnd", "bnhd"]), "state": rng.random() < 0.5, "ragged": rng.random() < 0.4,
            "dtype": dtype}


# --------------------------------------------------------------------------
# inputs


def _randn(gen, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    x = torch.randn(*shape, device="cuda", generator=gen)
    if scale != 1.0:
        x.mul_(scale)
    if shift:
        x.add_(shift)
    return x.to(dtype)


def _log_decay(heads):
    # the usual schedule 1 - 2^-(5 + i), spread over 5 .. 12 for any number of heads
    e = torch.linspace(5.0, 12.0, heads, dtype=torch.float64) if heads > 1 else torch.tensor([5.0], dtype=torch.float64)
    return torch.log1p(-torch.exp2(-e)).to(torch.float32).cuda()


def _shape(case, heads, dim):
    b, n = case["batch"], case["tokens"]
    return (b, heads, n, dim) if case["layout"] == "bhnd" else (b, n, heads, dim)


def _inv_freq(rot, scaling, factor):
    """Radians per position of every pair, float64, and the amplitude of the rotated parts."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    base, amplitude = 10000.0, 1.0
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    freq = base ** (-i / rot)
    if scaling == "linear":
        freq = freq / factor
    if scaling == "parts":
        turns = ORIGINAL * freq / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    return freq, amplitude


ORIGINAL = 8192  # context that the scaled frequencies were made for


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    op = case["op"]
    if op == "rotary":
        s["q"] = _randn(gen, *_shape(case, case["heads"], case["dim"]), dtype=dt)
        s["k"] = _randn(gen, *_shape(case, case["kv_heads"], case["dim"]), dtype=dt)
        start = torch.randint(0, SIDE, (case["batch"], 1), device="cuda", generator=gen)
        s["positions"] = start + torch.arange(case["tokens"], device="cuda")
        if own:
            from token_level_head_phi_gb300 import binding as mb
            s["plan"] = mb.mhla_rotary_plan(case["rot"], base=10000.0, scaling=case["scaling"], factor=case["factor"],
                                            original_length=ORIGINAL)
        else:
            freq, s["amplitude"] = _inv_freq(case["rot"], case["scaling"], case["factor"])
            s["freq"] = freq.cuda()
    elif op == "norm":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _randn(gen, rows, cols, dtype=dt, scale=2.0, shift=0.5)
        s["weight"] = _randn(gen, cols, dtype=dt, scale=0.3, shift=1.0) if case["affine"] else None
        s["bias"] = _randn(gen, cols, dtype=dt, scale=0.3) if case["affine"] else None
        if case["back"]:  # what the forward pass kept
            s["dy"] = _randn(gen, rows, cols, dtype=dt)
            x = s["x"].double() if rows * cols < 1 << 26 else s["x"].float()
            s["mean"] = x.mean(1).float()
            s["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + EPS).float()
    else:
        b, h, dk, dv = case["batch"], case["heads"], case["dk"], case["dv"]
        s["decay"] = _log_decay(h)
        s["scale"] = dk ** -0.5
        if op == "step":
            s["q"] = _randn(gen, b, h, dk, dtype=dt)
            s["k"] = _randn(gen, b, h, dk, dtype=dt)
            s["v"] = _randn(gen, b, h, dv, dtype=dt)
            s["state"] = _randn(gen, b, h, dk, dv, scale=4.0)
            return s
        s["q"] = _randn(gen, *_shape(case, h, dk), dtype=dt)
        s["k"] = _randn(gen, *_shape(case, h, dk), dtype=dt)
        s["v"] = _randn(gen, *_shape(case, h, dv), dtype=dt)
        s["state"] = _randn(gen, b, h, dk, dv, scale=4.0) if case["state"] else None
        s["lengths"] = (torch.randint(0, case["tokens"] + 1, (b,), device="cuda", generator=gen, dtype=torch.int32)
                        if case["ragged"] else None)
        if op == "decay_back":
            s["dout"] = _randn(gen, *_shape(case, h, dv), dtype=dt)
            s["dstate"] = _randn(gen, b, h, dk, dv) if case["state"] else None
    return s


# --------------------------------------------------------------------------
# the plain forms


def _rotate(x, cos, sin, rot, style, back):
    """x [..., dim] with cos, sin [..., rot / 2] that broadcast against it; float32."""
    y = x.float()
    r = y[..., :rot]
    if style == "half":
        a, b = r[..., : rot // 2], r[..., rot // 2:]
    else:
        a, b = r[..., 0::2], r[..., 1::2]
    if back:
        sin = -sin
    c, d = a * cos - b * sin, a * sin + b * cos
    r = torch.cat([c, d], -1) if style == "half" else torch.stack([c, d], -1).flatten(-2)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[..., None] * s["freq"]
    cos, sin = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
    axis = 1 if c["layout"] == "bhnd" else 2
    cos, sin = cos.unsqueeze(axis), sin.unsqueeze(axis)
    return {n: _rotate(s[n], cos, sin, c["rot"], c["style"], c["back"]) for n in ("q", "k")}


def _plain_norm(s):
    x = s["x"].float()
    if not s["case"]["back"]:
        mean = x.mean(1, keepdim=True)
        z = x - mean
        rstd = torch.rsqrt((z * z).mean(1, keepdim=True) + EPS)
        y = z * rstd
        if s["weight"] is not None:
            y = y * s["weight"].float() + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float() if s["weight"] is not None else dy
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    out = {"dx": dx.to(s["x"].dtype)}
    if s["weight"] is not None:
        out["dweight"], out["dbias"] = (dy * xh).sum(0), dy.sum(0)
    return out


def _powers(g, n):
    """exp(g n) for integers n >= 0 (0 where n < 0), exponents in float64, one row for each head."""
    n = n.to(torch.float64)
    w = torch.exp(g.double().view(-1, *([1] * n.dim())) * n.clamp(min=0))
    return torch.where(n >= 0, w, torch.zeros_like(w)).float()


def _chunks(s, x):
    """[B, H, chunks, CHUNK, d] float32, zeros past each sequence's length."""
    c = s["case"]
    x = x.float()
    if c["layout"] == "bnhd":
        x = x.transpose(1, 2)
    n = c["tokens"]
    if s["lengths"] is not None:
        past = torch.arange(n, device="cuda") >= s["lengths"][:, None]
        x = x.masked_fill(past[:, None, :, None], 0.0)
    pad = -n % CHUNK
    if pad:
        x = torch.nn.functional.pad(x, (0, 0, 0, pad))
    return x.unflatten(2, (-1, CHUNK))


def _tokens(s, x, dtype):
    x = x.flatten(2, 3)[:, :, : s["case"]["tokens"]]
    return (x if s["case"]["layout"] == "bhnd" else x.transpose(1, 2)).to(dtype).contiguous()


def _ends(s):
    """exp(g (length - 1 - t)) of every token before its sequence's length, and exp(g length): [B, H, N], [B, H]."""
    c = s["case"]
    n = c["tokens"]
    length = s["lengths"] if s["lengths"] is not None else torch.full((c["batch"],), n, device="cuda")
    at = length[:, None] - 1 - torch.arange(n, device="cuda")
    return _powers(s["decay"], at).transpose(0, 1), _powers(s["decay"], length).transpose(0, 1)


def _pairs(g, n, device="cuda"):
    i = torch.arange(n, device=device)
    return i[:, None] - i[None, :]


def _states(s, k, v):
    """The state before each chunk, [B, H, chunks, dk, dv]."""
    g, n = s["decay"], k.shape[2]
    i = torch.arange(CHUNK, device="cuda")
    u = (k * _powers(g, CHUNK - 1 - i)[:, None, :, None]).transpose(-1, -2) @ v
    mix = _powers(g, (_pairs(g, n) - 1) * CHUNK).masked_fill(_pairs(g, n) < 1, 0.0)
    before = (mix @ u.flatten(3)).unflatten(-1, u.shape[-2:])
    if s["state"] is not None:
        before = before + _powers(g, torch.arange(n, device="cuda") * CHUNK)[..., None, None] * s["state"][:, :, None]
    return before


def _plain_decay(s):
    c, g, scale = s["case"], s["decay"], s["scale"]
    q, k, v = (_chunks(s, s[n]) for n in ("q", "k", "v"))
    i = torch.arange(CHUNK, device="cuda")
    within = _powers(g, _pairs(g, CHUNK))[:, None]
    o = ((q @ k.transpose(-1, -2)) * within) @ v
    o = o + (q * _powers(g, i + 1)[:, None, :, None]) @ _states(s, k, v)
    weight, rest = _ends(s)
    last = (k.flatten(2, 3)[:, :, : c["tokens"]] * weight[..., None]).transpose(-1, -2) @ v.flatten(2, 3)[:, :, : c["tokens"]]
    if s["state"] is not None:
        last = last + rest[..., None, None] * s["state"]
    o = o * scale
    return {"out": _tokens(s, o, s["q"].dtype), "state": last}


def _plain_decay_back(s):
    c, g, scale = s["case"], s["decay"], s["scale"]
    q, k, v, do = (_chunks(s, s[n]) for n in ("q", "k", "v", "dout"))
    n = q.shape[2]
    i = torch.arange(CHUNK, device="cuda")
    within = _powers(g, _pairs(g, CHUNK))[:, None]
    score, part = (q @ k.transpose(-1, -2)) * within, (do @ v.transpose(-1, -2)) * within
    dq = part @ k + (do * _powers(g, i + 1)[:, None, :, None]) @ _states(s, k, v).transpose(-1, -2)
    u = (q * _powers(g, i + 1)[:, None, :, None]).transpose(-1, -2) @ do
    mix = _powers(g, (-_pairs(g, n) - 1) * CHUNK).masked_fill(-_pairs(g, n) < 1, 0.0)
    after = (mix @ u.flatten(3)).unflatten(-1, u.shape[-2:])
    w = _powers(g, CHUNK - 1 - i)[:, None, :, None]
    dk = part.transpose(-1, -2) @ q + (v * w) @ after.transpose(-1, -2)
    dv = score.transpose(-1, -2) @ do + (k * w) @ after
    dq, dk, dv = dq * scale, dk * scale, dv * scale
    dt = s["q"].dtype
    out = {}
    if s["dstate"] is not None:
        weight, rest = _ends(s)
        weight = torch.nn.functional.pad(weight, (0, n * CHUNK - c["tokens"])).unflatten(2, (-1, CHUNK))[..., None]
        ds = s["dstate"][:, :, None]
        dk = dk + (v * weight) @ ds.transpose(-1, -2)
        dv = dv + (k * weight) @ ds
        first = _powers(g, torch.arange(n, device="cuda") * CHUNK)[:, None] @ u.flatten(3)
        out["dstate"] = first.view_as(s["dstate"]) * scale + rest[..., None, None] * s["dstate"]
    out.update(dq=_tokens(s, dq, dt), dk=_tokens(s, dk, dt), dv=_tokens(s, dv, dt))
    return out


def _plain_step(s):
    state = s["state"]
    state.mul_(torch.exp(s["decay"])[:, None, None]).add_(s["k"].float()[..., :, None] * s["v"].float()[..., None, :])
    o = (s["q"].float()[..., None, :] @ state)[..., 0, :] * s["scale"]
    return {"out": o.to(s["q"].dtype), "state": state}


PLAIN = {"rotary": _plain_rotary, "norm": _plain_norm, "decay": _plain_decay, "decay_back": _plain_decay_back,
         "step": _plain_step}


# --------------------------------------------------------------------------
# the package's operators


def _own(s):
    from token_level_head_phi_gb300 import binding as mb
    c = s["case"]
    op = c["op"]
    if op == "rotary":
        call = mb.mhla_rotary_backward if c["back"] else mb.mhla_rotary_forward
        q, k = call(s["q"], s["k"], s["plan"], positions=s["positions"], style=c["style"], layout=c["layout"])
        return {"q": q, "k": k}
    if op == "norm":
        if not c["back"]:
            y, mean, rstd = mb.mhla_layernorm_forward(s["x"], s["weight"], s["bias"], eps=EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dweight, dbias = mb.mhla_layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], weight=s["weight"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias} if s["weight"] is not None else {"dx": dx}
    if op == "step":
        return {"out": mb.mhla_decay_step(s["q"], s["k"], s["v"], s["decay"], s["state"], scale=s["scale"]),
                "state": s["state"]}
    if op == "decay":
        out, state = mb.mhla_decay_forward(s["q"], s["k"], s["v"], s["decay"], state=s["state"], lengths=s["lengths"],
                                           scale=s["scale"], layout=c["layout"])
        return {"out": out, "state": state}
    dq, dk, dv, dstate = mb.mhla_decay_backward(s["q"], s["k"], s["v"], s["decay"], s["dout"], state=s["state"],
                                                dstate_out=s["dstate"], lengths=s["lengths"], scale=s["scale"],
                                                layout=c["layout"])
    out = {"dq": dq, "dk": dk, "dv": dv}
    if s["dstate"] is not None:
        out["dstate"] = dstate
    return out


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "rotary":
        n = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * e * n * case["dim"] + 8 * case["batch"] * case["tokens"], "flops": 3 * n * case["rot"]}
    if op == "norm":
        rows, cols, w = case["rows"], case["cols"], 2 * case["cols"] if case["affine"] else 0
        if not case["back"]:
            return {"bytes": 2 * e * rows * cols + e * w + 8 * rows, "flops": 8 * rows * cols}
        return {"bytes": 3 * e * rows * cols + 8 * rows + (e * w // 2 + 4 * w), "flops": 14 * rows * cols}
    dk, dv = case["dk"], case["dv"]
    units = case["batch"] * case["heads"]
    if op == "step":
        return {"bytes": units * (8 * dk * dv + 2 * e * (dk + dv)), "flops": 5 * units * dk * dv}
    tokens = units * case["tokens"]
    states = 4 * units * dk * dv * (2 if case["state"] else 1)
    if op == "decay":
        return {"bytes": tokens * 2 * e * (dk + dv) + states, "flops": 4 * tokens * dk * dv}
    states = 4 * units * dk * dv * 3 if case["state"] else 0
    return {"bytes": tokens * e * (4 * dk + 3 * dv) + states, "flops": 10 * tokens * dk * dv}


# --------------------------------------------------------------------------
# the definitions in float64


def _exact_rotary(s, case):
    freq = torch.empty(case["rot"] // 2, dtype=torch.float64)
    amplitude = 1.0
    for i in range(case["rot"] // 2):
        base = 10000.0
        if case["scaling"] == "base" and case["rot"] > 2:
            base *= case["factor"] ** (case["rot"] / (case["rot"] - 2))
        f = base ** (-2 * i / case["rot"])
        if case["scaling"] == "linear":
            f /= case["factor"]
        if case["scaling"] == "parts":
            keep = min(1.0, max(0.0, (ORIGINAL * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)))
            f = (1 - keep) * f / case["factor"] + keep * f
            amplitude = 1.0 + 0.1 * math.log(case["factor"])
        freq[i] = f
    freq = freq.cuda()
    out = {}
    for name in ("q", "k"):
        x = s[name] if case["layout"] == "bnhd" else s[name].transpose(1, 2)  # [B, N, H, d]
        turn = torch.polar(torch.full((), amplitude, dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, :, None, None] * freq)
        if case["back"]:
            turn = turn.conj()
        r = case["rot"]
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for h in range(x.shape[2]):
            part = x[:, :, h].double()
            re, im = (part[..., : r // 2], part[..., r // 2: r]) if case["style"] == "half" else (part[..., 0:r:2], part[..., 1:r:2])
            z = torch.complex(re.contiguous(), im.contiguous()) * turn[:, :, 0]
            if case["style"] == "half":
                y[:, :, h, : r // 2], y[:, :, h, r // 2: r] = z.real, z.imag
            else:
                y[:, :, h, 0:r:2], y[:, :, h, 1:r:2] = z.real, z.imag
            y[:, :, h, r:] = part[..., r:]
        out[name] = y if case["layout"] == "bnhd" else y.transpose(1, 2).contiguous()
    return out


def _exact_norm(s, case):
    rows, cols = case["rows"], case["cols"]
    w = s["weight"].double() if s["weight"] is not None else torch.ones(cols, dtype=torch.float64, device="cuda")
    b = s["bias"].double() if s["bias"] is not None else torch.zeros(cols, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 25) // cols)
    kept = []
    dw, db = torch.zeros_like(w), torch.zeros_like(w)
    for r in range(0, rows, step):
        x = s["x"][r: r + step].double()
        if not case["back"]:
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = 1.0 / torch.sqrt(var + EPS)
            kept.append(((x - mean[:, None]) * rstd[:, None] * w + b, mean, rstd))
            continue
        rstd = s["rstd"][r: r + step].double()[:, None]
        xh = (x - s["mean"][r: r + step].double()[:, None]) * rstd
        dy = s["dy"][r: r + step].double()
        dw += torch.einsum("rc,rc->c", dy, xh)
        db += dy.sum(0)
        g = dy * w
        along = torch.einsum("rc,rc->r", g, xh)[:, None] / cols
        kept.append((rstd * (g - g.sum(1, keepdim=True) / cols - xh * along),))
    parts = [torch.cat(p) for p in zip(*kept)]
    if not case["back"]:
        return dict(zip(("y", "mean", "rstd"), parts))
    return {"dx": parts[0], "dweight": dw, "dbias": db} if case["affine"] else {"dx": parts[0]}


def _exact_decay(s, case):
    """The recurrence, one token after another; the backward pass runs it forwards for dq and back for dk and dv."""
    back, scale = case["op"] == "decay_back", s["scale"]
    axis = 2 if case["layout"] == "bhnd" else 1
    token = lambda x, t: x.select(axis, t).double()  # noqa: E731  [B, H, d]
    b, h, n, dk, dv = case["batch"], case["heads"], case["tokens"], case["dk"], case["dv"]
    fade = torch.exp(s["decay"].double())[:, None, None]
    alive = [None] * n
    if s["lengths"] is not None:
        m = torch.arange(n, device="cuda")[:, None] < s["lengths"]
        alive = [m[t, :, None, None] for t in range(n)]
    S = s["state"].double() if s["state"] is not None else torch.zeros(b, h, dk, dv, dtype=torch.float64, device="cuda")
    empty = lambda like: torch.empty(like.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    first = empty(s["q"] if back else s["v"])
    for t in range(n):
        nxt = torch.addcmul(fade * S, token(s["k"], t)[..., :, None], token(s["v"], t)[..., None, :])
        S = nxt if alive[t] is None else torch.where(alive[t][..., None], nxt, S)
        o = S @ token(s["dout"], t)[..., None] if back else S.transpose(-1, -2) @ token(s["q"], t)[..., None]
        o = o[..., 0] * scale
        first.select(axis, t).copy_(o if alive[t] is None else torch.where(alive[t], o, torch.zeros_like(o)))
    if not back:
        return {"out": first, "state": S}
    R = s["dstate"].double() if s["dstate"] is not None else torch.zeros(b, h, dk, dv, dtype=torch.float64, device="cuda")
    dk_, dv_ = empty(s["k"]), empty(s["v"])
    for t in reversed(range(n)):
        with_t = torch.addcmul(R, token(s["q"], t)[..., :, None] * scale, token(s["dout"], t)[..., None, :])
        x, y = (with_t @ token(s["v"], t)[..., None])[..., 0], (with_t.transpose(-1, -2) @ token(s["k"], t)[..., None])[..., 0]
        if alive[t] is not None:
            x, y = torch.where(alive[t], x, torch.zeros_like(x)), torch.where(alive[t], y, torch.zeros_like(y))
        dk_.select(axis, t).copy_(x)
        dv_.select(axis, t).copy_(y)
        R = fade * with_t if alive[t] is None else torch.where(alive[t][..., None], fade * with_t, R)
    out = {"dq": first, "dk": dk_, "dv": dv_}
    if s["dstate"] is not None:
        out["dstate"] = R
    return out


def _exact_step(s, case):
    S = torch.exp(s["decay"].double())[:, None, None] * s["state"].double()
    S = S + torch.einsum("bhi,bhj->bhij", s["k"].double(), s["v"].double())
    return {"out": torch.einsum("bhi,bhij->bhj", s["q"].double(), S) * s["scale"], "state": S}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return _exact_rotary(s, case)
    if op == "norm":
        return _exact_norm(s, case)
    if op == "step":
        return _exact_step(s, case)
    return _exact_decay(s, case)
