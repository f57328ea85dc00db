"""Cases that time and check the operators of a recurrent layer and of normalised queries and keys.

Three operators, each with its training and its serving form:

* ``gated_*``: a linear recurrence with gates of each token and channel --
  prompts (with or without an incoming state and ragged lengths), single tokens
  on a kept state, and a training step's forward and backward pass;
* ``qknorm_*``: the norm of queries and keys over each head with the rotary
  positions in the same pass, and its gradients;
* ``conv_*``: the short causal convolution in front of the recurrence, single
  tokens of it, and its gradients.

``run`` computes an operator in its plain form (elementary torch operations in
float32, angles in float64, rounded once at the end) or, with ``own`` set,
through this package's entry points.  ``exact`` computes the same outputs in
float64 straight from the definitions, token by token.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6       # of the norm of queries and keys
SIDE = 1 << 20   # positions start anywhere below this


def listed():
    return [
        # one new token of 64 sequences through the recurrence (latency)
        {"name": "gated_token", "op": "gated_step", "batch": 64, "width": 1024, "kind": "decay", "scale": "norm",
         "input_gate": True, "dtype": "bf16"},
        # whole 32k-token prompts: the recurrence's largest call
        {"name": "gated_prompt", "op": "gated", "batch": 2, "tokens": 32768, "width": 1024, "kind": "decay",
         "scale": "norm", "input_gate": True, "state": False, "ragged": False, "dtype": "bf16"},
        # a padded batch of prompts that continue earlier ones, forget gates only, rows of an odd width
        {"name": "gated_ragged", "op": "gated", "batch": 5, "tokens": 1999, "width": 1010, "kind": "sigmoid",
         "scale": "mean", "input_gate": False, "state": True, "ragged": True, "dtype": "bf16"},
        # a training step of two 8k-token sequences: the layer's output and every gradient
        {"name": "gated_train", "op": "gated_train", "batch": 2, "tokens": 8192, "width": 1024, "kind": "decay",
         "scale": "norm", "input_gate": True, "state": False, "ragged": False, "dtype": "bf16"},
        # a small odd float32 training step with carried states
        {"name": "gated_train_f32", "op": "gated_train", "batch": 3, "tokens": 777, "width": 321, "kind": "decay",
         "scale": "norm", "input_gate": True, "state": True, "ragged": True, "dtype": "f32"},
        # one new token of 16 sequences: queries and keys between the projections and the state update (latency)
        {"name": "qknorm_token", "op": "qknorm", "batch": 16, "tokens": 1, "heads": 16, "kv_heads": 4, "dim": 64,
         "rot": 64, "style": "half", "layout": "bnhd", "weight": True, "dtype": "bf16"},
        # queries and keys of whole 32k-token prompts, fewer key heads
        {"name": "qknorm_prompt", "op": "qknorm", "batch": 4, "tokens": 32768, "heads": 16, "kv_heads": 4, "dim": 64,
         "rot": 64, "style": "half", "layout": "bnhd", "weight": True, "dtype": "bf16"},
        # a training step's way back through queries and keys of wide heads, with the weights' gradients
        {"name": "qknorm_train", "op": "qknorm_back", "batch": 2, "tokens": 8192, "heads": 16, "kv_heads": 4,
         "dim": 128, "rot": 128, "style": "half", "layout": "bnhd", "weight": True, "dtype": "bf16"},
        # the same of a small odd float32 problem, half of each head rotated, head-major
        {"name": "qknorm_train_part", "op": "qknorm_back", "batch": 3, "tokens": 1531, "heads": 8, "kv_heads": 2,
         "dim": 128, "rot": 64, "style": "interleaved", "layout": "bhnd", "weight": True, "dtype": "f32"},
        # one new token of 64 sequences through the convolution (latency)
        {"name": "conv_token", "op": "conv_step", "batch": 64, "width": 1024, "taps": 4, "bias": True,
         "activation": "silu", "dtype": "bf16"},
        # whole 32k-token prompts in front of the recurrence
        {"name": "conv_prompt", "op": "conv", "batch": 2, "tokens": 32768, "width": 1024, "taps": 4, "bias": True,
         "activation": "silu", "state": False, "ragged": False, "dtype": "bf16"},
        # the gradients of a training step, padded sequences with carried states
        {"name": "conv_train", "op": "conv_back", "batch": 4, "tokens": 8192, "width": 1024, "taps": 4, "bias": True,
         "activation": "silu", "state": True, "ragged": True, "dtype": "bf16"},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    kind = rng.choice(["gated", "gated", "gated_train", "gated_step", "qknorm", "qknorm_back", "conv", "conv_back",
                       "conv_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind.startswith("qknorm"):
        dim = rng.choice([16, 32, 48, 64, 64, 80, 96, 128, 128, 256])
        heads, batch = rng.randint(1, 24), _log(rng, 1, 32)
        most = (80_000_000 if kind == "qknorm" else 30_000_000) // (2 * heads * dim * batch)  # of elements
        return {"op": kind, "batch": batch, "tokens": _log(rng, 1, max(1, min(32768, most))), "heads": heads,
                "kv_heads": rng.choice([heads, rng.randint(1, heads)]), "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)]),
                "style": rng.choice(["half", "interleaved"]), "layout": rng.choice(["bhnd", "bnhd"]),
                "weight": rng.random() < 0.8, "dtype": dtype}
    width = rng.choice([8 * _log(rng, 1, 512), _log(rng, 1, 4096)])
    if kind.endswith("step"):
        case = {"op": kind, "batch": _log(rng, 1, 1024), "width": width}
    else:
        batch = _log(rng, 1, 32)
        most = (64_000_000 if kind in ("gated", "conv") else 16_000_000) // (batch * width * (2 if dtype == "f32" else 1))
        case = {"op": kind, "batch": batch, "tokens": _log(rng, 1, max(1, min(32768, most))), "width": width,
                "state": rng.random() < 0.5, "ragged": rng.random() < 0.4}
    if kind.startswith("gated"):
        case.update(kind=rng.choice(["decay", "decay", "sigmoid"]), scale=rng.choice(["norm", "norm", "mean", "none"]),
                    input_gate=rng.random() < 0.7)
    else:
        case.update(taps=rng.randint(2, 4), bias=rng.random() < 0.7, activation=rng.choice(["none", "silu"]))
    case["dtype"] = dtype
    return case


# --------------------------------------------------------------------------
# inputs


def _randn(gen, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    x = torch.randn(*shape, device="cuda", generator=gen)
    if scale != 1.0:
        x.mul_(scale)
    if shift:
        x.add_(shift)
    return x.to(dtype)


def _heads(case, heads):
    b, n, d = case["batch"], case["tokens"], case["dim"]
    return (b, heads, n, d) if case["layout"] == "bhnd" else (b, n, heads, d)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    op = case["op"]
    if op.startswith("qknorm"):
        for name, heads in (("q", case["heads"]), ("k", case["kv_heads"])):
            s[name] = _randn(gen, *_heads(case, heads), dtype=dt, scale=1.5)
            s[name + "_weight"] = _randn(gen, case["dim"], dtype=dt, scale=0.3, shift=1.0) if case["weight"] else None
            if op == "qknorm_back":
                s["d" + name] = _randn(gen, *_heads(case, heads), dtype=dt)
        start = torch.randint(0, SIDE, (case["batch"], 1), device="cuda", generator=gen)
        s["positions"] = start + torch.arange(case["tokens"], device="cuda")
        if own:
            from token_level_head_phi_gb300 import binding as mb
            s["plan"] = mb.mhla_rotary_plan(case["rot"])
        else:
            s["freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])).cuda()
        return s
    b, w = case["batch"], case["width"]
    rows = (b, w) if op.endswith("step") else (b, case["tokens"], w)
    s["x"] = _randn(gen, *rows, dtype=dt)
    carried = op.endswith("step") or case["state"]
    if not op.endswith("step"):
        s["lengths"] = (torch.randint(0, case["tokens"] + 1, (b,), device="cuda", generator=gen, dtype=torch.int32)
                        if case["ragged"] else None)
    if op.startswith("gated"):
        s["gate"] = _randn(gen, *rows, dtype=dt, scale=1.5, shift=0.5)
        s["input_gate"] = _randn(gen, *rows, dtype=dt) if case["input_gate"] else None
        # decays of a channel between 0.999 and 0.02 a token, over the logarithm of their rates
        rate = torch.rand(w, device="cuda", generator=gen) * math.log(4000.0) + math.log(0.001)
        s["log_decay"] = -rate.exp() if case["kind"] == "decay" else None
        s["state"] = _randn(gen, b, w) if carried else None
        if op == "gated_train":
            s["dout"] = _randn(gen, *rows, dtype=dt)
            s["dstate"] = _randn(gen, b, w) if carried else None
    else:
        taps = case["taps"]
        s["weight"] = _randn(gen, w, taps, dtype=dt, scale=taps ** -0.5)
        s["bias"] = _randn(gen, w, dtype=dt, scale=0.2) if case["bias"] else None
        s["state"] = _randn(gen, b, taps - 1, w, dtype=dt) if carried else None
        if op == "conv_back":
            s["dout"] = _randn(gen, *rows, dtype=dt)
            s["dstate"] = _randn(gen, b, taps - 1, w, dtype=dt) if carried else None
    return s


# --------------------------------------------------------------------------
# the plain forms


def _alive(s):
    """True before each sequence's length, [B, N, 1]; None where all are whole."""
    if s["lengths"] is None:
        return None
    return (torch.arange(s["case"]["tokens"], device="cuda") < s["lengths"][:, None])[..., None]


def _gates(s):
    """The gates' pieces in float32: a, c, u and what the gradients need of them."""
    c = s["case"]
    r = s["gate"].float()
    sig = torch.sigmoid(r)
    if c["kind"] == "decay":
        la = s["log_decay"] * sig
        # 1 - a without cancellation; a next to 1 rounded once, for it is multiplied with itself thousands of times
        a, less = torch.exp(s["log_decay"].double() * torch.sigmoid(r.double())).float(), -torch.expm1(la)
        slope = s["log_decay"] * (1 - sig) * sig   # dlog a / dr
    else:
        a, less = sig, torch.sigmoid(-r)
        slope = less
    if c["scale"] == "norm":
        scale = torch.sqrt(less * (1 + a))
    else:
        scale = less if c["scale"] == "mean" else torch.ones_like(a)
    q = torch.sigmoid(s["input_gate"].float()) if s["input_gate"] is not None else None
    x = s["x"].float()
    return a, scale, x if q is None else x * q, q, sig, slope


def _scan(a, b, first):
    """h_t = a_t h_{t-1} + b_t over axis 1, by doubling the span of what each entry holds."""
    if first is not None:
        b = torch.cat([b[:, :1] + a[:, :1] * first[:, None], b[:, 1:]], 1)
    n, step = a.shape[1], 1
    while step < n:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        if 2 * step < n:
            a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _plain_gated(s, train=False):
    c, dt = s["case"], s["x"].dtype
    a, scale, u, q, sig, slope = _gates(s)
    b = scale * u
    alive = _alive(s)
    if alive is not None:  # padding keeps the state
        a, b = torch.where(alive, a, 1.0), torch.where(alive, b, 0.0)
    if train:  # sums of gradients lose what errors of long spans' products leave
        a, b = a.double(), b.double()
    h = _scan(a, b, s["state"]).float()
    a = a.float()
    out = h if alive is None else torch.where(alive, h, 0.0)
    res = {"out": out.to(dt), "state": h[:, -1].contiguous()}
    if not train:
        return res
    del out
    first = s["state"] if s["state"] is not None else torch.zeros_like(h[:, 0])
    before = torch.cat([first[:, None], h[:, :-1]], 1)
    g = s["dout"].float()
    if alive is not None:
        g = torch.where(alive, g, 0.0)
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)  # the decay between a token and the next
    g = _scan(after.flip(1).double(), g.flip(1).double(), s["dstate"]).flip(1).float()
    if s["state"] is not None:
        res["dstate"] = a[:, 0] * g[:, 0]
    if alive is not None:
        g = torch.where(alive, g, 0.0)
    if c["scale"] == "norm":
        turn = -(a * a) / scale
    else:
        turn = -a if c["scale"] == "mean" else torch.zeros_like(a)
    dlog = g * (a * before + u * turn)
    res["dgate"] = (dlog * slope).to(dt)
    if c["kind"] == "decay":
        res["dlog_decay"] = (dlog * sig).sum((0, 1))
    du = g * scale
    res["dx"] = (du if q is None else du * q).to(dt)
    if q is not None:
        res["dinput_gate"] = (du * s["x"].float() * q * (1 - q)).to(dt)
    return res


def _plain_gated_step(s):
    a, scale, u, _, _, _ = _gates(s)
    s["state"].copy_(a * s["state"] + scale * u)
    return {"out": s["state"].to(s["x"].dtype), "state": s["state"]}


def _rotate(y, s, back):
    """Float32 rows [..., dim] of the case's layout; the transposed map for ``back``."""
    c = s["case"]
    angle = s["positions"].double()[..., None] * s["freq"]
    axis = 1 if c["layout"] == "bhnd" else 2
    cos, sin = angle.cos().float().unsqueeze(axis), angle.sin().float().unsqueeze(axis)
    if back:
        sin = -sin
    rot = c["rot"]
    r = y[..., :rot]
    a, b = (r[..., : rot // 2], r[..., rot // 2:]) if c["style"] == "half" else (r[..., 0::2], r[..., 1::2])
    x, z = a * cos - b * sin, a * sin + b * cos
    r = torch.cat([x, z], -1) if c["style"] == "half" else torch.stack([x, z], -1).flatten(-2)
    return torch.cat([r, y[..., rot:]], -1)


def _plain_qknorm(s):
    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s[name + "_weight"]
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if w is not None:
            y = y * w.float()
        out[name] = _rotate(y, s, False).to(s[name].dtype)
    return out


def _plain_qknorm_back(s):
    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s[name + "_weight"]
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * rstd
        t = _rotate(s["d" + name].float(), s, True)
        g = t if w is None else t * w.float()
        out["d" + name] = (rstd * (g - xh * (g * xh).mean(-1, keepdim=True))).to(s[name].dtype)
        if w is not None:
            out["d" + name + "_weight"] = (t * xh).sum((0, 1, 2))
    return out


def _behind(s, x):
    """Float32 rows of the K - 1 tokens before the first one and then x's, zeros past the lengths."""
    x = x.float()
    alive = _alive(s)
    if alive is not None:
        x = torch.where(alive, x, 0.0)
    b, _, w = x.shape
    first = s["state"].float() if s["state"] is not None else x.new_zeros(b, s["case"]["taps"] - 1, w)
    return torch.cat([first, x], 1), alive


def _conv(s, x, n):
    """Sum of the taps over x [B, K - 1 + N, D], and the bias."""
    w = s["weight"].float()
    z = sum(x[:, j: j + n] * w[:, j] for j in range(s["case"]["taps"]))
    return z if s["bias"] is None else z + s["bias"].float()


def _plain_conv(s):
    c, dt = s["case"], s["x"].dtype
    n, taps = c["tokens"], c["taps"]
    x, alive = _behind(s, s["x"])
    y = _conv(s, x, n)
    if c["activation"] == "silu":
        y = y * torch.sigmoid(y)
    if alive is not None:
        y = torch.where(alive, y, 0.0)
    length = s["lengths"].long() if alive is not None else torch.full((c["batch"],), n, device="cuda")
    rows = length[:, None] + torch.arange(taps - 1, device="cuda")
    return {"out": y.to(dt), "state": x[torch.arange(c["batch"], device="cuda")[:, None], rows].to(dt)}


def _plain_conv_back(s):
    c, dt = s["case"], s["x"].dtype
    n, taps = c["tokens"], c["taps"]
    x, alive = _behind(s, s["x"])
    dz = s["dout"].float()
    if c["activation"] == "silu":
        z = _conv(s, x, n)
        sig = torch.sigmoid(z)
        dz = dz * (sig * (1 + z * (1 - sig)))
    if alive is not None:
        dz = torch.where(alive, dz, 0.0)
    w = s["weight"].float()
    dx = torch.zeros_like(x)
    for j in range(taps):
        dx[:, j: j + n] += dz * w[:, j]
    if s["dstate"] is not None:
        length = s["lengths"].long() if alive is not None else torch.full((c["batch"],), n, device="cuda")
        rows = length[:, None] + torch.arange(taps - 1, device="cuda")
        dx[torch.arange(c["batch"], device="cuda")[:, None], rows] += s["dstate"].float()
    out = {"dx": dx[:, taps - 1:].to(dt),
           "dweight": torch.stack([(dz * x[:, j: j + n]).sum((0, 1)) for j in range(taps)], 1)}
    if s["bias"] is not None:
        out["dbias"] = dz.sum((0, 1))
    if s["state"] is not None:
        out["dstate"] = dx[:, : taps - 1].to(dt)
    return out


def _plain_conv_step(s):
    c, dt = s["case"], s["x"].dtype
    rows = torch.cat([s["state"], s["x"][:, None]], 1)
    y = _conv(s, rows.float(), 1)[:, 0]
    if c["activation"] == "silu":
        y = y * torch.sigmoid(y)
    s["state"].copy_(rows[:, 1:])
    return {"out": y.to(dt), "state": s["state"]}


PLAIN = {"gated": _plain_gated, "gated_train": lambda s: _plain_gated(s, True), "gated_step": _plain_gated_step,
         "qknorm": _plain_qknorm, "qknorm_back": _plain_qknorm_back, "conv": _plain_conv,
         "conv_back": _plain_conv_back, "conv_step": _plain_conv_step}


# --------------------------------------------------------------------------
# the package's operators


def _own(s):
    from token_level_head_phi_gb300 import binding as mb
    c = s["case"]
    op = c["op"]
    if op == "gated_step":
        out = mb.mhla_gated_step(s["x"], s["gate"], s["state"], log_decay=s["log_decay"], input_gate=s["input_gate"],
                                 scale=c["scale"])
        return {"out": out, "state": s["state"]}
    if op in ("gated", "gated_train"):
        args = dict(log_decay=s["log_decay"], input_gate=s["input_gate"], state=s["state"], lengths=s["lengths"],
                    scale=c["scale"])
        out, state, marks = mb.mhla_gated_forward(s["x"], s["gate"], keep=op == "gated_train", **args)
        res = {"out": out, "state": state}
        if op == "gated":
            return res
        dx, dgate, dinput, dlog, dstate = mb.mhla_gated_backward(s["x"], s["gate"], s["dout"], marks=marks,
                                                                 dstate_out=s["dstate"], **args)
        if s["state"] is not None:
            res["dstate"] = dstate
        res["dgate"] = dgate
        if c["kind"] == "decay":
            res["dlog_decay"] = dlog
        res["dx"] = dx
        if c["input_gate"]:
            res["dinput_gate"] = dinput
        return res
    if op == "qknorm":
        q, k = mb.mhla_qknorm_forward(s["q"], s["k"], s["plan"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                      eps=EPS, positions=s["positions"], style=c["style"], layout=c["layout"])
        return {"q": q, "k": k}
    if op == "qknorm_back":
        dq, dk, dqw, dkw = mb.mhla_qknorm_backward(s["dq"], s["dk"], s["q"], s["k"], s["plan"], q_weight=s["q_weight"],
                                                   k_weight=s["k_weight"], eps=EPS, positions=s["positions"],
                                                   style=c["style"], layout=c["layout"], params=c["weight"])
        return {"dq": dq, "dq_weight": dqw, "dk": dk, "dk_weight": dkw} if c["weight"] else {"dq": dq, "dk": dk}
    if op == "conv_step":
        out = mb.mhla_shortconv_step(s["x"], s["weight"], s["state"], bias=s["bias"], activation=c["activation"])
        return {"out": out, "state": s["state"]}
    if op == "conv":
        out, state = mb.mhla_shortconv_forward(s["x"], s["weight"], bias=s["bias"], state=s["state"],
                                               lengths=s["lengths"], activation=c["activation"])
        return {"out": out, "state": state}
    dx, dweight, dbias, dstate = mb.mhla_shortconv_backward(
        s["x"], s["weight"], s["dout"], bias=s["bias"], state=s["state"], dstate_out=s["dstate"], lengths=s["lengths"],
        activation=c["activation"])
    res = {"dx": dx, "dweight": dweight}
    if s["bias"] is not None:
        res["dbias"] = dbias
    if s["state"] is not None:
        res["dstate"] = dstate
    return res


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("qknorm"):
        rows = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"])
        side = 8 * case["batch"] * case["tokens"] + (2 * case["dim"] * e if case["weight"] else 0)
        if op == "qknorm":
            return {"bytes": 2 * e * rows * case["dim"] + side, "flops": rows * (4 * case["dim"] + 3 * case["rot"])}
        side += 8 * case["dim"] if case["weight"] else 0
        return {"bytes": 3 * e * rows * case["dim"] + side, "flops": rows * (10 * case["dim"] + 3 * case["rot"])}
    b, w = case["batch"], case["width"]
    n = b * w * case.get("tokens", 1)
    if op.startswith("gated"):
        ins = 3 if case["input_gate"] else 2
        side = 4 * w if case["kind"] == "decay" else 0
        if op == "gated_step":
            return {"bytes": n * (e * (ins + 1) + 8) + side, "flops": 20 * n}
        state = 4 * b * w * (2 if case["state"] else 1)
        if op == "gated":
            return {"bytes": n * e * (ins + 1) + state + side, "flops": 20 * n}
        state += 8 * b * w if case["state"] else 0
        return {"bytes": n * e * (3 * ins + 2) + state + 2 * side, "flops": 65 * n}
    taps = case["taps"]
    side = w * e * (taps + (1 if case["bias"] else 0))
    rows = b * w * (taps - 1) * e
    if op == "conv_step":
        return {"bytes": 2 * e * n + 2 * rows + side, "flops": n * (2 * taps + 5)}
    if op == "conv":
        return {"bytes": 2 * e * n + rows * (2 if case["state"] else 1) + side, "flops": n * (2 * taps + 5)}
    side += 4 * w * (taps + (1 if case["bias"] else 0))
    return {"bytes": 3 * e * n + (3 * rows if case["state"] else 0) + side, "flops": n * (6 * taps + 10)}


# --------------------------------------------------------------------------
# the definitions in float64


def _exact_decays(s, case):
    """[...] of a, c, u, dlog a / dr, dlog a / dlog_decay, dc / dlog a, sigma(i) in float64."""
    e = torch.exp(-s["gate"].double())
    sig, rest = 1 / (1 + e), 1 / (1 + 1 / e)
    if case["kind"] == "decay":
        g = s["log_decay"].double()
        a, gap = torch.exp(g * sig), -torch.special.expm1(g * sig)
        to_r, to_g = g * sig * rest, sig
    else:
        a, gap, to_r, to_g = sig, rest, rest, None
    if case["scale"] == "norm":
        c = (gap * (2 - gap)).sqrt()
        turn = -a.square() / c
    elif case["scale"] == "mean":
        c, turn = gap, -a
    else:
        c, turn = torch.ones_like(a), torch.zeros_like(a)
    q = 1 / (1 + torch.exp(-s["input_gate"].double())) if case["input_gate"] else None
    u = s["x"].double() * q if q is not None else s["x"].double()
    return a, c, u, to_r, to_g, turn, q


def _exact_gated(s, case):
    a, c, u, to_r, to_g, turn, q = _exact_decays(s, case)
    b_, w = case["batch"], case["width"]
    if case["op"] == "gated_step":
        h = a * s["state"].double() + c * u
        return {"out": h, "state": h}
    n = case["tokens"]
    lengths = [n] * b_ if s["lengths"] is None else s["lengths"].tolist()
    add = c * u
    if s["lengths"] is not None:
        for i, length in enumerate(lengths):
            a[i, length:], add[i, length:] = 1.0, 0.0
    h = s["state"].double() if s["state"] is not None else torch.zeros(b_, w, dtype=torch.float64, device="cuda")
    all_h = torch.empty_like(add)
    for t in range(n):
        torch.addcmul(add[:, t], a[:, t], h, out=all_h[:, t])
        h = all_h[:, t]
    res = {"out": all_h, "state": h.clone()}
    if case["op"] == "gated":
        for i, length in enumerate(lengths):
            all_h[i, length:] = 0.0
        return res
    g_all = s["dout"].double()
    for i, length in enumerate(lengths):
        g_all[i, length:] = 0.0
    g = s["dstate"].double() if s["dstate"] is not None else torch.zeros(b_, w, dtype=torch.float64, device="cuda")
    for t in reversed(range(n)):  # g: the gradient of the state behind token t
        g_all[:, t] += g
        g = a[:, t] * g_all[:, t]
    if s["state"] is not None:
        res["dstate"] = g
    for i, length in enumerate(lengths):
        g_all[i, length:] = 0.0
    dlog = g_all * u * turn
    dlog[:, 1:] += g_all[:, 1:] * a[:, 1:] * all_h[:, :-1]
    if s["state"] is not None:
        dlog[:, 0] += g_all[:, 0] * a[:, 0] * s["state"].double()
    res["dgate"] = dlog * to_r
    if case["kind"] == "decay":
        res["dlog_decay"] = torch.einsum("btd,btd->d", dlog, to_g)
    du = g_all * c
    res["dx"] = du if q is None else du * q
    if q is not None:
        res["dinput_gate"] = du * u * (1 - q)
    for i, length in enumerate(lengths):
        all_h[i, length:] = 0.0
    return res


def _exact_turn(z, s, case, back):
    """Complex multiplication of the pairs of z [B, N, H, dim] float64, in place."""
    r = case["rot"]
    freq = torch.tensor([10000.0 ** (-2 * i / r) for i in range(r // 2)], dtype=torch.float64, device="cuda")
    angle = s["positions"].double()[:, :, None, None] * freq
    turn = torch.complex(angle.cos(), -angle.sin() if back else angle.sin())
    if case["style"] == "half":
        re, im = z[..., : r // 2], z[..., r // 2: r]
    else:
        re, im = z[..., 0:r:2], z[..., 1:r:2]
    y = torch.complex(re.contiguous(), im.contiguous()) * turn
    re.copy_(y.real)
    im.copy_(y.imag)
    return z


def _exact_qknorm(s, case):
    swap = (lambda t: t) if case["layout"] == "bnhd" else (lambda t: t.transpose(1, 2))
    res = {}
    for name in ("q", "k"):
        x = swap(s[name])
        w = s[name + "_weight"].double() if case["weight"] else torch.ones(case["dim"], dtype=torch.float64, device="cuda")
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros_like(w)
        for h in range(x.shape[2]):
            xh = x[:, :, h: h + 1].double()
            size = (torch.linalg.vector_norm(xh, dim=-1, keepdim=True) ** 2 / case["dim"] + EPS).sqrt()
            xh = xh / size
            if case["op"] == "qknorm":
                y[:, :, h: h + 1] = _exact_turn(xh * w, s, case, False)
                continue
            t = _exact_turn(swap(s["d" + name])[:, :, h: h + 1].to(torch.float64, copy=True), s, case, True)
            dw += torch.einsum("bnhd,bnhd->d", t, xh)
            along = torch.einsum("bnhd,bnhd,d->bnh", t, xh, w)[..., None] / case["dim"]
            y[:, :, h: h + 1] = (t * w - along * xh) / size
        y = swap(y).contiguous()
        if case["op"] == "qknorm":
            res[name] = y
        else:
            res["d" + name] = y
            if case["weight"]:
                res["d" + name + "_weight"] = dw
    return res


def _exact_conv(s, case):
    """One sequence after another, cut at its length."""
    taps, op = case["taps"], case["op"]
    w = s["weight"].double()
    bias = s["bias"].double() if case["bias"] else 0.0
    silu = case["activation"] == "silu"
    width = case["width"]
    n = case.get("tokens", 1)
    xs = s["x"][:, None] if op == "conv_step" else s["x"]
    ragged = op != "conv_step" and s["lengths"] is not None
    lengths = s["lengths"].tolist() if ragged else [n] * case["batch"]
    dw, db = torch.zeros_like(w), torch.zeros(width, dtype=torch.float64, device="cuda")
    outs, states = [], []
    for i, length in enumerate(lengths):
        before = s["state"][i].double() if s["state"] is not None else torch.zeros(taps - 1, width, dtype=torch.float64, device="cuda")
        rows = torch.cat([before, xs[i, :length].double()])      # [K - 1 + length, D]
        window = rows.unfold(0, taps, 1)                         # [length, D, K]
        z = torch.einsum("tdk,dk->td", window, w) + bias
        if op != "conv_back":
            y = torch.zeros(n, width, dtype=torch.float64, device="cuda")
            y[:length] = z / (1 + torch.exp(-z)) if silu else z
            outs.append(y)
            states.append(rows[length:])
            continue
        dz = s["dout"][i, :length].double()
        if silu:
            p = 1 / (1 + torch.exp(-z))
            dz = dz * p * (1 + z * (1 - p))
        dw += torch.einsum("td,tdk->dk", dz, window)
        db += dz.sum(0)
        drows = torch.zeros(n + taps - 1, width, dtype=torch.float64, device="cuda")
        for j in range(taps):
            drows[j: j + length] += dz * w[:, j]
        if s["dstate"] is not None:
            drows[length: length + taps - 1] += s["dstate"][i].double()
        if length < n:  # what the outgoing state took lies before the length; nothing behind it has a gradient
            drows[length + taps - 1:] = 0.0
        outs.append(drows[taps - 1:])
        states.append(drows[: taps - 1])
    if op == "conv_step":
        return {"out": torch.stack(outs)[:, 0], "state": torch.stack(states)}
    if op == "conv":
        return {"out": torch.stack(outs), "state": torch.stack(states)}
    res = {"dx": torch.stack(outs), "dweight": dw}
    if case["bias"]:
        res["dbias"] = db
    if s["state"] is not None:
        res["dstate"] = torch.stack(states)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["op"].split("_")[0]
    return {"gated": _exact_gated, "qknorm": _exact_qknorm, "conv": _exact_conv}[kind](s, case)
