"""Host-side checks of the rotary, layer-norm and decayed-attention entries: no
call here reaches the device."""

import ctypes
import math

import pytest
import torch

from oracle import sequence_oracle as sq
from token_level_head_phi_gb300 import binding as mb
from token_level_head_phi_gb300 import build as mbuild

INVALID, UNSUPPORTED, WORKSPACE = mb.MHLA_ERR_INVALID_ARG, mb.MHLA_ERR_UNSUPPORTED, mb.MHLA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mb.load()


def at(i):
    return (1 << 40) + (i << 30)  # addresses that no check may look behind


def set_strides(field, b, h, t):
    field.batch, field.head, field.token = b, h, t


# ------------------------------------------------------------------ rotary


@pytest.mark.parametrize("rot,base,scaling,factor,length", [
    (64, 10000.0, "none", 1.0, 0.0), (2, 10000.0, "none", 1.0, 0.0), (256, 1e6, "linear", 4.0, 0.0),
    (32, 10000.0, "base", 8.0, 0.0), (2, 10000.0, "base", 8.0, 0.0), (128, 500000.0, "parts", 16.0, 8192.0),
    (16, 0.25, "none", 1.0, 0.0)])
def test_rotary_table(lib, rot, base, scaling, factor, length):
    plan = mb.mhla_rotary_plan(rot, base, scaling, factor, length)
    freq, amp = sq.rotary_frequencies64(rot, base, scaling, factor, length)
    assert plan.table.pairs == rot // 2 and plan.amplitude == pytest.approx(amp, rel=1e-7)
    for i, f in enumerate(freq):
        turn = f / (2 * math.pi) % 1.0
        got = plan.table.turns[i] / 2.0 ** 64
        assert min(abs(got - turn), 1 - abs(got - turn)) <= 4 * 2.0 ** -53 * max(1.0, f)


@pytest.mark.parametrize("args", [(0, 1e4, 0, 1.0, 0.0), (63, 1e4, 0, 1.0, 0.0), (258, 1e4, 0, 1.0, 0.0),
                                  (64, 0.0, 0, 1.0, 0.0), (64, -1.0, 0, 1.0, 0.0), (64, math.inf, 0, 1.0, 0.0),
                                  (64, math.nan, 0, 1.0, 0.0), (64, 1e4, 4, 1.0, 0.0), (64, 1e4, -1, 1.0, 0.0),
                                  (64, 1e4, 1, 0.0, 0.0), (64, 1e4, 1, math.inf, 0.0), (64, 1e4, 3, 0.5, 100.0),
                                  (64, 1e4, 3, 2.0, 0.0)])
def test_rotary_table_refusals(lib, args):
    table = mb.MhlaRotaryTable()
    assert lib.mhla_rotary_table_init(*args, ctypes.byref(table)) == INVALID
    assert lib.mhla_rotary_table_init(64, 1e4, 0, 1.0, 0.0, None) == INVALID


def rotary_params(**kw):
    p = mb.MhlaRotaryParams()
    p.batch, p.tokens, p.heads, p.kv_heads, p.head_dim = 2, 8, 4, 2, 64
    for f in (p.q, p.q_out):
        set_strides(f, 4 * 8 * 64, 8 * 64, 64)
    for f in (p.k, p.k_out):
        set_strides(f, 2 * 8 * 64, 8 * 64, 64)
    p.position_batch_stride, p.position_token_stride, p.position_dtype = 8, 1, 1
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def rotary(lib, p, q=at(1), k=at(2), pos=None, qo=at(3), ko=at(4), table="half"):
    table = mb.mhla_rotary_plan(64).table if table == "half" else table
    return lib.mhla_rotary(q, k, pos, table and ctypes.byref(table), p and ctypes.byref(p), qo, ko, None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(tokens=-1), dict(heads=-1), dict(kv_heads=-2), dict(head_dim=62),
                                 dict(head_dim=2000), dict(dtype=5), dict(style=2), dict(transpose=2),
                                 dict(position_dtype=2), dict(style=1, head_dim=65)])
def test_rotary_refuses_parameters(lib, bad):
    assert rotary(lib, rotary_params(**bad)) == INVALID


def test_rotary_refuses_pointers_and_overlap(lib):
    p = rotary_params()
    assert rotary(lib, None) == INVALID and rotary(lib, p, table=None) == INVALID
    assert rotary(lib, p, q=None) == INVALID and rotary(lib, p, qo=None) == INVALID
    assert rotary(lib, p, k=None) == INVALID  # k_out without k
    assert rotary(lib, p, q=at(1) + 1) == INVALID
    assert rotary(lib, p, qo=at(1) + 128) == INVALID            # overlaps q, not in place
    assert rotary(lib, p, qo=at(2)) == INVALID                  # overwrites k
    assert rotary(lib, p, ko=at(3)) == INVALID                  # both results in one place
    assert rotary(lib, p, pos=at(5) + 4) == INVALID             # misaligned int64
    assert rotary(lib, p, pos=at(3)) == INVALID                 # positions overwritten
    q = rotary_params()
    set_strides(q.q_out, 0, 8 * 64, 64)                         # an output that overlaps itself
    assert rotary(lib, q) == INVALID
    set_strides(q.q_out, 4 * 8 * 64, 8 * 64, 32)
    assert rotary(lib, q) == INVALID
    set_strides(q.q_out, 4 * 8 * 64, -1, 64)
    assert rotary(lib, q) == INVALID
    for empty in (dict(batch=0), dict(tokens=0), dict(heads=0, kv_heads=0)):
        assert rotary(lib, rotary_params(**empty)) == mb.MHLA_OK


# -------------------------------------------------------------- layer norm


def norm_params(**kw):
    p = mb.MhlaLayernormParams(rows=10, cols=64, dtype=0, weight_dtype=0, eps=1e-5, x_stride=64, y_stride=64, dy_stride=64)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=0), dict(dtype=2), dict(weight_dtype=-1), dict(eps=-1e-5),
                                 dict(eps=math.nan), dict(eps=math.inf)])
def test_layernorm_refuses_parameters(lib, bad):
    p, n = norm_params(**bad), ctypes.c_size_t(0)
    assert lib.mhla_layernorm_forward(at(1), at(2), at(3), ctypes.byref(p), at(4), at(5), at(6), None) == INVALID
    assert lib.mhla_layernorm_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == INVALID
    assert lib.mhla_layernorm_backward(at(1), at(2), at(3), at(4), at(5), ctypes.byref(p), at(6), at(7), at(8), None, 0,
                                       None) == INVALID


def test_layernorm_refuses_pointers(lib):
    f = lambda p=norm_params(), x=at(1), w=at(2), b=at(3), y=at(4), m=at(5), r=at(6): lib.mhla_layernorm_forward(  # noqa: E731
        x, w, b, ctypes.byref(p), y, m, r, None)
    assert lib.mhla_layernorm_forward(at(1), None, None, None, at(4), None, None, None) == INVALID
    assert f(x=None) == INVALID and f(y=None) == INVALID
    assert f(x=at(1) + 1) == INVALID and f(w=at(2) + 1) == INVALID and f(m=at(5) + 2) == INVALID
    assert f(y=at(1) + 64) == INVALID and f(y=at(2)) == INVALID and f(m=at(1)) == INVALID and f(m=at(6)) == INVALID
    assert f(p=norm_params(x_stride=63)) == INVALID and f(p=norm_params(y_stride=0)) == INVALID
    assert f(p=norm_params(cols=(1 << 20) + 1)) == UNSUPPORTED
    assert f(p=norm_params(rows=0), x=None, y=None) == mb.MHLA_OK
    p = norm_params()
    n = ctypes.c_size_t(0)
    assert lib.mhla_layernorm_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == mb.MHLA_OK and n.value > 0
    b = lambda dy=at(1), x=at(2), w=at(3), m=at(4), r=at(5), dx=at(6), dw=at(7), db=at(8), ws=at(9), k=n.value: (  # noqa: E731
        lib.mhla_layernorm_backward(dy, x, w, m, r, ctypes.byref(p), dx, dw, db, ws, k, None))
    assert b(dy=None) == INVALID and b(m=None) == INVALID and b(dx=None) == INVALID
    assert b(dw=at(8)) == INVALID and b(dw=at(6)) == INVALID and b(dx=at(3)) == INVALID and b(dx=at(2) + 128) == INVALID
    assert b(ws=at(9) + 16) == INVALID and b(ws=at(6)) == INVALID and b(ws=None) == INVALID
    assert b(k=n.value - 1) == WORKSPACE


# --------------------------------------------------- decayed linear attention


def decay_params(**kw):
    p = mb.MhlaDecayParams()
    p.batch, p.heads, p.tokens, p.key_dim, p.value_dim, p.scale = 2, 4, 100, 64, 32, 1.0
    for f in (p.q, p.k, p.dq, p.dk):
        set_strides(f, 4 * 100 * 64, 100 * 64, 64)
    for f in (p.v, p.out, p.dout, p.dv):
        set_strides(f, 4 * 100 * 32, 100 * 32, 32)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def decay_forward(lib, p, q=at(1), k=at(2), v=at(3), g=at(4), n=at(5), s=at(6), out=at(7), so=at(8), ws=None, nb=0):
    return lib.mhla_decay_forward(q, k, v, g, n, s, p and ctypes.byref(p), out, so, ws, nb, None)


def decay_backward(lib, p, q=at(1), k=at(2), v=at(3), g=at(4), n=at(5), s=at(6), do=at(7), ds=at(8), dq=at(9), dk=at(10),
                   dv=at(11), di=at(12), ws=None, nb=0):
    return lib.mhla_decay_backward(q, k, v, g, n, s, do, ds, p and ctypes.byref(p), dq, dk, dv, di, ws, nb, None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(heads=-1), dict(tokens=-1), dict(key_dim=48), dict(key_dim=0),
                                 dict(value_dim=256), dict(dtype=3), dict(variant=3), dict(scale=math.nan),
                                 dict(scale=math.inf)])
def test_decay_refuses_parameters(lib, bad):
    p, n = decay_params(**bad), ctypes.c_size_t(0)
    assert decay_forward(lib, p) == INVALID and decay_backward(lib, p) == INVALID
    assert lib.mhla_decay_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == INVALID
    assert lib.mhla_decay_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == INVALID
    assert lib.mhla_decay_workspace_bytes(ctypes.byref(decay_params()), None) == INVALID


def test_decay_tensor_cores_take_bf16_only(lib):
    assert decay_forward(lib, decay_params(dtype=1, variant=2)) == UNSUPPORTED
    assert decay_backward(lib, decay_params(dtype=1, variant=2)) == UNSUPPORTED


def test_decay_refuses_pointers(lib):
    p = decay_params()
    assert decay_forward(lib, None) == INVALID and decay_backward(lib, None) == INVALID
    for name in ("q", "k", "v", "g", "out"):
        assert decay_forward(lib, p, **{name: None}) == INVALID, name
        assert decay_forward(lib, p, **{name: at(20) + 1}) == INVALID, name
    assert decay_forward(lib, p, n=at(5) + 2) == INVALID
    assert decay_forward(lib, p, s=at(6) + 4) == INVALID and decay_forward(lib, p, so=at(8) + 8) == INVALID
    for other in (1, 2, 3, 4, 5, 6, 8):
        assert decay_forward(lib, p, out=at(other)) == INVALID, other
    for other in (1, 4, 5):
        assert decay_forward(lib, p, so=at(other)) == INVALID, other
    assert decay_forward(lib, p, so=at(6) + 64) == INVALID  # partly in place
    assert decay_forward(lib, p, ws=None, nb=16) == INVALID
    for name in ("q", "k", "v", "g", "do", "dq", "dk", "dv"):
        assert decay_backward(lib, p, **{name: None}) == INVALID, name
    for a, b in (("dq", 1), ("dk", 2), ("dv", 7), ("dq", 10), ("dk", 11), ("dv", 6), ("di", 1), ("di", 6), ("dq", 12)):
        assert decay_backward(lib, p, **{a: at(b)}) == INVALID, (a, b)
    q = decay_params()
    set_strides(q.out, 4 * 100 * 32, 100 * 32, 16)
    assert decay_forward(lib, q) == INVALID


def test_decay_workspace(lib):
    n = ctypes.c_size_t(0)
    p = decay_params()  # one segment: none needed
    assert lib.mhla_decay_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == mb.MHLA_OK and n.value == 0
    p = decay_params(batch=1, heads=1, tokens=32768)
    for f in (p.q, p.k):
        set_strides(f, 0, 0, 64)
    for f in (p.v, p.out):
        set_strides(f, 0, 0, 32)
    assert lib.mhla_decay_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == mb.MHLA_OK
    assert n.value >= 2 * 4 * 64 * 32 and n.value % (4 * 64 * 32) == 0
    assert decay_forward(lib, p, ws=at(15), nb=n.value - 1) == WORKSPACE
    assert decay_forward(lib, p, ws=at(15) + 128, nb=n.value) == INVALID
    assert decay_forward(lib, p, ws=at(7), nb=n.value) == INVALID


def test_decay_empty_problems(lib):
    for empty in (dict(batch=0), dict(heads=0)):
        p = decay_params(**empty)
        assert decay_forward(lib, p, q=None, k=None, v=None, g=None, n=None, s=None, out=None, so=None) == mb.MHLA_OK
        assert decay_backward(lib, p) == mb.MHLA_OK


def test_decay_step_refusals(lib):
    p = decay_params(tokens=1)
    f = lambda p=p, q=at(1), k=at(2), v=at(3), g=at(4), s=at(5), out=at(6), so=at(5): lib.mhla_decay_step(  # noqa: E731
        q, k, v, g, s, ctypes.byref(p), out, so, None)
    assert f(p=decay_params()) == INVALID  # more than one token
    for name in ("q", "k", "v", "g", "out"):
        assert f(**{name: None}) == INVALID
    assert f(s=at(5) + 8, so=at(5) + 8) == INVALID and f(so=at(5) + 256) == INVALID and f(out=at(5)) == INVALID
    assert f(out=at(3)) == INVALID


# ----------------------------------------------------- checks of the binding


def test_binding_refuses_tensors(lib):
    x = torch.zeros(1, 2, 4, 32)
    plan = mb.mhla_rotary_plan(32)
    g = torch.zeros(2)
    for call in (lambda: mb.mhla_rotary_forward(x, x, plan), lambda: mb.mhla_layernorm_forward(x),
                 lambda: mb.mhla_decay_forward(x, x, x, g),
                 lambda: mb.mhla_decay_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g, torch.zeros(1, 2, 32, 32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="layout"):
        mb.mhla_decay_forward(x, x, x, g, layout="nope")
    with pytest.raises(ValueError, match="style"):
        mb.mhla_rotary_forward(x, x, plan, style="nope")
    with pytest.raises(ValueError, match="scaling"):
        mb.mhla_rotary_plan(32, scaling="nope")
    with pytest.raises(mb.MhlaError):
        mb.mhla_rotary_plan(31)
