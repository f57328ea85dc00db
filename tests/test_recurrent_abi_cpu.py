"""Host-side checks of the entries of the recurrent layer and of the normalised
queries and keys: no call here reaches the device."""

import ctypes
import math

import pytest
import torch

from token_level_head_phi_gb300 import binding as mb
from token_level_head_phi_gb300 import build as mbuild

INVALID, UNSUPPORTED, WORKSPACE = mb.MHLA_ERR_INVALID_ARG, mb.MHLA_ERR_UNSUPPORTED, mb.MHLA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mb.load()


def at(i):
    return (1 << 40) + (i << 30)  # addresses that no check may look behind


def strides(p, **kw):
    for name, (b, h, t) in kw.items():
        f = getattr(p, name)
        f.batch, f.head, f.token = b, h, t
    return p


def put(p, kw):
    for k, v in kw.items():
        setattr(p, k, v)
    return p


# ------------------------------------------------- norm of queries and keys


def qk_params(**kw):
    p = mb.MhlaQknormParams(batch=2, tokens=8, heads=4, kv_heads=2, head_dim=64, eps=1e-6, position_dtype=1,
                            position_batch_stride=8, position_token_stride=1)
    q, k = (4 * 8 * 64, 8 * 64, 64), (2 * 8 * 64, 8 * 64, 64)
    return put(strides(p, q=q, q_out=q, dq_out=q, k=k, k_out=k, dk_out=k), kw)


def qk_forward(lib, p, q=at(1), k=at(2), w=at(5), kw=at(6), pos=None, table=64, qo=at(3), ko=at(4)):
    t = mb.mhla_rotary_plan(table).table if table else None
    return lib.mhla_qknorm_forward(q, k, w, kw, pos, t and ctypes.byref(t), p and ctypes.byref(p), qo, ko, None)


def qk_backward(lib, p, dq=at(1), dk=at(2), q=at(3), k=at(4), w=at(5), kw=at(6), pos=None, table=64, gq=at(7), gk=at(8),
                gw=at(9), gkw=at(10), ws=at(11), size=1 << 24):
    t = mb.mhla_rotary_plan(table).table if table else None
    return lib.mhla_qknorm_backward(dq, dk, q, k, w, kw, pos, t and ctypes.byref(t), p and ctypes.byref(p), gq, gk, gw,
                                    gkw, ws, size, None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(tokens=-1), dict(heads=-1), dict(kv_heads=-2), dict(head_dim=62),
                                 dict(head_dim=0), dict(dtype=5), dict(weight_dtype=2), dict(style=2), dict(eps=-1.0),
                                 dict(eps=math.nan), dict(eps=math.inf), dict(position_dtype=2),
                                 dict(style=1, head_dim=65)])
def test_qknorm_refuses_parameters(lib, bad):
    p, n = qk_params(**bad), ctypes.c_size_t(0)
    assert qk_forward(lib, p) == INVALID and qk_backward(lib, p) == INVALID
    if bad != dict(head_dim=62):  # smaller than the table, which this call does not see
        assert lib.mhla_qknorm_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == INVALID


def test_qknorm_refuses_sizes(lib):
    assert qk_forward(lib, qk_params(head_dim=257)) == UNSUPPORTED
    assert qk_forward(lib, qk_params(heads=40000)) == UNSUPPORTED


def test_qknorm_refuses_pointers(lib):
    p = qk_params()
    assert qk_forward(lib, None) == INVALID
    assert qk_forward(lib, p, q=None) == INVALID and qk_forward(lib, p, qo=None) == INVALID
    assert qk_forward(lib, p, k=None) == INVALID                    # k_out without k
    assert qk_forward(lib, p, k=None, ko=None) == INVALID           # k_weight without k
    assert qk_forward(lib, p, q=at(1) + 1) == INVALID and qk_forward(lib, p, w=at(5) + 1) == INVALID
    assert qk_forward(lib, p, qo=at(1) + 128) == INVALID            # overlaps q, not in place
    assert qk_forward(lib, p, qo=at(2)) == INVALID and qk_forward(lib, p, ko=at(3)) == INVALID
    assert qk_forward(lib, p, w=at(3)) == INVALID and qk_forward(lib, p, kw=at(4)) == INVALID
    assert qk_forward(lib, p, pos=at(5) + 4) == INVALID and qk_forward(lib, p, pos=at(3)) == INVALID
    assert qk_forward(lib, strides(qk_params(), q_out=(0, 8 * 64, 64))) == INVALID
    assert qk_forward(lib, strides(qk_params(), q=(4 * 8 * 64, -1, 64))) == INVALID
    for empty in (dict(batch=0), dict(tokens=0), dict(heads=0, kv_heads=0)):
        assert qk_forward(lib, qk_params(**empty)) == mb.MHLA_OK


def test_qknorm_backward_refuses_pointers(lib):
    p, n = qk_params(), ctypes.c_size_t(0)
    assert lib.mhla_qknorm_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == mb.MHLA_OK and n.value > 0
    f = lambda **kw: qk_backward(lib, p, **kw)  # noqa: E731
    for name in ("dq", "dk", "q", "gq", "gk"):
        assert f(**{name: None}) == INVALID, name
    assert f(k=None) == INVALID and f(k=None, dk=None, gk=None, kw=None) == INVALID
    assert f(gq=at(4)) == INVALID and f(gk=at(7)) == INVALID and f(gw=at(7)) == INVALID and f(gw=at(10)) == INVALID
    assert f(gw=at(5)) == INVALID and f(gw=at(9) + 2) == INVALID and f(gq=at(3) + 128) == INVALID
    assert f(ws=at(11) + 16) == INVALID and f(ws=at(7)) == INVALID and f(ws=None) == INVALID
    assert f(size=n.value - 1) == WORKSPACE


# --------------------------------------------------------- gated recurrence


def gated_params(**kw):
    s = (50 * 24, 0, 24)
    p = mb.MhlaGatedParams(batch=2, tokens=50, width=24)
    return put(strides(p, x=s, gate=s, input_gate=s, out=s, dout=s, dx=s, dgate=s, dinput_gate=s), kw)


def gated_forward(lib, p, x=at(1), r=at(2), i=at(3), g=at(4), n=None, s=at(5), o=at(6), so=at(7), m=at(8)):
    return lib.mhla_gated_forward(x, r, i, g, n, s, p and ctypes.byref(p), o, so, m, None)


def gated_backward(lib, p, x=at(1), r=at(2), i=at(3), g=at(4), n=None, s=at(5), m=None, do=at(6), ds=at(7), dx=at(8),
                   dr=at(9), di=at(10), dg=at(11), dsi=at(12), ws=at(13), size=1 << 20):
    return lib.mhla_gated_backward(x, r, i, g, n, s, m, do, ds, p and ctypes.byref(p), dx, dr, di, dg, dsi, ws, size,
                                   None)


def gated_step(lib, p, x=at(1), r=at(2), i=at(3), g=at(4), s=at(5), o=at(6), so=at(5)):
    return lib.mhla_gated_step(x, r, i, g, s, p and ctypes.byref(p), o, so, None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(tokens=-1), dict(width=-1), dict(dtype=2), dict(kind=2),
                                 dict(kind=-1), dict(scale=3), dict(scale=-1), dict(marks=2)])
def test_gated_refuses_parameters(lib, bad):
    p, n = gated_params(**bad), ctypes.c_size_t(0)
    assert gated_forward(lib, p) == INVALID and gated_backward(lib, p) == INVALID
    assert lib.mhla_gated_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == INVALID
    assert gated_step(lib, gated_params(**{"tokens": 1, **bad})) == INVALID


def test_gated_refuses_pointers(lib):
    p = gated_params()
    f = lambda p=p, **kw: gated_forward(lib, p, **kw)  # noqa: E731
    assert f(p=None) == INVALID
    for name in ("x", "r", "g", "o"):
        assert f(**{name: None}) == INVALID, name
    assert f(p=gated_params(kind=1)) == INVALID                     # log_decay without its kind
    assert f(x=at(1) + 1) == INVALID and f(g=at(4) + 2) == INVALID and f(s=at(5) + 1) == INVALID
    for name in ("o", "so", "m"):
        for src in (1, 2, 3, 4):
            assert f(**{name: at(src)}) == INVALID, (name, src)
    assert f(o=at(7)) == INVALID and f(m=at(7)) == INVALID and f(m=at(5)) == INVALID and f(o=at(5)) == INVALID
    assert f(so=at(5) + 4) == INVALID                               # overlaps, not in place
    assert f(n=at(6)) == INVALID and f(n=at(9) + 1) == INVALID
    assert f(p=strides(gated_params(), out=(50 * 24, 0, 23))) == INVALID
    assert f(p=strides(gated_params(), x=(50 * 24, 0, -24))) == INVALID
    assert f(p=gated_params(batch=0)) == mb.MHLA_OK and f(p=gated_params(width=0)) == mb.MHLA_OK
    assert f(p=gated_params(tokens=0x7fffffff)) == UNSUPPORTED


def test_gated_refuses_sizes_near_the_end_of_32_bits(lib):
    # rounds of at most 1024 tokens behind the last one are still counted
    need = ctypes.c_size_t()
    for kw in ({"tokens": 0x7ffff001}, {"tokens": 0x7fffff00}, {"width": 0x7ffff001}, {"width": 0x7fffffff}):
        p = gated_params(**{"batch": 1, "tokens": 1, "width": 1, **kw})
        assert gated_forward(lib, p) == UNSUPPORTED and gated_step(lib, p) == UNSUPPORTED, kw
        assert lib.mhla_gated_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == UNSUPPORTED, kw
    p = gated_params(batch=1, tokens=0x7ffff000, width=1)
    assert lib.mhla_gated_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(need)) == mb.MHLA_OK
    assert need.value >= 4 * (0x7ffff000 // mb.GATED_MARK)


def test_gated_backward_refuses_pointers(lib):
    p, n = gated_params(), ctypes.c_size_t(0)
    assert lib.mhla_gated_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == mb.MHLA_OK
    with_marks = ctypes.c_size_t(0)
    kept = gated_params(marks=1)
    assert lib.mhla_gated_backward_workspace_bytes(ctypes.byref(kept), ctypes.byref(with_marks)) == mb.MHLA_OK
    assert 0 < with_marks.value < n.value
    f = lambda p=p, **kw: gated_backward(lib, p, **kw)  # noqa: E731
    for name in ("x", "r", "g", "do", "dx", "dr"):
        assert f(**{name: None}) == INVALID, name
    assert f(i=None) == INVALID and f(di=None) == INVALID           # the input gate and its gradient go together
    assert f(m=at(14)) == INVALID and f(p=kept) == INVALID          # marks that are not announced, or missing
    assert f(p=gated_params(kind=1), g=None) == INVALID             # dlog_decay without log_decay
    for a, b in (("dx", 6), ("dr", 2), ("di", 8), ("dg", 4), ("dsi", 5), ("dg", 12), ("ws", 8), ("ws", 1)):
        assert f(**{a: at(b)}) == INVALID, (a, b)
    assert f(ws=at(13) + 16) == INVALID and f(ws=None) == INVALID
    assert f(size=n.value - 1) == WORKSPACE


def test_gated_step_refuses(lib):
    p = strides(gated_params(tokens=1), x=(24, 0, 0), gate=(24, 0, 0), input_gate=(24, 0, 0), out=(24, 0, 0))
    f = lambda p=p, **kw: gated_step(lib, p, **kw)  # noqa: E731
    assert f(p=None) == INVALID and f(p=gated_params()) == INVALID  # more than one token
    for name in ("x", "r", "g", "o"):
        assert f(**{name: None}) == INVALID, name
    assert f(o=at(1)) == INVALID and f(o=at(5)) == INVALID and f(so=at(5) + 4) == INVALID and f(so=at(3)) == INVALID


# -------------------------------------------------------- short convolution


def conv_params(**kw):
    s = (50 * 24, 0, 24)
    p = mb.MhlaShortconvParams(batch=2, tokens=50, width=24, taps=4)
    return put(strides(p, x=s, out=s, dout=s, dx=s), kw)


def conv_forward(lib, p, x=at(1), w=at(2), b=at(3), n=None, s=at(4), o=at(5), so=at(6)):
    return lib.mhla_shortconv_forward(x, w, b, n, s, p and ctypes.byref(p), o, so, None)


def conv_backward(lib, p, x=at(1), w=at(2), b=at(3), n=None, s=at(4), do=at(5), ds=at(6), dx=at(7), dw=at(8), db=at(9),
                  dsi=at(10), ws=at(11), size=1 << 24):
    return lib.mhla_shortconv_backward(x, w, b, n, s, do, ds, p and ctypes.byref(p), dx, dw, db, dsi, ws, size, None)


def conv_step(lib, p, x=at(1), w=at(2), b=at(3), s=at(4), o=at(5), so=at(4)):
    return lib.mhla_shortconv_step(x, w, b, s, p and ctypes.byref(p), o, so, None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(tokens=-1), dict(width=-1), dict(dtype=2), dict(weight_dtype=-1),
                                 dict(activation=2), dict(taps=0)])
def test_shortconv_refuses_parameters(lib, bad):
    p, n = conv_params(**bad), ctypes.c_size_t(0)
    assert conv_forward(lib, p) == INVALID and conv_backward(lib, p) == INVALID
    assert lib.mhla_shortconv_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == INVALID
    assert conv_step(lib, conv_params(**{"tokens": 1, **bad})) == INVALID


def test_shortconv_refuses_sizes(lib):
    assert conv_forward(lib, conv_params(taps=1)) == UNSUPPORTED and conv_forward(lib, conv_params(taps=5)) == UNSUPPORTED


def test_shortconv_refuses_pointers(lib):
    p = conv_params()
    f = lambda p=p, **kw: conv_forward(lib, p, **kw)  # noqa: E731
    assert f(p=None) == INVALID
    for name in ("x", "w", "o"):
        assert f(**{name: None}) == INVALID, name
    assert f(x=at(1) + 1) == INVALID and f(w=at(2) + 1) == INVALID and f(n=at(7) + 2) == INVALID
    for name in ("o", "so"):
        for src in (1, 2, 3):
            assert f(**{name: at(src)}) == INVALID, (name, src)
    assert f(o=at(4)) == INVALID and f(o=at(6)) == INVALID and f(so=at(4) + 2) == INVALID and f(n=at(5)) == INVALID
    assert f(p=strides(conv_params(), out=(0, 0, 24))) == INVALID
    assert f(p=strides(conv_params(), x=(-1, 0, 24))) == INVALID
    assert f(p=conv_params(batch=0)) == mb.MHLA_OK and f(p=conv_params(width=0)) == mb.MHLA_OK


def test_shortconv_backward_refuses_pointers(lib):
    p, n = conv_params(), ctypes.c_size_t(0)
    assert lib.mhla_shortconv_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == mb.MHLA_OK and n.value > 0
    f = lambda **kw: conv_backward(lib, p, **kw)  # noqa: E731
    for name in ("x", "w", "do", "dx"):
        assert f(**{name: None}) == INVALID, name
    for a, b in (("dx", 5), ("dx", 1), ("dw", 2), ("dw", 9), ("db", 3), ("dsi", 6), ("dsi", 4), ("ws", 7), ("ws", 1)):
        assert f(**{a: at(b)}) == INVALID, (a, b)
    assert f(dw=at(8) + 2) == INVALID and f(ws=at(11) + 16) == INVALID and f(ws=None) == INVALID
    assert f(size=n.value - 1) == WORKSPACE


def test_shortconv_step_refuses(lib):
    p = strides(conv_params(tokens=1), x=(24, 0, 0), out=(24, 0, 0))
    f = lambda p=p, **kw: conv_step(lib, p, **kw)  # noqa: E731
    assert f(p=None) == INVALID and f(p=conv_params()) == INVALID
    for name in ("x", "w", "o"):
        assert f(**{name: None}) == INVALID, name
    assert f(o=at(1)) == INVALID and f(o=at(4)) == INVALID and f(so=at(4) + 2) == INVALID


# ------------------------------------------------------------ the binding


def test_binding_refusals(monkeypatch):
    """Shapes, dtypes and options, on tensors that pass for CUDA tensors."""
    class Card(torch.Tensor):
        is_cuda = property(lambda self: True)

        def get_device(self):
            return 0

    mbuild.build()
    monkeypatch.setattr(mb, "_CALLS", {})
    card = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype).as_subclass(Card)  # noqa: E731
    x, g, plan = card(2, 5, 8), card(8), mb.mhla_rotary_plan(8)
    q, k, w = card(2, 3, 5, 8), card(2, 1, 5, 8), card(8)
    bad = [
        lambda: mb.mhla_gated_forward(card(2, 8), card(2, 8)),
        lambda: mb.mhla_gated_forward(torch.zeros(2, 5, 8), torch.zeros(2, 5, 8)),
        lambda: mb.mhla_gated_forward(x, card(2, 5, 7)),
        lambda: mb.mhla_gated_forward(x, card(2, 8, 5).transpose(1, 2)),
        lambda: mb.mhla_gated_forward(x, x, card(7)),
        lambda: mb.mhla_gated_forward(x, x, g, scale="sqrt"),
        lambda: mb.mhla_gated_forward(x, x, g, state=card(8, 2).T),
        lambda: mb.mhla_gated_forward(x, x, g, marks=card(2, 2, 8)),
        lambda: mb.mhla_gated_forward(x, x, g, lengths=card(3, dtype=torch.int32)),
        lambda: mb.mhla_gated_backward(x, x, card(2, 5, 9)),
        lambda: mb.mhla_gated_backward(x, x, x, dinput_gate=x),
        lambda: mb.mhla_gated_backward(x, x, x, dlog_decay=g),
        lambda: mb.mhla_gated_backward(x, x, x, g, dlog_decay=g, params=False),
        lambda: mb.mhla_gated_step(x[:, 0], x[:, 0], None),
        lambda: mb.mhla_gated_step(x, x, card(2, 8)),
        lambda: mb.mhla_qknorm_forward(q[0], None, plan),
        lambda: mb.mhla_qknorm_forward(q, card(2, 1, 4, 8), plan),
        lambda: mb.mhla_qknorm_forward(q, None, plan, k_weight=w),
        lambda: mb.mhla_qknorm_forward(q, None, plan, k_out=k),
        lambda: mb.mhla_qknorm_forward(q, k, mb.mhla_rotary_plan(16)),
        lambda: mb.mhla_qknorm_forward(q, k, plan, q_weight=card(7)),
        lambda: mb.mhla_qknorm_forward(q, k, plan, style="both"),
        lambda: mb.mhla_qknorm_forward(q, k, plan, positions=card(4, dtype=torch.int64)),
        lambda: mb.mhla_qknorm_backward(q, None, q, k, plan),
        lambda: mb.mhla_qknorm_backward(q, k, q, None, plan),
        lambda: mb.mhla_qknorm_backward(q, k, q, k, plan, dq_weight=w, params=False),
        lambda: mb.mhla_shortconv_forward(x, card(8)),
        lambda: mb.mhla_shortconv_forward(x, card(7, 4)),
        lambda: mb.mhla_shortconv_forward(x, card(4, 8).T),
        lambda: mb.mhla_shortconv_forward(x, card(8, 4), state=card(2, 4, 8)),
        lambda: mb.mhla_shortconv_forward(x, card(8, 4), activation="gelu"),
        lambda: mb.mhla_shortconv_backward(x, card(8, 4), x, dbias=g, params=False),
        lambda: mb.mhla_shortconv_step(x[:, 0], card(8, 4), None),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    half = torch.float16
    for call in (lambda: mb.mhla_gated_forward(card(2, 5, 8, dtype=half), card(2, 5, 8, dtype=half)),
                 lambda: mb.mhla_gated_forward(x, card(2, 5, 8, dtype=torch.bfloat16)),
                 lambda: mb.mhla_gated_forward(x, x, card(8, dtype=torch.bfloat16)),
                 lambda: mb.mhla_qknorm_forward(q, k, plan, q_weight=w, k_weight=card(8, dtype=torch.bfloat16)),
                 lambda: mb.mhla_qknorm_forward(q, k, plan, positions=card(5)),
                 lambda: mb.mhla_shortconv_forward(x, card(8, 4, dtype=half)),
                 lambda: mb.mhla_shortconv_forward(x, card(8, 4), bias=card(8, dtype=torch.bfloat16)),
                 lambda: mb.mhla_shortconv_forward(x, card(8, 4), state=card(2, 3, 8, dtype=torch.bfloat16))):
        with pytest.raises(TypeError):
            call()
