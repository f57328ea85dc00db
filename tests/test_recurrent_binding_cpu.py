"""Streams, memory and scalars of the wrappers of the recurrent layer and of the
normalised queries and keys, on the CPU: tensors that pass for CUDA tensors,
entries that record how they were called, no kernel."""

import types

import pytest
import torch

from test_sequence_binding_cpu import RAW, card, gpu  # noqa: F401
from token_level_head_phi_gb300 import binding as mb

ENTRIES = ("mhla_qknorm_forward", "mhla_qknorm_backward", "mhla_gated_forward", "mhla_gated_backward", "mhla_gated_step",
           "mhla_shortconv_forward", "mhla_shortconv_backward", "mhla_shortconv_step")


@pytest.fixture
def card0(gpu):  # noqa: F811
    lib = mb.load()
    for n in ENTRIES:
        setattr(lib, n, gpu.entry(n))
    return gpu


def calls(eps=1e-6):
    q, k, w, plan = card(1, 2, 9, 64), card(1, 1, 9, 64), card(64), mb.mhla_rotary_plan(64)
    x, s = card(2, 200, 64), card(2, 64, dtype=torch.float32)
    g, cw, rows = card(64, dtype=torch.float32), card(64, 4), card(2, 3, 64)
    return {
        "qknorm": lambda **a: mb.mhla_qknorm_forward(q, k, plan, q_weight=w, eps=eps, **a),
        "qknorm backward": lambda **a: mb.mhla_qknorm_backward(q, k, q, k, plan, q_weight=w, eps=eps, **a),
        "gated": lambda **a: mb.mhla_gated_forward(x, x, g, x, state=s, keep=True, **a),
        "gated backward": lambda **a: mb.mhla_gated_backward(x, x, x, g, x, state=s, **a),
        "gated step": lambda **a: mb.mhla_gated_step(x[:, 0], x[:, 0], s, g, **a),
        "conv": lambda **a: mb.mhla_shortconv_forward(x, cw, state=rows, **a),
        "conv backward": lambda **a: mb.mhla_shortconv_backward(x, cw, x, state=rows, **a),
        "conv step": lambda **a: mb.mhla_shortconv_step(x[:, 0], cw, rows, **a),
    }


NAMES = ["qknorm", "qknorm backward", "gated", "gated backward", "gated step", "conv",
         "conv backward", "conv step"]
WITH_WORKSPACE = ["qknorm backward", "gated backward", "conv backward"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_object", [False, True])
def test_memory_comes_from_the_stream_of_the_call(card0, name, as_object):
    given = types.SimpleNamespace(cuda_stream=RAW) if as_object else RAW
    results = calls()[name](stream=given)
    assert card0.calls[-1].stream == RAW and card0.now == 0
    assert card0.allocated and all(at == RAW for at, _ in card0.allocated)
    if name in WITH_WORKSPACE:
        assert any(t.dtype == torch.uint8 for _, t in card0.allocated)
    for t in results if isinstance(results, tuple) else (results,):
        assert t is None or t.recorded.cuda_stream == 0


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_and_device(card0, name):
    card0.now = 0x4400
    call = calls()[name]
    call()
    assert card0.calls[-1].stream == 0x4400 and all(at == 0x4400 for at, _ in card0.allocated)
    card0.device = 1
    with pytest.raises(ValueError, match="current device"):
        call()
    assert len(card0.calls) == 1


@pytest.mark.parametrize("name", ["qknorm", "qknorm backward"])
def test_eps_is_taken_by_value(card0, name):
    value = torch.tensor(0.5)
    call = calls(eps=value)[name]
    call()
    value.mul_(2)
    call()
    value.mul_(0.5)
    call()
    assert [c.params.eps for c in card0.calls] == [0.5, 1.0, 0.5]


def test_offsets_change_from_call_to_call(card0):
    for offset in (0, 5, 7, 0):
        calls()["qknorm"](offset=offset)
    assert [c.params.position_offset for c in card0.calls] == [0, 5, 7, 0]


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspace_of_the_caller(card0, name):
    ws = card(1 << 20, dtype=torch.uint8)
    calls()[name](workspace=ws)
    args = card0.calls[-1].args
    assert ws.data_ptr() in args and ws.numel() in args
    for bad in (torch.zeros(1 << 20, dtype=torch.uint8), card(2, 1 << 20, dtype=torch.uint8)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous CUDA tensor"):
            calls()[name](workspace=bad)
    assert len(card0.calls) == 1


def test_own_results_are_left_alone(card0):
    x, s, m = card(2, 20, 64), card(2, 64, dtype=torch.float32), card(2, 2, 64, dtype=torch.float32)
    out, last = card(2, 20, 64), card(2, 64, dtype=torch.float32)
    got = mb.mhla_gated_forward(x, x, state=s, out=out, state_out=last, marks=m, stream=RAW)
    assert got[0] is out and got[1] is last and got[2] is m and not card0.allocated
    assert not any(hasattr(t, "recorded") for t in (out, last, m))
