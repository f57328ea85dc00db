"""Streams, memory and scalars of the binding's wrappers, on the CPU: tensors
that pass for CUDA tensors, entries that record how they were called, no
kernel."""

import contextlib
import types

import pytest
import torch

from token_level_head_phi_gb300 import binding as mb
from token_level_head_phi_gb300 import build as mbuild

RAW = 0x7700  # a stream's handle
ENTRIES = ("mhla_rotary", "mhla_layernorm_forward", "mhla_layernorm_backward", "mhla_decay_forward",
           "mhla_decay_backward", "mhla_decay_step", "mhla_forward", "mhla_backward", "mhla_forward_noalloc",
           "mhla_forward_host")


class Card(torch.Tensor):
    """A CPU tensor that says it is on the GPU."""

    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.recorded = stream


def card(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Card)


class Gpu:
    """torch's streams and allocations, and the entries' calls."""

    def __init__(self):
        self.now, self.device, self.allocated, self.calls = 0, 0, [], []

    def entry(self, name):
        def call(*args):
            params = [type(a._obj).from_buffer_copy(a._obj) for a in args if type(a).__name__ == "CArgObject"]
            self.calls.append(types.SimpleNamespace(name=name, args=args, params=params[-1], stream=args[-1]))
            return 0
        return call


@pytest.fixture
def gpu(monkeypatch):
    mbuild.build()
    real, g = mb.load(), Gpu()
    lib = types.SimpleNamespace(**{n: getattr(real, n) for n, _, _ in mb.SIGNATURES})
    for n in ENTRIES:
        setattr(lib, n, g.entry(n))
    empty, empty_like = torch.empty, torch.empty_like

    def made(t):
        t = t.as_subclass(Card)
        g.allocated.append((g.now, t))
        return t

    @contextlib.contextmanager
    def stream(s):
        before, g.now = g.now, s.cuda_stream
        yield
        g.now = before

    monkeypatch.setattr(mb, "load", lambda path=None: lib)
    monkeypatch.setattr(mb, "_CALLS", {})
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made(empty(*a, **k)))
    monkeypatch.setattr(torch, "empty_like", lambda *a, **k: made(empty_like(*a, **k)))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i=None: types.SimpleNamespace(cuda_stream=g.now))
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda h, device=None: types.SimpleNamespace(cuda_stream=h))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: g.now, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: g.device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: g.device)
    return g


def calls(scale=1.0, eps=1e-5):
    """Every wrapper; decay with several segments."""
    q = card(1, 2, 4096, 64)
    x, m = card(8, 64), card(8, dtype=torch.float32)
    g, s = card(2, dtype=torch.float32), card(1, 2, 64, 64, dtype=torch.float32)
    plan = mb.mhla_rotary_plan(64)
    return {
        "rotary": lambda **k: mb.mhla_rotary_forward(q, q, plan, **k),
        "rotary backward": lambda **k: mb.mhla_rotary_backward(q, q, plan, **k),
        "norm": lambda **k: mb.mhla_layernorm_forward(x, eps=eps, **k),
        "norm backward": lambda **k: mb.mhla_layernorm_backward(x, x, m, m, **k),
        "decay": lambda **k: mb.mhla_decay_forward(q, q, q, g, scale=scale, **k),
        "decay backward": lambda **k: mb.mhla_decay_backward(q, q, q, g, q, state=s, scale=scale, **k),
        "step": lambda **k: mb.mhla_decay_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], g, s, scale=scale, **k),
    }


NAMES = ["rotary", "rotary backward", "norm", "norm backward", "decay", "decay backward", "step"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_object", [False, True])
def test_memory_comes_from_the_stream_of_the_call(gpu, name, as_object):
    """A block of another stream's pool could be handed out again while the kernels use it."""
    given = types.SimpleNamespace(cuda_stream=RAW) if as_object else RAW
    results = calls()[name](stream=given)
    assert gpu.calls[-1].stream == RAW and gpu.now == 0
    assert gpu.allocated and all(at == RAW for at, _ in gpu.allocated)
    if name in ("norm backward", "decay", "decay backward"):  # the workspace among them
        assert any(t.dtype == torch.uint8 for _, t in gpu.allocated)
    for t in results if isinstance(results, tuple) else (results,):
        assert t.recorded.cuda_stream == 0  # may be dropped on the stream that was current


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_is_the_default(gpu, name):
    gpu.now = 0x4400
    calls()[name]()
    assert gpu.calls[-1].stream == 0x4400 and all(at == 0x4400 for at, _ in gpu.allocated)


def test_own_results_are_left_alone(gpu):
    q, g = card(1, 2, 8, 64), card(2, dtype=torch.float32)
    out, state = card(1, 2, 8, 64), card(1, 2, 64, 64, dtype=torch.float32)
    mb.mhla_decay_forward(q, q, q, g, out=out, state_out=state, stream=RAW)
    assert not hasattr(out, "recorded") and not hasattr(state, "recorded") and not gpu.allocated


@pytest.mark.parametrize("name,field", [("norm", "eps"), ("decay", "scale"), ("decay backward", "scale"),
                                        ("step", "scale")])
def test_scalars_are_taken_by_value(gpu, name, field):
    """A zero-dimensional tensor hashes by identity: its value may change between two calls."""
    value = torch.tensor(0.5)
    call = calls(**{field: value})[name]
    call()
    value.mul_(2)
    call()
    value.mul_(0.5)
    call()
    assert [getattr(c.params, field) for c in gpu.calls] == [0.5, 1.0, 0.5]


GRID, BLOCK = (1, 8, 8), (1, 4, 4)


@pytest.mark.parametrize("name", ["mhla_forward", "mhla_backward", "mhla_forward_noalloc"])
@pytest.mark.parametrize("stream", [None, RAW])
def test_block_attention_memory_comes_from_the_stream_of_the_call(gpu, name, stream):
    q, mc = card(1, 2, 64, 64), card(4, 4, dtype=torch.float32)
    gpu.now = 0x4400
    args = (q, q, q, mc) + ((q,) if name == "mhla_backward" else ())
    results = getattr(mb, name)(*args, GRID, BLOCK, stream=stream)
    want = stream or 0x4400
    assert gpu.calls[-1].name == name and gpu.calls[-1].stream == want
    assert len(gpu.allocated) == {"mhla_forward": 2, "mhla_backward": 5, "mhla_forward_noalloc": 1}[name]
    assert all(at == want for at, _ in gpu.allocated)
    for t in results if isinstance(results, tuple) else (results,):
        assert not stream or t.recorded.cuda_stream == 0x4400


@pytest.mark.parametrize("name", NAMES + ["mhla_forward", "mhla_backward"])
def test_tensors_of_another_device_than_the_current_one(gpu, name):
    """The entries launch on the current device, where other devices' pointers would fault."""
    if name.startswith("mhla"):
        call = lambda: given_workspace(name, None)  # noqa: E731
    else:
        call = calls()[name]
    call()  # also once the checks of these shapes are behind
    gpu.device = 1
    with pytest.raises(ValueError, match="current device"):
        call()
    gpu.device = 0
    call()
    assert len(gpu.calls) == 2


def given_workspace(name, ws):
    q, mc = card(1, 2, 64, 64), card(4, 4, dtype=torch.float32)
    if name == "mhla_forward":
        return mb.mhla_forward(q, q, q, mc, GRID, BLOCK, workspace=ws)
    if name == "mhla_backward":
        return mb.mhla_backward(q, q, q, mc, q, GRID, BLOCK, workspace=ws)
    if name == "mhla_forward_host":
        c = lambda t: t.as_subclass(torch.Tensor)  # noqa: E731
        return mb.mhla_forward_host(c(q), c(q), c(q), c(mc), GRID, BLOCK, out=torch.zeros(1, 2, 64, 64), dev_buffer=ws)
    return calls()[name](workspace=ws)


@pytest.mark.parametrize("name", ["norm backward", "decay", "decay backward", "mhla_forward", "mhla_backward",
                                  "mhla_forward_host"])
def test_workspace_of_the_caller(gpu, name):
    """The kernels write its first bytes: it has to be on the GPU and without gaps."""
    ws = card(1 << 16, dtype=torch.uint8)
    given_workspace(name, ws)
    args = gpu.calls[-1].args
    assert ws.data_ptr() in args and ws.numel() in args
    for bad in (torch.zeros(1 << 16, dtype=torch.uint8), card(2, 1 << 16, dtype=torch.uint8)[:, ::2],
                card(1, dtype=torch.uint8).expand(1 << 16)):
        with pytest.raises(ValueError, match="contiguous CUDA tensor"):
            given_workspace(name, bad)
    assert len(gpu.calls) == 1


def test_host_call_buffer_comes_from_the_stream_of_the_call(gpu, monkeypatch):
    q, mc = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16), torch.zeros(4, 4)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    mb.mhla_forward_host(q, q, q, mc, GRID, BLOCK, out=torch.zeros_like(q), stream=RAW)
    assert gpu.calls[-1].stream == RAW and [at for at, _ in gpu.allocated] == [RAW]


def test_stream_needs_cuda_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        mb.mhla_layernorm_forward(x, stream=RAW)
