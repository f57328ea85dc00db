"""ctypes binding of libmhla.so (include/mhla.h), same names as the C ABI.

Only argument marshalling happens here: tensors are checked for device,
dtype, shape and contiguity, their ``data_ptr()`` and the current CUDA
stream are handed to the library, and a non-OK status raises
:class:`MhlaError`.  Every step of the forward pass runs in the library's
kernels; there is no fallback of any kind -- if ``libmhla.so`` is missing the
first call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmhla.so")

MHLA_OK = 0
MHLA_ERR_INVALID_ARG = 1
MHLA_ERR_UNSUPPORTED = 2
MHLA_ERR_WORKSPACE = 3
MHLA_ERR_CUDA = 4
MHLA_ERR_DEVICE_TIMEOUT = 5
MHLA_ERR_OVERFLOW = 6

DTYPE_BF16 = 0
DTYPE_F32 = 1
FEATURE_ELU1 = 0
FEATURE_IDENTITY = 1
FEATURE_RELU = 2
FEATURE_EXP = 3
NORM_DIVISIVE = 0
NORM_MALA = 1
NORM_NONE = 2
VARIANT_AUTO = 0
VARIANT_SIMT = 1
VARIANT_MULTIPASS = 2
VARIANT_FUSED = 3
NUM_PHASE_EVENTS = 6
NUM_BWD_PHASE_EVENTS = 6

NORMS = {"divisive": NORM_DIVISIVE, "mala": NORM_MALA, "none": NORM_NONE}
FEATURE_MAPS = {"elu1": FEATURE_ELU1, "identity": FEATURE_IDENTITY, "relu": FEATURE_RELU, "exp": FEATURE_EXP}
VARIANTS = {"auto": VARIANT_AUTO, "simt": VARIANT_SIMT, "multipass": VARIANT_MULTIPASS, "fused": VARIANT_FUSED}
DTYPES = {"bf16": DTYPE_BF16, "f32": DTYPE_F32}
LAYOUT_BHND = 0
LAYOUT_BNHD = 1
LAYOUTS = {"bhnd": LAYOUT_BHND, "bnhd": LAYOUT_BNHD}
ROTARY_STYLES = {"half": 0, "interleaved": 1}
ROTARY_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}
ROTARY_MAX_PAIRS = 128
DECAY_VARIANTS = {"auto": 0, "simt": 1, "tensor": 2}


class MhlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _lib_or_none()
        text = lib.mhla_status_string(status).decode() if lib else f"status {status}"
        detail = lib.mhla_last_error_string().decode() if (lib and status == MHLA_ERR_CUDA) else ""
        super().__init__(f"{where}: {text}" + (f" ({detail})" if detail else ""))
        self.status = status


class MhlaParams(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("grid", ctypes.c_int * 3), ("block", ctypes.c_int * 3),
        ("dtype", ctypes.c_int), ("feature_map", ctypes.c_int), ("norm", ctypes.c_int),
        ("variant", ctypes.c_int), ("causal", ctypes.c_int), ("layout", ctypes.c_int),
        ("mc_per_head", ctypes.c_int),
    ]


class MhlaPlanInfo(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int), ("n_blocks", ctypes.c_int), ("block_tokens", ctypes.c_int),
        ("variant", ctypes.c_int), ("kernels_per_call", ctypes.c_int), ("summary_splits", ctypes.c_int),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class MhlaStrides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("token", ctypes.c_int64)]


class MhlaRotaryTable(ctypes.Structure):
    _fields_ = [("pairs", ctypes.c_int), ("amplitude", ctypes.c_float), ("turns", ctypes.c_uint64 * ROTARY_MAX_PAIRS)]


class MhlaRotaryParams(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int), ("tokens", ctypes.c_int), ("heads", ctypes.c_int), ("kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("style", ctypes.c_int), ("transpose", ctypes.c_int),
        ("position_dtype", ctypes.c_int), ("position_offset", ctypes.c_int64),
        ("position_batch_stride", ctypes.c_int64), ("position_token_stride", ctypes.c_int64),
        ("q", MhlaStrides), ("k", MhlaStrides), ("q_out", MhlaStrides), ("k_out", MhlaStrides),
    ]


class MhlaLayernormParams(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int), ("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int),
        ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
        ("dy_stride", ctypes.c_int64),
    ]


class MhlaDecayParams(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int), ("heads", ctypes.c_int), ("tokens", ctypes.c_int), ("key_dim", ctypes.c_int),
        ("value_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("variant", ctypes.c_int), ("scale", ctypes.c_float),
        ("q", MhlaStrides), ("k", MhlaStrides), ("v", MhlaStrides), ("out", MhlaStrides),
        ("dout", MhlaStrides), ("dq", MhlaStrides), ("dk", MhlaStrides), ("dv", MhlaStrides),
    ]


_LIB = None
_P = ctypes.c_void_p

# (name, restype, argtypes) of every entry point in include/mhla.h
SIGNATURES = [
    ("mhla_plan", ctypes.c_int, [ctypes.POINTER(MhlaParams), ctypes.POINTER(MhlaPlanInfo)]),
    ("mhla_workspace_bytes", ctypes.c_int, [ctypes.POINTER(MhlaParams), ctypes.POINTER(ctypes.c_size_t)]),
    ("mhla_forward", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.POINTER(MhlaParams), ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]),
    ("mhla_forward_noalloc", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.POINTER(MhlaParams), ctypes.c_void_p, ctypes.c_void_p]),
    ("mhla_host_buffer_bytes", ctypes.c_int, [ctypes.POINTER(MhlaParams), ctypes.POINTER(ctypes.c_size_t)]),
    ("mhla_forward_host", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.POINTER(MhlaParams), ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_size_t, ctypes.c_void_p]),
    ("mhla_device_status", ctypes.c_int, [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    ("mhla_set_phase_events", ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]),
    ("mhla_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("mhla_last_error_string", ctypes.c_char_p, []),
    ("mhla_abi_version", ctypes.c_int, []),
    ("mhla_set_debug", ctypes.c_int, [ctypes.c_int, ctypes.c_longlong]),
    ("mhla_set_backward_phase_events", ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]),
    ("mhla_backward_workspace_bytes", ctypes.c_int, [ctypes.POINTER(MhlaParams), ctypes.POINTER(ctypes.c_size_t)]),
    ("mhla_backward", ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.POINTER(MhlaParams)] + [ctypes.c_void_p] * 5
     + [ctypes.c_size_t, ctypes.c_void_p]),
    ("mhla_rotary_table_init", ctypes.c_int, [ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_double,
                                              ctypes.c_double, ctypes.POINTER(MhlaRotaryTable)]),
    ("mhla_rotary", ctypes.c_int, [_P, _P, _P, ctypes.POINTER(MhlaRotaryTable), ctypes.POINTER(MhlaRotaryParams),
                                   _P, _P, _P]),
    ("mhla_layernorm_forward", ctypes.c_int, [_P, _P, _P, ctypes.POINTER(MhlaLayernormParams), _P, _P, _P, _P]),
    ("mhla_layernorm_backward_workspace_bytes", ctypes.c_int, [ctypes.POINTER(MhlaLayernormParams),
                                                               ctypes.POINTER(ctypes.c_size_t)]),
    ("mhla_layernorm_backward", ctypes.c_int, [_P] * 5 + [ctypes.POINTER(MhlaLayernormParams)] + [_P] * 4
     + [ctypes.c_size_t, _P]),
    ("mhla_decay_workspace_bytes", ctypes.c_int, [ctypes.POINTER(MhlaDecayParams), ctypes.POINTER(ctypes.c_size_t)]),
    ("mhla_decay_forward", ctypes.c_int, [_P] * 6 + [ctypes.POINTER(MhlaDecayParams), _P, _P, _P, ctypes.c_size_t, _P]),
    ("mhla_decay_backward_workspace_bytes", ctypes.c_int, [ctypes.POINTER(MhlaDecayParams),
                                                           ctypes.POINTER(ctypes.c_size_t)]),
    ("mhla_decay_backward", ctypes.c_int, [_P] * 8 + [ctypes.POINTER(MhlaDecayParams)] + [_P] * 5
     + [ctypes.c_size_t, _P]),
    ("mhla_decay_step", ctypes.c_int, [_P] * 5 + [ctypes.POINTER(MhlaDecayParams), _P, _P, _P]),
]


def _lib_or_none():
    return _LIB


def load(path: Optional[str] = None):
    """Load libmhla.so (once) and declare every entry point's signature."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m token_level_head_phi_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, restype, argtypes in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = restype
        fn.argtypes = argtypes
    _LIB = lib
    return lib


def _check(status: int, where: str):
    if status != MHLA_OK:
        raise MhlaError(status, where)


def make_params(batch: int, heads: int, head_dim: int, grid: Sequence[int], block: Sequence[int],
                dtype: str = "bf16", feature_map: str = "elu1", norm: str = "divisive",
                variant: str = "auto", causal: bool = False, layout: str = "bhnd",
                mc_per_head: bool = False) -> MhlaParams:
    p = MhlaParams()
    p.batch, p.heads, p.head_dim = int(batch), int(heads), int(head_dim)
    for i in range(3):
        p.grid[i] = int(grid[i])
        p.block[i] = int(block[i])
    p.dtype = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    p.feature_map = FEATURE_MAPS[feature_map] if isinstance(feature_map, str) else int(feature_map)
    p.norm = NORMS[norm] if isinstance(norm, str) else int(norm)
    p.variant = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    p.causal = int(causal)
    p.layout = LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    p.mc_per_head = int(mc_per_head)
    return p


def mhla_plan(p: MhlaParams) -> MhlaPlanInfo:
    info = MhlaPlanInfo()
    _check(load().mhla_plan(ctypes.byref(p), ctypes.byref(info)), "mhla_plan")
    return info


def mhla_workspace_bytes(p: MhlaParams) -> int:
    n = ctypes.c_size_t(0)
    _check(load().mhla_workspace_bytes(ctypes.byref(p), ctypes.byref(n)), "mhla_workspace_bytes")
    return n.value


def mhla_host_buffer_bytes(p: MhlaParams) -> int:
    n = ctypes.c_size_t(0)
    _check(load().mhla_host_buffer_bytes(ctypes.byref(p), ctypes.byref(n)), "mhla_host_buffer_bytes")
    return n.value


def _torch_dtype_name(t) -> str:
    import torch
    if t.dtype == torch.bfloat16:
        return "bf16"
    if t.dtype == torch.float32:
        return "f32"
    raise TypeError(f"unsupported dtype {t.dtype}; MHLA takes bfloat16 or float32")


def _mc_per_head(mc, p) -> int:
    """1 when mc is [H, M, M] (one matrix per head), 0 when it is [M, M]."""
    if mc.dim() == 3:
        if mc.shape[0] != p.heads:
            raise ValueError(f"per-head mc must be [H={p.heads}, M, M], got {tuple(mc.shape)}")
        return 1
    if mc.dim() != 2:
        raise ValueError("mc must be [M, M] or [H, M, M]")
    return 0


def _params_for(q, grid, block, feature_map, norm, variant, causal=False, layout="bhnd") -> MhlaParams:
    if q.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d] (layout 'bhnd') or [B, N, H, d] (layout 'bnhd')")
    if layout == "bnhd":
        B, N, H, d = q.shape
    else:
        B, H, N, d = q.shape
    if grid[0] * grid[1] * grid[2] != N:
        raise ValueError(f"grid {tuple(grid)} has {grid[0] * grid[1] * grid[2]} tokens, tensors have {N}")
    return make_params(B, H, d, grid, block, _torch_dtype_name(q), feature_map, norm, variant, causal, layout)


def _buffer_bytes(name, t, device) -> int:
    """Bytes of a caller's scratch buffer, which the kernels write from its first element on."""
    if not t.is_cuda or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on {device}")
    return t.numel() * t.element_size()


def _not_current(index):
    """The entries launch on the current device, whatever the pointers' device."""
    return ValueError(f"the tensors are on cuda:{index}, which is not the current device")


def _stream_handle(like) -> int:
    """Handle of torch's current stream on the device of ``like``."""
    import torch
    index = like.get_device()
    if torch.cuda.current_device() != index:
        raise _not_current(index)
    return torch.cuda.current_stream(index).cuda_stream


def _torch_stream(stream, index):
    """A torch stream or a raw handle as a torch stream of device ``index``."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        # 1 is another name of the default stream, which torch knows as 0
        return torch.cuda.default_stream(index) if handle < 2 else torch.cuda.ExternalStream(handle, device=index)
    if stream.device.index != index:
        raise ValueError(f"stream must be on cuda:{index}")
    return stream


def _on_stream(stream, like, outputs, call):
    """call() with ``stream`` (a torch stream or a raw handle) as torch's current one.

    So the workspace and the results come from that stream's memory, and no
    other stream gets the workspace's block while the kernels still use it.
    The results (all but the caller's own ``outputs``) may be read on the stream
    that was current, behind a wait, and dropped there.
    """
    import torch
    if not like.is_cuda:
        raise ValueError("stream needs CUDA tensors")
    index = like.get_device()
    before = torch.cuda.current_stream(index)
    with torch.cuda.stream(_torch_stream(stream, index)):
        results = call()
    for t in results if isinstance(results, tuple) else (results,):
        if t is not None and not any(t is o for o in outputs):
            t.record_stream(before)
    return results


def mhla_forward(q, k, v, mc, grid, block, norm: str = "divisive", feature_map: str = "elu1",
                 variant: str = "auto", out=None, workspace=None, stream=None, causal: bool = False,
                 layout: str = "bhnd"):
    """MHLA forward on CUDA tensors [B, H, N, d]; returns ``out``.

    ``mc`` is a float32 [M, M] CUDA tensor.  ``out`` and ``workspace`` are
    allocated with torch when not given.  The call is enqueued on ``stream``
    (default: torch's current stream) and does not synchronise.
    """
    import torch
    if stream is not None:
        return _on_stream(stream, q, (out,), lambda: mhla_forward(
            q, k, v, mc, grid, block, norm, feature_map, variant, out, workspace, None, causal, layout))
    p = _params_for(q, grid, block, feature_map, norm, variant, causal, layout)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or not t.is_contiguous() or t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{name} must be a contiguous CUDA tensor shaped and typed like q")
    if not mc.is_cuda or mc.dtype != torch.float32 or not mc.is_contiguous():
        raise ValueError("mc must be a contiguous float32 CUDA tensor")
    p.mc_per_head = _mc_per_head(mc, p)
    if out is None:
        out = torch.empty_like(q)
    elif not out.is_cuda or not out.is_contiguous() or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must be a contiguous CUDA tensor shaped and typed like q")
    need = mhla_workspace_bytes(p)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = _buffer_bytes("workspace", workspace, q.device)
    handle = _stream_handle(q)
    status = load().mhla_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), mc.data_ptr(), ctypes.byref(p),
                                 out.data_ptr(), workspace.data_ptr(), ws_bytes, handle)
    _check(status, "mhla_forward")
    return out


def mhla_backward_workspace_bytes(p: MhlaParams) -> int:
    n = ctypes.c_size_t(0)
    _check(load().mhla_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)), "mhla_backward_workspace_bytes")
    return n.value


def mhla_backward(q, k, v, mc, dout, grid, block, norm: str = "divisive", feature_map: str = "elu1",
                  dq=None, dk=None, dv=None, dmc=None, workspace=None, stream=None, variant: str = "auto",
                  layout: str = "bhnd", causal: bool = False):
    """Gradients of sum(dout * mhla_forward(q, k, v, mc)): returns (dq, dk, dv, dmc).

    dq, dk, dv are shaped and typed like q; dmc is float32 [M, M] (summed
    over every batch and head).  Outputs and workspace are allocated with
    torch when not given; enqueued on ``stream`` without synchronising.
    ``variant``: "auto" (tensor cores for bf16 with d = 64, else float32 CUDA
    cores) or "simt" (float32 CUDA cores).  ``causal``: the block-ordered
    causal form (float32 CUDA cores).
    """
    import torch
    if stream is not None:
        return _on_stream(stream, q, (dq, dk, dv, dmc), lambda: mhla_backward(
            q, k, v, mc, dout, grid, block, norm, feature_map, dq, dk, dv, dmc, workspace, None, variant, layout,
            causal))
    p = _params_for(q, grid, block, feature_map, norm, variant, causal, layout)
    for name, t in (("q", q), ("k", k), ("v", v), ("dout", dout)):
        if not t.is_cuda or not t.is_contiguous() or t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{name} must be a contiguous CUDA tensor shaped and typed like q")
    if not mc.is_cuda or mc.dtype != torch.float32 or not mc.is_contiguous():
        raise ValueError("mc must be a contiguous float32 CUDA tensor")
    p.mc_per_head = _mc_per_head(mc, p)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        if not t.is_cuda or not t.is_contiguous() or t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{name} must be a contiguous CUDA tensor shaped and typed like q")
    if dmc is None:
        dmc = torch.empty_like(mc)
    elif not dmc.is_cuda or dmc.dtype != torch.float32 or not dmc.is_contiguous() or dmc.shape != mc.shape:
        raise ValueError("dmc must be a contiguous float32 CUDA tensor shaped like mc")
    need = mhla_backward_workspace_bytes(p)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = _buffer_bytes("workspace", workspace, q.device)
    handle = _stream_handle(q)
    status = load().mhla_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), mc.data_ptr(), dout.data_ptr(),
                                  ctypes.byref(p), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dmc.data_ptr(),
                                  workspace.data_ptr(), ws_bytes, handle)
    _check(status, "mhla_backward")
    return dq, dk, dv, dmc


def mhla_forward_raw(q_ptr: int, k_ptr: int, v_ptr: int, mc_ptr: int, p: MhlaParams, out_ptr: int,
                     ws_ptr: int, ws_bytes: int, stream_handle: int) -> int:
    """Direct call with raw device pointers; returns the status code."""
    return load().mhla_forward(q_ptr, k_ptr, v_ptr, mc_ptr, ctypes.byref(p), out_ptr, ws_ptr, ws_bytes,
                               stream_handle)


def mhla_forward_noalloc(q, k, v, mc, grid, block, norm: str = "divisive", feature_map: str = "elu1",
                         variant: str = "auto", out=None, stream=None, layout: str = "bhnd"):
    """mhla_forward without any device allocation by the library: its scratch
    is a static 32 MiB device array (see include/mhla.h).  For callers that
    cannot allocate at call time; ``out`` must be given by such callers (when
    it is None this wrapper allocates it with torch, for convenience)."""
    import torch
    if stream is not None:
        return _on_stream(stream, q, (out,), lambda: mhla_forward_noalloc(
            q, k, v, mc, grid, block, norm, feature_map, variant, out, None, layout))
    p = _params_for(q, grid, block, feature_map, norm, variant, False, layout)
    p.mc_per_head = _mc_per_head(mc, p)
    if out is None:
        out = torch.empty_like(q)
    handle = _stream_handle(q)
    status = load().mhla_forward_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), mc.data_ptr(), ctypes.byref(p),
                                         out.data_ptr(), handle)
    _check(status, "mhla_forward_noalloc")
    return out


def mhla_forward_host(q, k, v, mc, grid, block, norm: str = "divisive", feature_map: str = "elu1",
                      variant: str = "auto", out=None, dev_buffer=None, stream=None, causal: bool = False,
                      layout: str = "bhnd"):
    """End-to-end call on CPU tensors (pinned for asynchronous copies).

    Copies the inputs into ``dev_buffer`` (a CUDA uint8 tensor of at least
    ``mhla_host_buffer_bytes`` bytes), runs the forward pass and copies the
    result back into ``out``; returns when ``out`` is complete.
    """
    import torch
    if stream is not None:  # a new dev_buffer comes from that stream's memory
        index = torch.cuda.current_device() if dev_buffer is None else dev_buffer.get_device()
        with torch.cuda.stream(_torch_stream(stream, index)):
            return mhla_forward_host(q, k, v, mc, grid, block, norm, feature_map, variant, out, dev_buffer, None, causal,
                                     layout)
    p = _params_for(q, grid, block, feature_map, norm, variant, causal, layout)
    p.mc_per_head = _mc_per_head(mc, p)
    for name, t in (("q", q), ("k", k), ("v", v), ("mc", mc)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU tensor")
    if out is None:
        out = torch.empty_like(q)
    need = mhla_host_buffer_bytes(p)
    if dev_buffer is None:
        dev_buffer = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    buffer_bytes = _buffer_bytes("dev_buffer", dev_buffer, dev_buffer.device)
    handle = _stream_handle(dev_buffer)
    status = load().mhla_forward_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), mc.data_ptr(), ctypes.byref(p),
                                      out.data_ptr(), dev_buffer.data_ptr(), buffer_bytes, handle)
    _check(status, "mhla_forward_host")
    return out


def mhla_device_status():
    """(code, detail) of the device error word; blocks until the device is idle."""
    code, detail = ctypes.c_int(0), ctypes.c_int(0)
    _check(load().mhla_device_status(ctypes.byref(code), ctypes.byref(detail)), "mhla_device_status")
    return code.value, detail.value


def mhla_set_phase_events(events) -> None:
    """Install (list of NUM_PHASE_EVENTS torch.cuda.Event) or clear (None) the phase-timing hook."""
    if events is None:
        _check(load().mhla_set_phase_events(None, 0), "mhla_set_phase_events")
        return
    for e in events:  # torch creates the CUDA event on its first record
        if not e.cuda_event:
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(load().mhla_set_phase_events(arr, len(events)), "mhla_set_phase_events")


def mhla_set_backward_phase_events(events) -> None:
    """The same hook for mhla_backward (NUM_BWD_PHASE_EVENTS events, or None)."""
    if events is None:
        _check(load().mhla_set_backward_phase_events(None, 0), "mhla_set_backward_phase_events")
        return
    for e in events:
        if not e.cuda_event:
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(load().mhla_set_backward_phase_events(arr, len(events)), "mhla_set_backward_phase_events")


def mhla_backward_raw(q_ptr: int, k_ptr: int, v_ptr: int, mc_ptr: int, dout_ptr: int, p: MhlaParams, dq_ptr: int,
                      dk_ptr: int, dv_ptr: int, dmc_ptr: int, ws_ptr: int, ws_bytes: int, stream_handle: int) -> int:
    """Direct call with raw device pointers; returns the status code."""
    return load().mhla_backward(q_ptr, k_ptr, v_ptr, mc_ptr, dout_ptr, ctypes.byref(p), dq_ptr, dk_ptr, dv_ptr,
                                dmc_ptr, ws_ptr, ws_bytes, stream_handle)


def mhla_status_string(status: int) -> str:
    return load().mhla_status_string(status).decode()


DEBUG_FLOW_WAIT_NS = 1
DEBUG_FLOW_STALL = 2


def mhla_set_debug(option: int, value: int) -> None:
    """Testing hooks of the fused launch's waits (see mhla.h)."""
    _check(load().mhla_set_debug(int(option), int(value)), "mhla_set_debug")


def mhla_abi_version() -> int:
    return load().mhla_abi_version()


# --------------------------------------------------------------------------
# Operators around the attention.  Tensors may have any strides as long as
# the last axis is contiguous; nothing is copied to make them contiguous.
#
# A call's checks and its parameter block depend only on the arguments' shapes,
# strides, dtypes and devices, so they are made once for each such set and kept
# (a decoding loop calls with the same ones for every token).  Scalars among
# the arguments are taken by value before they become part of that key.
#
# Everything runs on torch's current stream, or on ``stream`` as it would under
# ``torch.cuda.stream(stream)``: what a call allocates belongs to that stream.

_CALLS: dict = {}
_MOST_CALLS = 4096


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _remember(key, call):
    if len(_CALLS) >= _MOST_CALLS:
        _CALLS.clear()
    _CALLS[key] = call
    return call


def _ptr(t):
    return None if t is None else t.data_ptr()


def _contiguous_like(t):
    import torch
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _axes(layout: str):
    """Positions of the batch, head and token axes."""
    if layout == "bhnd":
        return 0, 1, 2
    if layout == "bnhd":
        return 0, 2, 1
    raise ValueError(f"unknown layout {layout!r}; expected 'bhnd' or 'bnhd'")


def _choice(name, value, table):
    if value not in table:
        raise ValueError(f"unknown {name} {value!r}; expected one of {sorted(table)}")
    return table[value]


def _rows(name, t, like=None, dtype=None, shape=None):
    """Checks one tensor of rows (last axis contiguous, on the GPU)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")


def _flat(name, t, like, dtype, shape):
    """Checks one contiguous side tensor (None: not given)."""
    if t is None:
        return
    _rows(name, t, like, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _set_strides(field, t, axes) -> None:
    st = t.stride()
    field.batch, field.head, field.token = st[axes[0]], st[axes[1]], st[axes[2]]


def _set_output(field, name, t, like, shape, axes) -> None:
    """Strides of an output: the given tensor's, or those of a new contiguous one."""
    if t is not None:
        _rows(name, t, like, like.dtype, shape)
        _set_strides(field, t, axes)
        return
    st, step = [0, 0, 0], shape[3]
    for a in (2, 1, 0):
        st[a] = step
        step *= max(shape[a], 1)
    field.batch, field.head, field.token = st[axes[0]], st[axes[1]], st[axes[2]]


def _current_stream(index) -> int:
    import torch
    return torch.cuda.current_stream(index).cuda_stream


class _Call:
    """An entry point with its parameter block and what its wrapper needs beside them."""

    def __init__(self, entry, like, params, need=0, **kw):
        import torch
        self.entry, self.call = entry, getattr(load(), entry)
        self.params, self.ref, self.need = params, ctypes.byref(params), need
        self.device, self.index = like.device, like.get_device()
        self.empty, self.f32, self.u8 = torch.empty, torch.float32, torch.uint8
        # the current stream's handle without a Stream object (0.1 us against 1.1)
        self.current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _current_stream
        self.current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        self.__dict__.update(kw)

    def stream(self) -> int:
        if self.current_device() != self.index:
            raise _not_current(self.index)
        return self.current(self.index)

    def workspace(self, given):
        """(tensor or None, bytes): the caller's workspace or a new one."""
        if given is not None:
            return given, _buffer_bytes("workspace", given, self.device)
        if not self.need:
            return None, 0
        return self.empty(self.need, dtype=self.u8, device=self.device), self.need


def _fresh(t):
    """What makes a contiguous tensor shaped and typed like t."""
    import torch
    return torch.empty_like if t.is_contiguous() else _contiguous_like


class RotaryPlan:
    """The frequencies of a rotation, made once by :func:`mhla_rotary_plan`."""

    def __init__(self, rot_dim: int, table: MhlaRotaryTable):
        self.rot_dim = rot_dim
        self.table = table
        self._ref = ctypes.byref(table)

    @property
    def amplitude(self) -> float:
        return self.table.amplitude


def mhla_rotary_plan(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_length: float = 0.0) -> RotaryPlan:
    """Frequencies for the first ``rot_dim`` entries of a head (see mhla_rotary_table_init in mhla.h).

    ``scaling``: "none", "linear" (positions divided by ``factor``), "base"
    (a larger base) or "parts" (slow frequencies interpolated, fast ones kept;
    needs ``original_length``).
    """
    table = MhlaRotaryTable()
    _check(load().mhla_rotary_table_init(int(rot_dim), float(base), _choice("scaling", scaling, ROTARY_SCALINGS),
                                         float(factor), float(original_length), ctypes.byref(table)),
           "mhla_rotary_table_init")
    return RotaryPlan(int(rot_dim), table)


def _rotary_call(q, k, positions, style, layout, q_out, k_out, transpose):
    import torch
    axes = _axes(layout)
    p = MhlaRotaryParams()
    p.style, p.transpose = _choice("style", style, ROTARY_STYLES), transpose
    if q.dim() != 4:
        raise ValueError("q and k must be [B, H, N, d] (layout 'bhnd') or [B, N, H, d] (layout 'bnhd')")
    _rows("q", q)
    shape = q.shape
    p.batch, p.heads, p.tokens, p.head_dim = shape[0], shape[axes[1]], shape[axes[2]], shape[3]
    p.dtype = DTYPES[_torch_dtype_name(q)]
    _set_strides(p.q, q, axes)
    _set_output(p.q_out, "q_out", q_out, q, shape, axes)
    if k is not None:
        want = list(shape)
        want[axes[1]] = k.shape[axes[1]] if k.dim() == 4 else -1
        _rows("k", k, q, q.dtype, want)
        p.kv_heads = k.shape[axes[1]]
        _set_strides(p.k, k, axes)
        _set_output(p.k_out, "k_out", k_out, q, k.shape, axes)
    elif k_out is not None:
        raise ValueError("k_out needs k")
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
        if not positions.is_cuda or positions.device != q.device:
            raise ValueError(f"positions must be on {q.device}")
        if positions.dim() == 1 and positions.shape[0] == p.tokens:
            p.position_token_stride = positions.stride(0)
        elif positions.dim() == 2 and tuple(positions.shape) in ((p.batch, p.tokens), (1, p.tokens)):
            p.position_batch_stride = positions.stride(0) if positions.shape[0] > 1 else 0
            p.position_token_stride = positions.stride(1)
        else:
            raise ValueError(f"positions must be [N] or [B, N], got {tuple(positions.shape)}")
        p.position_dtype = 1 if positions.dtype == torch.int64 else 0
    return _Call("mhla_rotary", q, p, new_q=_fresh(q), new_k=None if k is None else _fresh(k))


def _rotary(q, k, plan, positions, offset, style, layout, q_out, k_out, stream, transpose, where):
    if stream is not None:
        return _on_stream(stream, q, (q_out, k_out), lambda: _rotary(
            q, k, plan, positions, offset, style, layout, q_out, k_out, None, transpose, where))
    key = ("rotary", transpose, style, layout, _sig(q), _sig(k), _sig(positions), _sig(q_out), _sig(k_out))
    c = _CALLS.get(key) or _remember(key, _rotary_call(q, k, positions, style, layout, q_out, k_out, transpose))
    if q_out is None:
        q_out = c.new_q(q)
    if k_out is None and k is not None:
        k_out = c.new_k(k)
    ref = c.ref
    if offset:  # changes from token to token: in a block of its own
        p = MhlaRotaryParams.from_buffer_copy(c.params)
        p.position_offset = int(offset)
        ref = ctypes.byref(p)
    status = c.call(q.data_ptr(), None if k is None else k.data_ptr(),
                    None if positions is None else positions.data_ptr(), plan._ref, ref, q_out.data_ptr(),
                    None if k is None else k_out.data_ptr(), c.stream())
    if status:
        raise MhlaError(status, where)
    return q_out, k_out


def mhla_rotary_forward(q, k, plan: RotaryPlan, positions=None, offset: int = 0, style: str = "half",
                        layout: str = "bhnd", q_out=None, k_out=None, stream=None):
    """Rotary positions on queries and keys; returns ``(q_out, k_out)``.

    ``k`` may be None and may have another number of heads than ``q``.
    ``positions``: int32 or int64 [N] or [B, N] on the GPU; without it token t
    has position ``offset + t``.  ``style``: "half" pairs entry i with
    i + rot_dim / 2, "interleaved" 2i with 2i + 1.  ``q_out is q`` and
    ``k_out is k`` rotate in place.
    """
    return _rotary(q, k, plan, positions, offset, style, layout, q_out, k_out, stream, 0, "mhla_rotary_forward")


def mhla_rotary_backward(dq_out, dk_out, plan: RotaryPlan, positions=None, offset: int = 0, style: str = "half",
                         layout: str = "bhnd", dq=None, dk=None, stream=None):
    """Gradients of q and k from those of mhla_rotary_forward's results: ``(dq, dk)``."""
    return _rotary(dq_out, dk_out, plan, positions, offset, style, layout, dq, dk, stream, 1, "mhla_rotary_backward")


def _norm_rows(name, t, like=None):
    """(rows, cols, stride) of a tensor whose leading axes collapse into rows of one stride."""
    _rows(name, t, like, like.dtype if like is not None else None, like.shape if like is not None else None)
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one axis")
    cols = t.shape[-1]
    rows, stride = 1, None
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * rows and t.numel():
            raise ValueError(f"the leading axes of {name} must collapse into rows of one stride")
        rows *= n
    return rows, cols, cols if stride is None else stride


def _norm_params(x, weight, bias, eps):
    p = MhlaLayernormParams()
    p.rows, p.cols, p.x_stride = _norm_rows("x", x)
    p.y_stride = p.cols
    if p.cols < 1:
        raise ValueError("x must have at least one column")
    p.dtype = DTYPES[_torch_dtype_name(x)]
    p.weight_dtype = DTYPE_F32
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _flat(name, t, x, None, (p.cols,))
            p.weight_dtype = DTYPES[_torch_dtype_name(t)]
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same dtype")
    p.eps = eps
    return p


def _norm_forward_call(x, weight, bias, eps, out, mean, rstd):
    import torch
    p = _norm_params(x, weight, bias, eps)
    if out is not None:
        _, _, p.y_stride = _norm_rows("out", out, x)
    _flat("mean", mean, x, torch.float32, x.shape[:-1])
    _flat("rstd", rstd, x, torch.float32, x.shape[:-1])
    return _Call("mhla_layernorm_forward", x, p, new=_fresh(x), lead=x.shape[:-1])


def mhla_layernorm_forward(x, weight=None, bias=None, eps: float = 1e-5, out=None, mean=None, rstd=None, stream=None):
    """Layer norm over the last axis; returns ``(y, mean, rstd)``.

    ``weight`` and ``bias`` are [cols], bfloat16 or float32; ``mean`` and
    ``rstd`` are float32 of x's leading shape, for the backward call.
    ``out is x`` normalises in place.
    """
    if stream is not None:
        return _on_stream(stream, x, (out, mean, rstd), lambda: mhla_layernorm_forward(
            x, weight, bias, eps, out, mean, rstd))
    eps = float(eps)
    key = ("norm", eps, _sig(x), _sig(weight), _sig(bias), _sig(out), _sig(mean), _sig(rstd))
    c = _CALLS.get(key) or _remember(key, _norm_forward_call(x, weight, bias, eps, out, mean, rstd))
    if out is None:
        out = c.new(x)
    if mean is None:
        mean = c.empty(c.lead, dtype=c.f32, device=c.device)
    if rstd is None:
        rstd = c.empty(c.lead, dtype=c.f32, device=c.device)
    status = c.call(x.data_ptr(), _ptr(weight), _ptr(bias), c.ref, out.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                    c.stream())
    if status:
        raise MhlaError(status, "mhla_layernorm_forward")
    return out, mean, rstd


def mhla_layernorm_backward_workspace_bytes(p: MhlaLayernormParams) -> int:
    n = ctypes.c_size_t(0)
    _check(load().mhla_layernorm_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)),
           "mhla_layernorm_backward_workspace_bytes")
    return n.value


def _norm_backward_call(dy, x, mean, rstd, weight, dx, dweight, dbias, params):
    import torch
    p = _norm_params(x, weight, None, 0.0)
    _, _, p.dy_stride = _norm_rows("dy", dy, x)
    if dx is not None:
        _, _, p.y_stride = _norm_rows("dx", dx, x)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _flat(name, t, x, torch.float32, x.shape[:-1])
    for name, t in (("dweight", dweight), ("dbias", dbias)):
        if t is not None and not params:
            raise ValueError(f"{name} needs params=True")
        _flat(name, t, x, torch.float32, (p.cols,))
    return _Call("mhla_layernorm_backward", x, p, mhla_layernorm_backward_workspace_bytes(p) if params else 0,
                 new=_fresh(x), cols=p.cols)


def mhla_layernorm_backward(dy, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, workspace=None,
                            stream=None, params: bool = True):
    """Gradients of mhla_layernorm_forward: ``(dx, dweight, dbias)``.

    ``dweight`` and ``dbias`` are float32 [cols], summed over the rows in a
    fixed order; ``params=False`` leaves them out (None).  ``dx is dy`` or
    ``dx is x`` overwrites that input.
    """
    if stream is not None:
        return _on_stream(stream, x, (dx, dweight, dbias), lambda: mhla_layernorm_backward(
            dy, x, mean, rstd, weight, dx, dweight, dbias, workspace, params=params))
    params = bool(params)
    key = ("norm backward", params, _sig(dy), _sig(x), _sig(mean), _sig(rstd), _sig(weight), _sig(dx), _sig(dweight),
           _sig(dbias))
    c = _CALLS.get(key) or _remember(key, _norm_backward_call(dy, x, mean, rstd, weight, dx, dweight, dbias, params))
    if dx is None:
        dx = c.new(x)
    ws_bytes = 0
    if params:
        if dweight is None:
            dweight = c.empty(c.cols, dtype=c.f32, device=c.device)
        if dbias is None:
            dbias = c.empty(c.cols, dtype=c.f32, device=c.device)
        workspace, ws_bytes = c.workspace(workspace)
    status = c.call(dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(), c.ref, dx.data_ptr(),
                    _ptr(dweight), _ptr(dbias), _ptr(workspace) if params else None, ws_bytes, c.stream())
    if status:
        raise MhlaError(status, "mhla_layernorm_backward")
    return dx, dweight, dbias


def _decay_params(q, k, v, log_decay, scale, layout, variant):
    """(params, axes) of q, k [B, H, N, dk] and v [B, H, N, dv] ('bhnd') or their token-major forms."""
    import torch
    axes = _axes(layout)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d] (layout 'bhnd') or [B, N, H, d] (layout 'bnhd')")
    _rows("q", q)
    _rows("k", k, q, q.dtype, q.shape)
    _rows("v", v, q, q.dtype, tuple(q.shape[:3]) + (v.shape[3],))
    p = MhlaDecayParams()
    shape = q.shape
    p.batch, p.heads, p.tokens = shape[0], shape[axes[1]], shape[axes[2]]
    p.key_dim, p.value_dim = shape[3], v.shape[3]
    p.dtype = DTYPES[_torch_dtype_name(q)]
    p.variant = _choice("variant", variant, DECAY_VARIANTS)
    p.scale = scale
    _flat("log_decay", log_decay, q, torch.float32, (p.heads,))
    _set_strides(p.q, q, axes)
    _set_strides(p.k, k, axes)
    _set_strides(p.v, v, axes)
    return p, axes


def _decay_side(p, like, lengths, **states):
    import torch
    _flat("lengths", lengths, like, torch.int32, (p.batch,))
    shape = (p.batch, p.heads, p.key_dim, p.value_dim)
    for name, t in states.items():
        _flat(name, t, like, torch.float32, shape)
    return shape


def mhla_decay_workspace_bytes(p: MhlaDecayParams) -> int:
    n = ctypes.c_size_t(0)
    _check(load().mhla_decay_workspace_bytes(ctypes.byref(p), ctypes.byref(n)), "mhla_decay_workspace_bytes")
    return n.value


def _decay_forward_call(q, k, v, log_decay, state, lengths, scale, layout, variant, out, state_out):
    p, axes = _decay_params(q, k, v, log_decay, scale, layout, variant)
    _set_output(p.out, "out", out, q, v.shape, axes)
    shape = _decay_side(p, q, lengths, state=state, state_out=state_out)
    return _Call("mhla_decay_forward", q, p, mhla_decay_workspace_bytes(p), new=_fresh(v), shape=shape)


def mhla_decay_forward(q, k, v, log_decay, state=None, lengths=None, scale: float = 1.0, layout: str = "bhnd",
                       variant: str = "auto", out=None, state_out=None, workspace=None, stream=None):
    """Linear attention with a decay for each head over whole prompts: ``(out, state_out)``.

    S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T and o_t = scale S_t^T q_t.
    q, k: [B, H, N, dk], v: [B, H, N, dv] ('bhnd'; 'bnhd' is token-major), dk
    and dv each 16, 32, 64 or 128, bfloat16 or float32.  ``log_decay``:
    float32 [H].  ``state``: float32 [B, H, dk, dv] to start from (None:
    zeros); ``state_out is state`` updates it in place.  ``lengths``: int32
    [B] for sequences padded to N; rows past a length come out as zeros.
    bfloat16 runs on the tensor cores with operands rounded to bfloat16 from
    N = 128 on, padding included (see mhla.h); ``variant="simt"`` rounds the
    results only.
    """
    if stream is not None:
        return _on_stream(stream, q, (out, state_out), lambda: mhla_decay_forward(
            q, k, v, log_decay, state, lengths, scale, layout, variant, out, state_out, workspace))
    scale = float(scale)
    key = ("decay", scale, layout, variant, _sig(q), _sig(k), _sig(v), _sig(log_decay), _sig(state), _sig(lengths),
           _sig(out), _sig(state_out))
    c = _CALLS.get(key) or _remember(key, _decay_forward_call(q, k, v, log_decay, state, lengths, scale, layout,
                                                              variant, out, state_out))
    if out is None:
        out = c.new(v)
    if state_out is None:
        state_out = c.empty(c.shape, dtype=c.f32, device=c.device)
    workspace, ws_bytes = c.workspace(workspace)
    status = c.call(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(lengths), _ptr(state), c.ref,
                    out.data_ptr(), state_out.data_ptr(), _ptr(workspace), ws_bytes, c.stream())
    if status:
        raise MhlaError(status, "mhla_decay_forward")
    return out, state_out


def mhla_decay_backward_workspace_bytes(p: MhlaDecayParams) -> int:
    n = ctypes.c_size_t(0)
    _check(load().mhla_decay_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(n)),
           "mhla_decay_backward_workspace_bytes")
    return n.value


def _decay_backward_call(q, k, v, log_decay, dout, state, dstate_out, lengths, scale, layout, variant, dq, dk, dv,
                         dstate):
    p, axes = _decay_params(q, k, v, log_decay, scale, layout, variant)
    _rows("dout", dout, q, q.dtype, v.shape)
    _set_strides(p.dout, dout, axes)
    _set_output(p.dq, "dq", dq, q, q.shape, axes)
    _set_output(p.dk, "dk", dk, q, q.shape, axes)
    _set_output(p.dv, "dv", dv, q, v.shape, axes)
    shape = _decay_side(p, q, lengths, state=state, dstate_out=dstate_out, dstate=dstate)
    return _Call("mhla_decay_backward", q, p, mhla_decay_backward_workspace_bytes(p), new_q=_fresh(q), new_k=_fresh(k),
                 new_v=_fresh(v), shape=shape)


def mhla_decay_backward(q, k, v, log_decay, dout, state=None, dstate_out=None, lengths=None, scale: float = 1.0,
                        layout: str = "bhnd", variant: str = "auto", dq=None, dk=None, dv=None, dstate=None,
                        workspace=None, stream=None):
    """Gradients of mhla_decay_forward: ``(dq, dk, dv, dstate)``.

    ``dout`` is the gradient of out and ``dstate_out`` that of the final state
    (None: zeros); ``dstate`` is the gradient of the starting state (float32
    [B, H, dk, dv]; None without one, unless a tensor is given for it).
    Arguments as in the forward call.
    """
    if stream is not None:
        return _on_stream(stream, q, (dq, dk, dv, dstate), lambda: mhla_decay_backward(
            q, k, v, log_decay, dout, state, dstate_out, lengths, scale, layout, variant, dq, dk, dv, dstate, workspace))
    scale = float(scale)
    key = ("decay backward", scale, layout, variant, _sig(q), _sig(k), _sig(v), _sig(log_decay), _sig(dout),
           _sig(state), _sig(dstate_out), _sig(lengths), _sig(dq), _sig(dk), _sig(dv), _sig(dstate))
    c = _CALLS.get(key) or _remember(key, _decay_backward_call(q, k, v, log_decay, dout, state, dstate_out, lengths,
                                                               scale, layout, variant, dq, dk, dv, dstate))
    dq = c.new_q(q) if dq is None else dq
    dk = c.new_k(k) if dk is None else dk
    dv = c.new_v(v) if dv is None else dv
    if dstate is None and state is not None:
        dstate = c.empty(c.shape, dtype=c.f32, device=c.device)
    workspace, ws_bytes = c.workspace(workspace)
    status = c.call(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(lengths), _ptr(state),
                    dout.data_ptr(), _ptr(dstate_out), c.ref, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(dstate),
                    _ptr(workspace), ws_bytes, c.stream())
    if status:
        raise MhlaError(status, "mhla_decay_backward")
    return dq, dk, dv, dstate


def _decay_step_call(q, k, v, log_decay, state, scale, out, state_out):
    import torch
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be [B, H, d]")
    _rows("q", q)
    _rows("k", k, q, q.dtype, q.shape)
    _rows("v", v, q, q.dtype, tuple(q.shape[:2]) + (v.shape[2],))
    p = MhlaDecayParams()
    p.batch, p.heads, p.key_dim = q.shape
    p.tokens, p.value_dim = 1, v.shape[2]
    p.dtype = DTYPES[_torch_dtype_name(q)]
    p.scale = scale
    _flat("log_decay", log_decay, q, torch.float32, (p.heads,))
    if state is None:
        raise ValueError("state must be given")
    _decay_side(p, q, None, state=state, state_out=state_out)
    for field, t in ((p.q, q), (p.k, k), (p.v, v)):
        field.batch, field.head = t.stride(0), t.stride(1)
    if out is not None:
        _rows("out", out, q, q.dtype, v.shape)
        p.out.batch, p.out.head = out.stride(0), out.stride(1)
    else:
        p.out.batch, p.out.head = v.shape[1] * v.shape[2], v.shape[2]
    return _Call("mhla_decay_step", q, p, new=_fresh(v))


def mhla_decay_step(q, k, v, log_decay, state, scale: float = 1.0, out=None, state_out=None, stream=None):
    """One token of every sequence: returns ``out`` [B, H, dv].

    q, k: [B, H, dk], v: [B, H, dv]; ``state`` float32 [B, H, dk, dv] is
    updated in place unless ``state_out`` is given.
    """
    if stream is not None:
        return _on_stream(stream, q, (out,), lambda: mhla_decay_step(
            q, k, v, log_decay, state, scale, out, state_out))
    scale = float(scale)
    key = ("decay step", scale, _sig(q), _sig(k), _sig(v), _sig(log_decay), _sig(state), _sig(out), _sig(state_out))
    c = _CALLS.get(key) or _remember(key, _decay_step_call(q, k, v, log_decay, state, scale, out, state_out))
    if out is None:
        out = c.new(v)
    at = state.data_ptr()
    status = c.call(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), at, c.ref, out.data_ptr(),
                    at if state_out is None else state_out.data_ptr(), c.stream())
    if status:
        raise MhlaError(status, "mhla_decay_step")
    return out
