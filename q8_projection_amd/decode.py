"""Python binding of include/q8_decode.h: the mixture-of-experts layer and the
sampler.

As in the package's other wrappers, argument marshalling only.  Every tensor of
a call lives on one device, and the call runs on that device whichever is
current, on ``stream`` (a torch stream or a raw handle) or else on that device's
current stream.  Outputs and workspaces that are not passed are allocated here,
and cleared where that is needed, on the same stream.
"""
from __future__ import annotations

import ctypes

import torch

import q8_projection_amd as _q8

_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8


class _MoeLayerC(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("k", ctypes.c_int64), ("ff", ctypes.c_int64),
                ("router", ctypes.c_void_p), ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p)]


def _need(t, name: str, dtype, shape, device):
    """Raise ValueError unless t is a contiguous tensor of this dtype, shape and device."""
    if type(t) is torch.Tensor and t.dtype == dtype and t.device == device and t.shape == shape and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, not {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_fns = {}


def _call(fn: str, device, rows: int, *args):
    """Call a library function on `device` and its current stream."""
    if rows == 0:
        return  # an empty tensor has no address; there is nothing to enqueue
    f = _fns.get(fn)
    if f is None:
        f = _fns[fn] = getattr(_q8.lib(), fn)
    raw = _raw_stream(device.index)
    if _current_device() == device.index:
        status = f(*args, raw)
    else:
        with torch.cuda.device(device):
            status = f(*args, raw)
    if status != 0:
        raise _q8.Q8Error(fn, status)


def _on_stream(stream, device, fn, *args):
    """fn(*args) with `stream` (a torch stream or a raw handle) current, so that what the
    call allocates, and the workspace it clears, is ordered on that stream as well."""
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream must be one of {device}, not of {stream.device}")
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        result = fn(*args)
    for t in result if isinstance(result, tuple) else (result,):
        if t is not None:
            t.record_stream(caller)  # where the caller, once it has waited, reads it
    return result


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


_current_device = torch.cuda.current_device
# the same two answers without the wrappers around them, where torch has them (1-2 us a call)
if hasattr(torch._C, "_cuda_getCurrentRawStream") and hasattr(torch._C, "_cuda_getDevice"):
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice


def _ptr(t):
    return None if t is None else t.data_ptr()


class MoeLayer:
    """A layer's Q8_0 experts and router, checked once.

    w_gate, w_up: uint8 Q8_0 blocks [experts][ff][k/32*34]; w_down [experts][k][ff/32*34];
    router f32 [experts][k] (None: choices are given to ``moe_experts``).  The tensors
    are used in place and kept alive by this object.
    """

    def __init__(self, mode, w_gate, w_up, w_down, k: int, ff: int, top_k: int, router=None,
                 renormalize: bool = True):
        if not isinstance(w_gate, torch.Tensor) or w_gate.dim() < 2:
            raise ValueError("w_gate must be a tensor [experts][ff][k/32*34]")
        if not w_gate.is_cuda:
            raise ValueError("w_gate must be a device tensor")
        self.device = w_gate.device
        experts = w_gate.shape[0]
        for name, t, n, cols in (("w_gate", w_gate, ff, k), ("w_up", w_up, ff, k), ("w_down", w_down, k, ff)):
            _need(t, name, _U8, (experts, n, cols // _q8.BLOCK * _q8.BLOCK_BYTES), self.device)
        if router is not None:
            _need(router, "router", _F32, (experts, k), self.device)
        self.mode = _q8._mode(mode)
        self.experts, self.top_k, self.k, self.ff = experts, int(top_k), int(k), int(ff)
        self._tensors = (w_gate, w_up, w_down, router)
        self._c = _MoeLayerC(self.mode, experts, self.top_k, int(bool(renormalize)), k, ff,
                             None if router is None else router.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
                             w_down.data_ptr())
        self._ref = ctypes.addressof(self._c)
        self._bytes = {}
        if self.workspace_bytes(1) == 0:
            raise ValueError(f"the library does not take this layer: mode {mode}, {experts} experts, top_k {top_k}, "
                             f"k {k}, ff {ff}")

    def workspace_bytes(self, rows: int) -> int:
        """Bytes of the workspace for `rows` rows."""
        rows = min(int(rows), 64)
        if rows not in self._bytes:
            self._bytes[rows] = int(_q8.lib().q8_moe_workspace_bytes(self._ref, rows))
        return self._bytes[rows]

    def workspace(self, rows: int) -> torch.Tensor:
        """A zero-filled workspace for calls of up to `rows` rows."""
        return torch.zeros(self.workspace_bytes(rows), dtype=_U8, device=self.device)


def moe_workspace_bytes(layer: MoeLayer, rows: int) -> int:
    return layer.workspace_bytes(rows)


def _rows(layer, x):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a tensor [rows][k]")
    _need(x, "x", _F32, (x.shape[0], layer.k), layer.device)
    return x.shape[0]


def _work(layer, rows, workspace):
    if workspace is None:
        return layer.workspace(rows)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != _U8 or workspace.device != layer.device or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the layer's device")
    return workspace


def _out(t, name, dtype, shape, layer):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=layer.device)
    _need(t, name, dtype, shape, layer.device)
    return t


def moe_route(layer: MoeLayer, x: torch.Tensor, ids=None, gates=None, workspace=None, stream=None):
    """(ids int32, gates f32) [rows][top_k] that the layer's router chooses."""
    if stream is not None:
        return _on_stream(stream, layer.device, moe_route, layer, x, ids, gates, workspace)
    rows = _rows(layer, x)
    ids = _out(ids, "ids", _I32, (rows, layer.top_k), layer)
    gates = _out(gates, "gates", _F32, (rows, layer.top_k), layer)
    workspace = _work(layer, rows, workspace)
    _call("q8_moe_route", layer.device, rows, layer._ref, x.data_ptr(), rows, ids.data_ptr(), gates.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return ids, gates


def moe_experts(layer: MoeLayer, x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor, residual=None, out=None,
                workspace=None, stream=None) -> torch.Tensor:
    """y [rows][k] = residual + the gated sum of the given experts (ids outside the layer add nothing)."""
    if stream is not None:
        return _on_stream(stream, layer.device, moe_experts, layer, x, ids, gates, residual, out, workspace)
    rows = _rows(layer, x)
    _need(ids, "ids", _I32, (rows, layer.top_k), layer.device)
    _need(gates, "gates", _F32, (rows, layer.top_k), layer.device)
    if residual is not None:
        _need(residual, "residual", _F32, (rows, layer.k), layer.device)
    out = _out(out, "out", _F32, (rows, layer.k), layer)
    workspace = _work(layer, rows, workspace)
    _call("q8_moe_experts", layer.device, rows, layer._ref, x.data_ptr(), rows, ids.data_ptr(),
          gates.data_ptr(), _ptr(residual), out.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    return out


def moe(layer: MoeLayer, x: torch.Tensor, residual=None, out=None, ids=None, gates=None, workspace=None, stream=None):
    """(y [rows][k], ids, gates): the whole layer, router and experts."""
    if stream is not None:
        return _on_stream(stream, layer.device, moe, layer, x, residual, out, ids, gates, workspace)
    rows = _rows(layer, x)
    if residual is not None:
        _need(residual, "residual", _F32, (rows, layer.k), layer.device)
    out = _out(out, "out", _F32, (rows, layer.k), layer)
    ids = _out(ids, "ids", _I32, (rows, layer.top_k), layer)
    gates = _out(gates, "gates", _F32, (rows, layer.top_k), layer)
    workspace = _work(layer, rows, workspace)
    _call("q8_moe", layer.device, rows, layer._ref, x.data_ptr(), rows,
          _ptr(residual), out.data_ptr(), ids.data_ptr(), gates.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return out, ids, gates


def sample_workspace_bytes(rows: int, n: int) -> int:
    """Bytes of the sample workspace for `rows` rows of `n` logits (0: refused)."""
    return int(_q8.lib().q8_sample_workspace_bytes(rows, n))


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=None, top_k=None, top_p=None, min_p=None, idx=None,
           prob=None, workspace=None, stream=None):
    """(idx int32 [rows], prob f32 [rows]): one token drawn from each row of f32
    logits [rows][n] with the random numbers u f32 [rows].

    logits may have any row stride (a view of a wider buffer).  temperature,
    top_p, min_p (f32 [rows]) and top_k (int32 [rows]) are device tensors, or None
    where the filter is off.  The workspace (uint8, at least
    sample_workspace_bytes) is scratch and may be kept from call to call.
    """
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or logits.dtype != _F32 or not logits.is_cuda:
        raise ValueError("logits must be a f32 device tensor [rows][n]")
    if stream is not None:
        return _on_stream(stream, logits.device, sample, logits, u, temperature, top_k, top_p, min_p, idx, prob, workspace)
    rows, n = logits.shape
    if n > 1 and logits.stride(1) != 1:
        raise ValueError("logits must have unit stride within a row")
    ld = logits.stride(0) if rows > 1 else n
    dev = logits.device
    for t, name, dtype in ((u, "u", _F32), (temperature, "temperature", _F32), (top_k, "top_k", _I32),
                           (top_p, "top_p", _F32), (min_p, "min_p", _F32), (idx, "idx", _I32), (prob, "prob", _F32)):
        if t is not None:
            _need(t, name, dtype, (rows,), dev)
    if u is None:
        raise ValueError("u is required")
    if idx is None:
        idx = torch.empty(rows, dtype=_I32, device=dev)
    if prob is None:
        prob = torch.empty(rows, dtype=_F32, device=dev)
    if workspace is None:
        workspace = torch.empty(sample_workspace_bytes(rows, n), dtype=_U8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype != _U8 or workspace.device != dev or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the logits' device")
    _call("q8_sample", dev, rows, logits.data_ptr(), ld, rows, n, _ptr(temperature), _ptr(top_k), _ptr(top_p),
          _ptr(min_p), u.data_ptr(), idx.data_ptr(), prob.data_ptr(), workspace.data_ptr(), workspace.numel())
    return idx, prob
