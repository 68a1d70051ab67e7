"""The layers around the weight matrices, and their gradients (see include/muon_b200.h).

Argument marshalling only, like api.py: every operation runs in libmuon_b200.so.  The
functions take and return plain tensors and record nothing for autograd; the backward
functions write the gradients that `muon_step` and `adamw_step` read (fp32, into the
buffers given, optionally added to what they hold).

All matrices are 2-D with unit stride along the last dimension (flatten leading dimensions
with `reshape`); bf16 and fp32 may be mixed as each function says.  Work is queued on
`stream`, by default the current stream of the tensors' device; outputs and scratch that a
call allocates come from PyTorch's allocator on that stream, so calls on different streams
and captured graphs share nothing.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import MUON_ACTS, check, lib

_CODES = {torch.float32: _lib.MUON_F32, torch.bfloat16: _lib.MUON_BF16}
_ABSENT = (None, 0, 0, 0)
_byref = ctypes.byref
# Short calls are bound by this file's host time, so the current device and stream are asked
# for without building Python objects (0.2 us for both, against 2.4 us).
_device_index = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _matrix(t, what: str, rows: int, cols: int, device, dtype=None):
    """The four fields of a muon_view_t for a rows x cols matrix."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    code = _CODES.get(t.dtype)
    if code is None or (dtype is not None and t.dtype is not dtype):
        raise TypeError(f"{what} has dtype {t.dtype}, expected {dtype or 'float32 or bfloat16'}")
    if t.shape != (rows, cols):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{what} must have unit stride along its last dimension")
    if rows <= 1:
        s0 = cols
    elif s0 < cols:
        raise ValueError(f"{what} must not repeat rows (stride {s0} for {cols} columns)")
    return t.data_ptr(), s0, code, 0


def _vector(t, what: str, n: int, device, dtype=None):
    """The four fields of a muon_view_t for a contiguous vector of n elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    code = _CODES.get(t.dtype)
    if code is None or (dtype is not None and t.dtype is not dtype):
        raise TypeError(f"{what} has dtype {t.dtype}, expected {dtype or 'float32 or bfloat16'}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n} elements, got shape {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    return t.data_ptr(), n, code, 0


def _first(t, what: str):
    """Rows, columns and device of the call's first matrix."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must live on a CUDA device")
    return t.shape[0], t.shape[1], t.device


def _act_code(act) -> int:
    code = MUON_ACTS.get("none" if act is None else act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}, expected one of {tuple(MUON_ACTS)}")
    return code


def _elsewhere(device, stream):
    """A context in which `device` is current and `stream` its current stream, or None when
    that is so already."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    if _device_index() != device.index:
        return torch.cuda.device(device)
    return None


def _new(like: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """An uninitialised rows x cols matrix of like's dtype, on its device."""
    if like.is_contiguous() and like.shape == (rows, cols):
        return torch.empty_like(like)
    return like.new_empty((rows, cols))


def _scratch(size_fn, desc, workspace, device, stream: int):
    """(pointer, bytes, owner) of the call's scratch; the owner is held until it is queued."""
    need = ctypes.c_size_t(0)
    st = size_fn(_byref(desc), _byref(need))
    if st:
        check(st, size_fn.__name__)
    n = need.value
    if n == 0:
        return None, 0, None
    if workspace is not None:
        ptr, _ = workspace.ensure(n, stream)
        return ptr, n, workspace
    buf = torch.empty(n, dtype=torch.uint8, device=device)
    return buf.data_ptr(), n, buf


def layer_norm(x: torch.Tensor, gain: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
               eps: float = 1e-5, out: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """y = (x - mean) rstd gain + bias over the rows of x; returns (y, mean, rstd).

    x [tokens, width] fp32 or bf16, y the same dtype; gain and bias [width], each fp32 or
    bf16, or None; mean and rstd are fp32 [tokens], what layer_norm_backward reads.
    """
    rows, cols, device = _first(x, "x")
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return layer_norm(x, gain, bias, eps=eps, out=out)
    if out is None:
        out = _new(x, rows, cols)
    mean = x.new_empty(rows, dtype=torch.float32)
    rstd = torch.empty_like(mean)
    d = _lib.MuonLayerNorm(*_matrix(x, "x", rows, cols, device),
                           *(_ABSENT if gain is None else _vector(gain, "gain", cols, device)),
                           *(_ABSENT if bias is None else _vector(bias, "bias", cols, device)),
                           *_matrix(out, "out", rows, cols, device, x.dtype),
                           mean.data_ptr(), rstd.data_ptr(), rows, cols, eps, 0)
    st = lib().muon_layer_norm(_byref(d), _raw_stream(device.index))
    if st:
        check(st, "muon_layer_norm")
    return out, mean, rstd


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        gain: Optional[torch.Tensor] = None, *, skip: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, dgain: Optional[torch.Tensor] = None,
                        dbias: Optional[torch.Tensor] = None, accumulate: bool = False, workspace=None,
                        stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of layer_norm: (dx, dgain, dbias).

    dy and dx have x's dtype; mean and rstd are what layer_norm returned.  `skip` (fp32 or
    bf16) is added to dx: the gradient that the residual connection around the norm carries;
    dx may be the same tensor.  dgain and dbias are fp32 [width] (allocated when None); with
    `accumulate` they must be given and the gradients are added to them.
    """
    rows, cols, device = _first(x, "x")
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return layer_norm_backward(dy, x, mean, rstd, gain, skip=skip, dx=dx, dgain=dgain, dbias=dbias,
                                       accumulate=accumulate, workspace=workspace)
    if accumulate and (dgain is None or dbias is None):
        raise ValueError("accumulate needs dgain and dbias")
    f32 = torch.float32
    if dx is None:
        dx = _new(x, rows, cols)
    if dgain is None:
        dgain = x.new_empty(cols, dtype=f32)
    if dbias is None:
        dbias = x.new_empty(cols, dtype=f32)
    d = _lib.MuonLayerNormGrad(*_matrix(dy, "dy", rows, cols, device, x.dtype),
                               *_matrix(x, "x", rows, cols, device),
                               *(_ABSENT if gain is None else _vector(gain, "gain", cols, device)),
                               *(_ABSENT if skip is None else _matrix(skip, "skip", rows, cols, device)),
                               *_matrix(dx, "dx", rows, cols, device, x.dtype),
                               _vector(mean, "mean", rows, device, f32)[0],
                               _vector(rstd, "rstd", rows, device, f32)[0],
                               _vector(dgain, "dgain", cols, device, f32)[0],
                               _vector(dbias, "dbias", cols, device, f32)[0], rows, cols, 1 if accumulate else 0, 0)
    h, s = lib(), _raw_stream(device.index)
    ptr, size, _keep = _scratch(h.muon_layer_norm_backward_workspace, d, workspace, device, s)
    st = h.muon_layer_norm_backward(_byref(d), ptr, size, s)
    if st:
        check(st, "muon_layer_norm_backward")
    return dx, dgain, dbias


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *, act: Optional[str] = None,
           residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, save_preact: bool = False,
           preact: Optional[torch.Tensor] = None, workspace=None, stream=None):
    """y = act(z) + residual with z = x w^T + bias; returns y, or (y, z) when z is kept.

    x [tokens, in], w [out, in], bias [out], residual [tokens, out], each fp32 or bf16; y
    (`out`) and z (`preact`) are allocated in x's dtype when not given.  `out` may be the
    residual tensor.  z is kept with `save_preact` or when `preact` is given; it is what
    linear_backward and activation_backward take for the derivative.  act: None, "relu",
    "relu2", "gelu" (exact), "gelu_tanh" or "silu".
    """
    rows, n_in, device = _first(x, "x")
    n_out = _first(w, "w")[0]
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return linear(x, w, bias, act=act, residual=residual, out=out, save_preact=save_preact, preact=preact,
                          workspace=workspace)
    code = _act_code(act)
    xv = _matrix(x, "x", rows, n_in, device)
    if out is None:
        out = _new(x, rows, n_out)
    if save_preact and preact is None:
        preact = _new(x, rows, n_out)
    d = _lib.MuonLinear(*xv, *_matrix(w, "w", n_out, n_in, device),
                        *(_ABSENT if bias is None else _vector(bias, "bias", n_out, device)),
                        *(_ABSENT if residual is None else _matrix(residual, "residual", rows, n_out, device)),
                        *_matrix(out, "out", rows, n_out, device),
                        *(_ABSENT if preact is None else _matrix(preact, "preact", rows, n_out, device)),
                        rows, n_in, n_out, code, 0)
    h, s = lib(), _raw_stream(device.index)
    ptr, size, _keep = _scratch(h.muon_linear_workspace, d, workspace, device, s)
    st = h.muon_linear(_byref(d), ptr, size, s)
    if st:
        check(st, "muon_linear")
    return out if preact is None else (out, preact)


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, *, in_act: Optional[str] = None,
                    in_preact: Optional[torch.Tensor] = None, skip: Optional[torch.Tensor] = None,
                    dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                    db: Optional[torch.Tensor] = None, need_dx: bool = True, need_dw: bool = True,
                    need_db: bool = True, accumulate: bool = False, workspace=None, stream=None):
    """Gradients of z = x w^T + bias from dy = dL/dz: (dx, dw, db), None where not needed.

      dx = (dy w) act'(in_preact) + skip     dw (+)= dy^T x     db (+)= sum of dy over tokens

    When x is itself an activation's output, `in_act` and `in_preact` (the z that linear
    kept) fold that activation's derivative into dx, which is then the gradient of in_preact
    and the dy of the layer before.  (An activation whose output goes elsewhere has
    activation_backward; the residual's gradient is the output's own.)  `skip` is added to
    dx, which may be the same tensor.  dx is allocated in dy's dtype when not given; dw
    [out, in] and db [out] are fp32, what muon_step and adamw_step take; dw may be a strided
    view.  With `accumulate` the gradients are added to dw and db, which must be given.
    """
    rows, n_out, device = _first(dy, "dy")
    n_in = _first(w, "w")[1]
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return linear_backward(dy, x, w, in_act=in_act, in_preact=in_preact, skip=skip, dx=dx, dw=dw, db=db,
                                   need_dx=need_dx, need_dw=need_dw, need_db=need_db, accumulate=accumulate,
                                   workspace=workspace)
    code = _act_code(in_act)
    if code and need_dx and in_preact is None:
        raise ValueError("in_act needs in_preact")
    if accumulate and ((need_dw and dw is None) or (need_db and db is None)):
        raise ValueError("accumulate needs dw and db")
    if not (need_dx or need_dw or need_db):
        raise ValueError("nothing to compute")
    f32 = torch.float32
    dyv = _matrix(dy, "dy", rows, n_out, device)
    if not need_dx:
        dx = None
    elif dx is None:
        dx = _new(dy, rows, n_in)
    if not need_dw:
        dw = None
    elif dw is None:
        dw = dy.new_empty((n_out, n_in), dtype=f32)
    if not need_db:
        db = None
    elif db is None:
        db = dy.new_empty(n_out, dtype=f32)
    d = _lib.MuonLinearGrad(*dyv, *_matrix(x, "x", rows, n_in, device), *_matrix(w, "w", n_out, n_in, device),
                            *(_ABSENT if in_preact is None or not code
                              else _matrix(in_preact, "in_preact", rows, n_in, device)),
                            *(_ABSENT if skip is None or dx is None else _matrix(skip, "skip", rows, n_in, device)),
                            *(_ABSENT if dx is None else _matrix(dx, "dx", rows, n_in, device)),
                            *(_ABSENT if dw is None else _matrix(dw, "dw", n_out, n_in, device, f32)),
                            None if db is None else _vector(db, "db", n_out, device, f32)[0],
                            rows, n_in, n_out, code, 1 if accumulate else 0)
    h, s = lib(), _raw_stream(device.index)
    ptr, size, _keep = _scratch(h.muon_linear_backward_workspace, d, workspace, device, s)
    st = h.muon_linear_backward(_byref(d), ptr, size, s)
    if st:
        check(st, "muon_linear_backward")
    return dx, dw, db


def activation_backward(dy: torch.Tensor, preact: torch.Tensor, act: str, *, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """dz = dy act'(z) for z = preact; dy and dz of one dtype, z fp32 or bf16."""
    rows, cols, device = _first(dy, "dy")
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return activation_backward(dy, preact, act, out=out)
    code = _act_code(act)
    if code == 0:
        raise ValueError("act must name an activation")
    dyv = _matrix(dy, "dy", rows, cols, device)
    if out is None:
        out = _new(dy, rows, cols)
    d = _lib.MuonActivationGrad(*dyv, *_matrix(preact, "preact", rows, cols, device),
                                *_matrix(out, "out", rows, cols, device, dy.dtype), rows, cols, code, 0)
    st = lib().muon_activation_backward(_byref(d), _raw_stream(device.index))
    if st:
        check(st, "muon_activation_backward")
    return out


def layers_status(device=None, *, clear: bool = False, stream=None) -> Tuple[int, int]:
    """(code, where) of the device's status word for the functions above (synchronises the
    stream): MUON_OK, or MUON_ERR_TIMEOUT and the wait site of a bounded wait that ran out."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    code, where = ctypes.c_int32(0), ctypes.c_int32(0)
    with torch.cuda.device(device):
        s = _raw_stream(device.index) if stream is None else stream.cuda_stream
        check(lib().muon_layers_status(s, 1 if clear else 0, _byref(code), _byref(where)), "muon_layers_status")
    return int(code.value), int(where.value)
