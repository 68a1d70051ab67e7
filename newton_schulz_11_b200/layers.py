"""The layers around the weight matrices, and their gradients (see include/muon_b200.h).

Every operation runs in libmuon_b200.so; the module _layers (csrc/layers_binding.cpp) checks
the tensors, allocates what is not given and makes the call.  The functions take and return
plain tensors and record nothing for autograd; the backward functions write the gradients
that `muon_step` and `adamw_step` read (fp32, into the buffers given, optionally added to
what they hold).

All matrices are 2-D with unit stride along the last dimension (flatten leading dimensions
with `reshape`); bf16 and fp32 may be mixed as each function says.  Work is queued on
`stream`, by default the current stream of the tensors' device; outputs and scratch that a
call allocates come from PyTorch's allocator on that stream, so calls on different streams
and captured graphs share nothing.  A `workspace` given is the caller's to keep to one call
at a time, on the tensors' device; it may be the one that `muon_step` uses, whose status the
layers leave alone.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import MUON_ACTS, MuonError, MuonLibraryError, check, lib

_binding = None
_lock = threading.Lock()


def _ops():
    """The module _layers, imported on first use."""
    global _binding
    if _binding is None:
        with _lock:
            if _binding is None:
                lib()  # the library's own errors first
                try:
                    from . import _layers
                except ImportError as e:
                    raise MuonLibraryError(f"cannot load {os.path.join(_lib.PKG, '_layers.so')} ({e}); run "
                                           "`python -m newton_schulz_11_b200.build`") from e
                _layers.set_error(MuonError)
                _binding = _layers
    return _binding


def _act_code(act) -> int:
    code = MUON_ACTS.get("none" if act is None else act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}, expected one of {tuple(MUON_ACTS)}")
    return code


def _on(stream, t):
    """A context in which `stream`, which has to be on t's device, is the current stream."""
    if isinstance(t, torch.Tensor) and t.is_cuda and stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


def layer_norm(x: torch.Tensor, gain: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
               eps: float = 1e-5, out: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """y = (x - mean) rstd gain + bias over the rows of x; returns (y, mean, rstd).

    x [tokens, width] fp32 or bf16, y the same dtype; gain and bias [width], each fp32 or
    bf16, or None; mean and rstd are fp32 [tokens], what layer_norm_backward reads.
    """
    if stream is not None:
        with _on(stream, x):
            return layer_norm(x, gain, bias, eps=eps, out=out)
    return _ops().layer_norm(x, gain, bias, eps, out)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        gain: Optional[torch.Tensor] = None, *, skip: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, dgain: Optional[torch.Tensor] = None,
                        dbias: Optional[torch.Tensor] = None, need_dx: bool = True, need_dgain: bool = True,
                        need_dbias: bool = True, accumulate: bool = False, workspace=None, stream=None):
    """Gradients of layer_norm: (dx, dgain, dbias), None where not needed.

    dy and dx have x's dtype; mean and rstd are what layer_norm returned.  `skip` (fp32 or
    bf16) is added to dx: the gradient that the residual connection around the norm carries;
    dx may be the same tensor.  dgain and dbias are fp32 [width] (allocated when None); with
    `accumulate` those that are needed must be given and the gradients are added to them.  A
    norm without a bias has need_dbias=False.
    """
    if stream is not None:
        with _on(stream, x):
            return layer_norm_backward(dy, x, mean, rstd, gain, skip=skip, dx=dx, dgain=dgain, dbias=dbias,
                                       need_dx=need_dx, need_dgain=need_dgain, need_dbias=need_dbias,
                                       accumulate=accumulate, workspace=workspace)
    return _ops().layer_norm_backward(dy, x, mean, rstd, gain, skip, dx, dgain, dbias, need_dx, need_dgain, need_dbias,
                                      accumulate, workspace)


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
    if stream is not None:
        with _on(stream, x):
            return linear(x, w, bias, act=act, residual=residual, out=out, save_preact=save_preact, preact=preact,
                          workspace=workspace)
    return _ops().linear(x, w, bias, _act_code(act), residual, out, save_preact, preact, workspace)


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
    if stream is not None:
        with _on(stream, dy):
            return linear_backward(dy, x, w, in_act=in_act, in_preact=in_preact, skip=skip, dx=dx, dw=dw, db=db,
                                   need_dx=need_dx, need_dw=need_dw, need_db=need_db, accumulate=accumulate,
                                   workspace=workspace)
    return _ops().linear_backward(dy, x, w, _act_code(in_act), in_preact, skip, dx, dw, db, need_dx, need_dw, need_db,
                                  accumulate, workspace)


def activation_backward(dy: torch.Tensor, preact: torch.Tensor, act: str, *, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """dz = dy act'(z) for z = preact; dy and dz of one dtype, z fp32 or bf16."""
    if stream is not None:
        with _on(stream, dy):
            return activation_backward(dy, preact, act, out=out)
    return _ops().activation_backward(dy, preact, _act_code(act), out)


def layers_status(device=None, *, clear: bool = False, stream=None) -> Tuple[int, int]:
    """(code, where) of the device's status word for the functions above (synchronises the
    stream): MUON_OK, or MUON_ERR_TIMEOUT and the wait site of a bounded wait that ran out."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    code, where = ctypes.c_int32(0), ctypes.c_int32(0)
    with torch.cuda.device(device):
        s = (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream
        check(lib().muon_layers_status(s, 1 if clear else 0, ctypes.byref(code), ctypes.byref(where)),
              "muon_layers_status")
    return int(code.value), int(where.value)
