"""Sequence mixers beside the SDM core: CausalConv.

Bindings of the sdm_conv_* calls of include/sdm.h.
Like SDM, each class borrows its parameters, runs on the current stream of its
inputs' device, raises SDMError for what the library refuses, and has no
fallback.  Inputs may be views with any batch and token strides; outputs are
new dense tensors unless given.
"""
from __future__ import annotations

import ctypes
from ctypes import c_int, c_int64

import torch

from . import (BF16, F32, FLAG_CONTINUE, SDMError, _check, _dev_tensor, _out_tensor, _same_device,
               _workspace, lib)

_F32, _BF16 = torch.float32, torch.bfloat16


def _p(t):
    return None if t is None else t.data_ptr()


class _On:
    """Makes a device current for a call, if another one is."""

    def __init__(self, device):
        self.index = device.index
        self.other = torch.cuda.current_device()

    def __enter__(self):
        if self.index != self.other:
            torch.cuda.set_device(self.index)
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        if self.index != self.other:
            torch.cuda.set_device(self.other)


def _dtype(t, name):
    if t.dtype == _F32:
        return F32
    if t.dtype == _BF16:
        return BF16
    raise SDMError(1, f"{name} must be float32 or bfloat16, got {t.dtype}")


def _param(t, name, shape, device=None):
    """A float32 parameter: a dense GPU tensor of this shape."""
    _dev_tensor(t, name, _F32)
    if tuple(t.shape) != tuple(shape):
        raise SDMError(1, f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise SDMError(1, f"{name} is on {t.device}, the other parameters on {device}")
    return t


def _view(t, name, like, shape, inner):
    """A strided input: a GPU tensor of this shape and of like's dtype and
    device, whose last `inner` dimensions are dense."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise SDMError(1, f"{name} must be a GPU tensor")
    if t.dtype != like.dtype:
        raise SDMError(1, f"{name} must be {like.dtype}, got {t.dtype}")
    _same_device(t, like, name)
    if tuple(t.shape) != tuple(shape):
        raise SDMError(1, f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    n = 1
    for d in range(t.dim() - 1, t.dim() - 1 - inner, -1):
        if t.shape[d] > 1 and t.stride(d) != n:
            raise SDMError(1, f"the last {inner} dimension(s) of {name} must be dense")
        n *= t.shape[d]
    return t


def _lengths(t, B, like):
    if t is not None:
        _out_tensor(t, "lengths", (B,), torch.int32, like)
    return t


class _ConvDesc(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int64), ("C", c_int), ("K", c_int), ("silu", c_int),
                ("dtype", c_int), ("x_batch", c_int64), ("x_token", c_int64)]


class CausalConv:
    """Short causal depthwise convolution, y = silu(bias + sum_k w[:, k] x[t - K + 1 + k]).

    weight [C, K] and bias [C] (or None) are float32 GPU tensors, borrowed.
    """

    def __init__(self, weight, bias=None, silu: bool = True):
        _dev_tensor(weight, "weight", _F32)
        if weight.dim() != 2:
            raise SDMError(1, "weight must be [C, K]")
        self.C, self.K = weight.shape
        if bias is not None:
            _param(bias, "bias", (self.C,), weight.device)
        self.weight, self.bias, self.silu = weight, bias, bool(silu)

    def _desc(self, x):
        if not isinstance(x, torch.Tensor) or x.dim() != 3:
            raise SDMError(1, f"x must be [B, T, {self.C}]")
        B, T = x.shape[:2]
        _view(x, "x", x, (B, T, self.C), 1)
        _same_device(self.weight, x, "weight")
        return _ConvDesc(B, T, self.C, self.K, int(self.silu), _dtype(x, "x"), x.stride(0),
                         x.stride(1))

    def forward(self, x, state=None, cont: bool = False, lengths=None, y=None):
        """(y, state): y [B, T, C], and the last K - 1 rows [B, K - 1, C].

        With cont=True `state` holds the rows before x and is updated in
        place; otherwise the rows before x are zeros (a given `state` is
        overwritten).  lengths [B] int32: tokens of each sequence.
        """
        d = self._desc(x)
        rows = (d.B, self.K - 1, self.C)
        if state is None:
            if cont:
                raise SDMError(1, "cont=True needs the state")
            state = torch.empty(rows, dtype=x.dtype, device=x.device)
        else:
            _out_tensor(state, "state", rows, x.dtype, x)
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            _out_tensor(y, "y", x.shape, x.dtype, x)
        _lengths(lengths, d.B, x)
        with _On(x.device) as stream:
            _check(lib().sdm_conv_forward(ctypes.byref(d), _p(x), _p(self.weight), _p(self.bias),
                                          _p(lengths), FLAG_CONTINUE if cont else 0, _p(y),
                                          _p(state), stream))
        return y, state

    def backward_workspace_size(self, x) -> int:
        """Bytes of workspace backward needs for inputs like x."""
        n = ctypes.c_size_t()
        _check(lib().sdm_conv_backward_workspace_size(ctypes.byref(self._desc(x)),
                                                      ctypes.byref(n)))
        return n.value

    def backward(self, x, dy, state=None, dstate=None, lengths=None, workspace=None) -> dict:
        """Gradients for dy [B, T, C] (and dstate, that of the final state, or
        None for zero): dx, float32 dweight and (with a bias) dbias, and, for a
        forward that started from `state`, dstate, its gradient."""
        d = self._desc(x)
        rows = (d.B, self.K - 1, self.C)
        _out_tensor(dy, "dy", x.shape, x.dtype, x)
        for t, name in ((state, "state"), (dstate, "dstate")):
            if t is not None:
                _out_tensor(t, name, rows, x.dtype, x)
        _lengths(lengths, d.B, x)
        workspace = _workspace(workspace, self.backward_workspace_size(x), x)
        out = dict(dx=torch.empty(x.shape, dtype=x.dtype, device=x.device),
                   dweight=torch.empty_like(self.weight))
        if self.bias is not None:
            out["dbias"] = torch.empty_like(self.bias)
        if state is not None:
            out["dstate"] = torch.empty(rows, dtype=x.dtype, device=x.device)
        with _On(x.device) as stream:
            _check(lib().sdm_conv_backward(
                ctypes.byref(d), _p(x), _p(self.weight), _p(self.bias), _p(lengths), _p(dy),
                _p(state), _p(dstate), _p(workspace), workspace.numel(), _p(out["dx"]),
                _p(out["dweight"]), _p(out.get("dbias")), _p(out.get("dstate")), stream))
        return out
