"""Sequence mixers beside the SDM core: CausalConv, SelectiveScan, WindowAttention.

Bindings of the sdm_conv_*, sdm_scan_* and sdm_window_* calls of include/sdm.h.
Like SDM, each class borrows its parameters, runs on the current stream of its
inputs' device, raises SDMError for what the library refuses, and has no
fallback.  Inputs may be views with any batch and token strides; outputs are
new dense tensors unless given.
"""
from __future__ import annotations

import ctypes
from ctypes import c_float, c_int, c_int64

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


class _ScanDesc(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int64), ("H", c_int), ("P", c_int), ("N", c_int),
                ("G", c_int), ("softplus", c_int), ("dtype", c_int), ("x_batch", c_int64),
                ("x_token", c_int64), ("B_batch", c_int64), ("B_token", c_int64),
                ("C_batch", c_int64), ("C_token", c_int64)]


class SelectiveScan:
    """Selective state space scan with one decay per head and token.

        S_t = exp(D_t A) S_{t-1} + D_t x_t B_t^T,   y_t = S_t C_t + D x_t,
        D_t = softplus(dt_t + dt_bias)  (softplus=False: dt_t + dt_bias)

    A [H], and D, dt_bias [H] or None, are float32 GPU tensors, borrowed.
    """

    def __init__(self, A, D=None, dt_bias=None, softplus: bool = True):
        _dev_tensor(A, "A", _F32)
        if A.dim() != 1:
            raise SDMError(1, "A must be [H]")
        self.H = A.shape[0]
        for t, name in ((D, "D"), (dt_bias, "dt_bias")):
            if t is not None:
                _param(t, name, (self.H,), A.device)
        self.A, self.D, self.dt_bias, self.softplus = A, D, dt_bias, bool(softplus)

    def _desc(self, x, dt, Bm, Cm):
        if not isinstance(x, torch.Tensor) or x.dim() != 4 or x.shape[2] != self.H:
            raise SDMError(1, f"x must be [B, T, {self.H}, P]")
        if not isinstance(Bm, torch.Tensor) or Bm.dim() != 4:
            raise SDMError(1, "Bm must be [B, T, G, N]")
        B, T, H, P = x.shape
        G, N = Bm.shape[2:]
        _view(x, "x", x, (B, T, H, P), 2)
        _view(Bm, "Bm", x, (B, T, G, N), 2)
        _view(Cm, "Cm", x, (B, T, G, N), 2)
        _out_tensor(dt, "dt", (B, T, H), x.dtype, x)
        _same_device(self.A, x, "A")
        return _ScanDesc(B, T, H, P, N, G, int(self.softplus), _dtype(x, "x"), x.stride(0),
                         x.stride(1), Bm.stride(0), Bm.stride(1), Cm.stride(0), Cm.stride(1))

    @staticmethod
    def _need(call, d) -> int:
        n = ctypes.c_size_t()
        _check(call(ctypes.byref(d), ctypes.byref(n)))
        return n.value

    def workspace_size(self, x, dt, Bm, Cm) -> int:
        """Bytes of workspace forward needs for inputs like these."""
        return self._need(lib().sdm_scan_workspace_size, self._desc(x, dt, Bm, Cm))

    def backward_workspace_size(self, x, dt, Bm, Cm) -> int:
        """Bytes of workspace backward needs for inputs like these."""
        return self._need(lib().sdm_scan_backward_workspace_size, self._desc(x, dt, Bm, Cm))

    def forward(self, x, dt, Bm, Cm, state=None, cont: bool = False, lengths=None, y=None,
                workspace=None):
        """(y, state): y [B, T, H, P] and the last state [B, H, P, N] (float32).

        x [B, T, H, P], dt [B, T, H], Bm and Cm [B, T, G, N].  With cont=True
        the scan starts from `state`, which is updated in place; otherwise from
        zero (a given `state` is overwritten).  lengths [B] int32: tokens of
        each sequence.
        """
        d = self._desc(x, dt, Bm, Cm)
        shape = (d.B, d.H, d.P, d.N)
        if state is None:
            if cont:
                raise SDMError(1, "cont=True needs the state")
            state = torch.empty(shape, dtype=_F32, device=x.device)
        else:
            _out_tensor(state, "state", shape, _F32, x)
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            _out_tensor(y, "y", x.shape, x.dtype, x)
        _lengths(lengths, d.B, x)
        workspace = _workspace(workspace, self._need(lib().sdm_scan_workspace_size, d), x)
        with _On(x.device) as stream:
            _check(lib().sdm_scan_forward(
                ctypes.byref(d), _p(x), _p(dt), _p(Bm), _p(Cm), _p(self.A), _p(self.D),
                _p(self.dt_bias), _p(lengths), FLAG_CONTINUE if cont else 0, _p(workspace),
                workspace.numel(), _p(y), _p(state), stream))
        return y, state

    def backward(self, x, dt, Bm, Cm, dy, state=None, dstate=None, lengths=None,
                 workspace=None) -> dict:
        """Gradients for dy [B, T, H, P] (and dstate, that of the final state,
        or None for zero): dx, ddt, dB, dC, float32 dA, dD and ddt_bias (where
        given), and, for a forward that started from `state`, dstate."""
        d = self._desc(x, dt, Bm, Cm)
        shape = (d.B, d.H, d.P, d.N)
        _out_tensor(dy, "dy", x.shape, x.dtype, x)
        for t, name in ((state, "state"), (dstate, "dstate")):
            if t is not None:
                _out_tensor(t, name, shape, _F32, x)
        _lengths(lengths, d.B, x)
        workspace = _workspace(workspace, self._need(lib().sdm_scan_backward_workspace_size, d), x)
        new = dict(dtype=x.dtype, device=x.device)
        out = dict(dx=torch.empty(x.shape, **new), ddt=torch.empty(dt.shape, **new),
                   dB=torch.empty(Bm.shape, **new), dC=torch.empty(Cm.shape, **new),
                   dA=torch.empty_like(self.A))
        if self.D is not None:
            out["dD"] = torch.empty_like(self.D)
        if self.dt_bias is not None:
            out["ddt_bias"] = torch.empty_like(self.dt_bias)
        if state is not None:
            out["dstate"] = torch.empty(shape, dtype=_F32, device=x.device)
        with _On(x.device) as stream:
            _check(lib().sdm_scan_backward(
                ctypes.byref(d), _p(x), _p(dt), _p(Bm), _p(Cm), _p(self.A), _p(self.D),
                _p(self.dt_bias), _p(lengths), _p(dy), _p(state), _p(dstate), _p(workspace),
                workspace.numel(), _p(out["dx"]), _p(out["ddt"]), _p(out["dB"]), _p(out["dC"]),
                _p(out["dA"]), _p(out.get("dD")), _p(out.get("ddt_bias")), _p(out.get("dstate")),
                stream))
        return out


class _WindowDesc(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int64), ("Hq", c_int), ("Hk", c_int), ("D", c_int),
                ("window", c_int64), ("sinks", c_int), ("scale", c_float), ("dtype", c_int)] + \
               [(f"{t}_{s}", c_int64) for t in "qkv" for s in ("batch", "token", "head")]


class WindowAttention:
    """Causal attention with a sliding window and sinks.

    The query at i sees the key at j where j <= i and (i - j < window or
    j < sinks).  Hq / Hk neighbouring query heads share a key head; scale
    defaults to 1 / sqrt(D).
    """

    def __init__(self, Hq: int, Hk: int, D: int, window: int, sinks: int = 0, scale=None):
        self.Hq, self.Hk, self.D = int(Hq), int(Hk), int(D)
        self.window, self.sinks = int(window), int(sinks)
        if self.D < 1 or self.window < 1 or self.sinks < 0 or max(
                self.D, self.window, self.sinks, abs(self.Hq), abs(self.Hk)) >= 1 << 31:
            raise SDMError(1, "D and window must be >= 1, sinks >= 0, and all below 2^31")
        self.scale = self.D ** -0.5 if scale is None else float(scale)

    def new_cache(self, B: int, dtype=_BF16, device="cuda"):
        """An empty rolling cache for B streams: (keys, values), each
        [B, sinks + window, Hk, D]."""
        shape = (B, self.sinks + self.window, self.Hk, self.D)
        return (torch.zeros(shape, dtype=dtype, device=device),
                torch.zeros(shape, dtype=dtype, device=device))

    def _desc(self, q, k, v):
        if not isinstance(q, torch.Tensor) or q.dim() != 4:
            raise SDMError(1, f"q must be [B, T, {self.Hq}, {self.D}]")
        B, T = q.shape[:2]
        _view(q, "q", q, (B, T, self.Hq, self.D), 1)
        _view(k, "k", q, (B, T, self.Hk, self.D), 1)
        _view(v, "v", q, (B, T, self.Hk, self.D), 1)
        return _WindowDesc(B, T, self.Hq, self.Hk, self.D, self.window, self.sinks, self.scale,
                           _dtype(q, "q"), *q.stride()[:3], *k.stride()[:3], *v.stride()[:3])

    def workspace_size(self, q, k, v, cont: bool = False) -> int:
        """Bytes of workspace forward needs for inputs like these."""
        n = ctypes.c_size_t()
        _check(lib().sdm_window_workspace_size(ctypes.byref(self._desc(q, k, v)),
                                               FLAG_CONTINUE if cont else 0, ctypes.byref(n)))
        return n.value

    def forward(self, q, k, v, cache=None, pos=None, cont: bool = False, lengths=None, o=None,
                lse=None, workspace=None):
        """(o, lse): o [B, T, Hq, D] and the log of the softmax's sum [B, T, Hq]
        (float32), for q [B, T, Hq, D] and k, v [B, T, Hk, D].

        cache: (keys, values) of new_cache, updated in place with the call's
        tokens.  With cont=True the tokens follow the pos[b] tokens that
        sequence b has in the cache (pos [B] int64, which the caller advances);
        otherwise they start a sequence.  lengths [B] int32: tokens of each
        sequence in this call.
        """
        d = self._desc(q, k, v)
        ck = cv = None
        if cache is not None:
            ck, cv = cache
            shape = (d.B, self.sinks + self.window, self.Hk, self.D)
            _out_tensor(ck, "the cache's keys", shape, q.dtype, q)
            _out_tensor(cv, "the cache's values", shape, q.dtype, q)
        if cont and (cache is None or pos is None):
            raise SDMError(1, "cont=True needs the cache and pos")
        if pos is not None:
            _out_tensor(pos, "pos", (d.B,), torch.int64, q)
        if o is None:
            o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        else:
            _out_tensor(o, "o", q.shape, q.dtype, q)
        if lse is None:
            lse = torch.empty(q.shape[:3], dtype=_F32, device=q.device)
        else:
            _out_tensor(lse, "lse", q.shape[:3], _F32, q)
        _lengths(lengths, d.B, q)
        flags = FLAG_CONTINUE if cont else 0
        n = ctypes.c_size_t()
        _check(lib().sdm_window_workspace_size(ctypes.byref(d), flags, ctypes.byref(n)))
        if n.value or workspace is not None:
            workspace = _workspace(workspace, n.value, q)
        with _On(q.device) as stream:
            _check(lib().sdm_window_forward(
                ctypes.byref(d), _p(q), _p(k), _p(v), _p(lengths), flags, _p(ck), _p(cv), _p(pos),
                _p(workspace), 0 if workspace is None else workspace.numel(), _p(o), _p(lse),
                stream))
        return o, lse

    def backward_workspace_size(self, q, k, v) -> int:
        """Bytes of workspace backward needs for inputs like these."""
        n = ctypes.c_size_t()
        _check(lib().sdm_window_backward_workspace_size(ctypes.byref(self._desc(q, k, v)),
                                                        ctypes.byref(n)))
        return n.value

    def backward(self, q, k, v, o, lse, do, lengths=None, workspace=None) -> dict:
        """Gradients dq, dk, dv for do [B, T, Hq, D], with the o and lse that a
        forward without a cache returned."""
        d = self._desc(q, k, v)
        _out_tensor(o, "o", q.shape, q.dtype, q)
        _out_tensor(do, "do", q.shape, q.dtype, q)
        _out_tensor(lse, "lse", q.shape[:3], _F32, q)
        _lengths(lengths, d.B, q)
        workspace = _workspace(workspace, self.backward_workspace_size(q, k, v), q)
        out = {n: torch.empty(t.shape, dtype=q.dtype, device=q.device)
               for n, t in (("dq", q), ("dk", k), ("dv", v))}
        with _On(q.device) as stream:
            _check(lib().sdm_window_backward(
                ctypes.byref(d), _p(q), _p(k), _p(v), _p(o), _p(lse), _p(do), _p(lengths),
                _p(workspace), workspace.numel(), _p(out["dq"]), _p(out["dk"]), _p(out["dv"]),
                stream))
        return out
