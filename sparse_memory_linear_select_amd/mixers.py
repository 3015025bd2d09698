"""Sequence mixers beside the SDM core: CausalConv, SelectiveScan, WindowAttention.

Bindings of the sdm_conv_*, sdm_scan_* and sdm_window_* calls of include/sdm.h.
Like SDM, each class borrows its parameters, runs on the current stream of its
inputs' device, raises SDMError for what the library refuses, and has no
fallback.  Inputs may be views with any batch and token strides; outputs are
new dense tensors unless given.
"""
from __future__ import annotations

import ctypes
from ctypes import byref, c_float, c_int, c_int64

import torch
from torch._C import _cuda_getCurrentRawStream, _cuda_getDevice

from . import (BF16, F32, FLAG_CONTINUE, SDMError, _check, _dev_tensor, _out_tensor, _same_device,
               _workspace, lib)

_F32, _BF16 = torch.float32, torch.bfloat16


def _p(t):
    return None if t is None else t.data_ptr()


def _call(f, device, *args):
    """f(*args, stream) with `device` current, on its current stream."""
    index = device.index
    if _cuda_getDevice() == index:
        status = f(*args, _cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = f(*args, _cuda_getCurrentRawStream(index))
    if status:
        _check(status)


def _dense(t, name, shape, dtype, ref):
    """t, which must be a dense tensor of this shape and dtype on ref's device."""
    try:
        if (t.shape == shape and t.dtype is dtype and t.device == ref.device
                and t.is_contiguous()):
            return t
    except AttributeError:
        pass
    return _out_tensor(t, name, shape, dtype, ref)  # names what is wrong


# Checked descriptors by a layer's settings and the shapes, strides and types of
# a call's inputs: a decode loop or training run repeats a few.
_plans = {}


def _keep(key, plan):
    if len(_plans) >= 256:
        _plans.clear()
    _plans[key] = plan
    return plan


def _key(settings, *tensors):
    try:
        return (settings, *[(t.shape, t.stride(), t.dtype, t.device) for t in tensors])
    except AttributeError:
        raise SDMError(1, "the inputs must be GPU tensors") from None


def _dtype(t, name):
    if t.dtype == _F32:
        return F32
    if t.dtype == _BF16:
        return BF16
    raise SDMError(1, f"{name} must be float32 or bfloat16, got {t.dtype}")


def _param(t, name, shape, device=None):
    """A float32 parameter: a dense GPU tensor of this shape."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is _F32 and t.shape == shape
            and t.is_contiguous() and (device is None or t.device == device)):
        return t
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


def _strides(t, n):
    """The first n strides, 0 for dimensions of one element (where they say nothing)."""
    return [s if m > 1 else 0 for s, m in zip(t.stride()[:n], t.shape)]


def _lengths(t, B, like):
    return None if t is None else _dense(t, "lengths", (B,), torch.int32, like).data_ptr()


def _bytes(call, *args) -> int:
    n = ctypes.c_size_t()
    _check(call(*args, byref(n)))
    return n.value


class _Plan:
    """A checked descriptor and the workspaces it asks for."""

    def __init__(self, desc, shape):
        self.desc, self.ref, self.shape, self.ws = desc, byref(desc), shape, {}

    def workspace(self, call, given, like, *args):
        """(tensor or None, its bytes) for a call that asks `call` for the size."""
        key = (call.__name__, args)
        need = self.ws.get(key)
        if need is None:
            need = self.ws[key] = _bytes(call, self.ref, *args)
        if given is None and need == 0:
            return None, 0
        ws = _workspace(given, need, like)
        return ws, ws.numel()


class _ConvDesc(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int64), ("C", c_int), ("K", c_int), ("silu", c_int),
                ("dtype", c_int), ("x_batch", c_int64), ("x_token", c_int64)]


class CausalConv:
    """Short causal depthwise convolution, y = silu(bias + sum_k w[:, k] x[t - K + 1 + k]).

    weight [C, K] and bias [C] (or None) are float32 GPU tensors, borrowed.
    """

    def __init__(self, weight, bias=None, silu: bool = True):
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
            raise SDMError(1, "weight must be [C, K]")
        self.C, self.K = _param(weight, "weight", weight.shape).shape
        if bias is not None:
            _param(bias, "bias", (self.C,), weight.device)
        self.weight, self.bias, self.silu = weight, bias, bool(silu)
        self._settings = ("conv", self.C, self.K, self.silu, weight.device)

    def _plan(self, x):
        key = _key(self._settings, x)
        plan = _plans.get(key)
        if plan is not None:
            return plan
        if x.dim() != 3:
            raise SDMError(1, f"x must be [B, T, {self.C}]")
        B, T = x.shape[:2]
        _view(x, "x", x, (B, T, self.C), 1)
        _same_device(self.weight, x, "weight")
        d = _ConvDesc(B, T, self.C, self.K, int(self.silu), _dtype(x, "x"), *_strides(x, 2))
        return _keep(key, _Plan(d, (B, self.K - 1, self.C)))

    def forward(self, x, state=None, cont: bool = False, lengths=None, y=None):
        """(y, state): y [B, T, C], and the last K - 1 rows [B, K - 1, C].

        With cont=True `state` holds the rows before x and is updated in
        place; otherwise the rows before x are zeros (a given `state` is
        overwritten).  lengths [B] int32: tokens of each sequence.
        """
        plan = self._plan(x)
        if state is not None:
            _dense(state, "state", plan.shape, x.dtype, x)
        elif cont:
            raise SDMError(1, "cont=True needs the state")
        else:
            state = x.new_empty(plan.shape)
        y = x.new_empty(x.shape) if y is None else _dense(y, "y", x.shape, x.dtype, x)
        _call(lib().sdm_conv_forward, x.device, plan.ref, x.data_ptr(), self.weight.data_ptr(),
              _p(self.bias), _lengths(lengths, plan.desc.B, x), FLAG_CONTINUE if cont else 0,
              y.data_ptr(), state.data_ptr())
        return y, state

    def backward_workspace_size(self, x) -> int:
        """Bytes of workspace backward needs for inputs like x."""
        return _bytes(lib().sdm_conv_backward_workspace_size, self._plan(x).ref)

    def backward(self, x, dy, state=None, dstate=None, lengths=None, workspace=None) -> dict:
        """Gradients for dy [B, T, C] (and dstate, that of the final state, or
        None for zero): dx, float32 dweight and (with a bias) dbias, and, for a
        forward that started from `state`, dstate, its gradient."""
        plan = self._plan(x)
        _dense(dy, "dy", x.shape, x.dtype, x)
        for t, name in ((state, "state"), (dstate, "dstate")):
            if t is not None:
                _dense(t, name, plan.shape, x.dtype, x)
        ws, ws_bytes = plan.workspace(lib().sdm_conv_backward_workspace_size, workspace, x)
        out = dict(dx=x.new_empty(x.shape), dweight=torch.empty_like(self.weight))
        if self.bias is not None:
            out["dbias"] = torch.empty_like(self.bias)
        if state is not None:
            out["dstate"] = x.new_empty(plan.shape)
        _call(lib().sdm_conv_backward, x.device, plan.ref, _p(x), _p(self.weight), _p(self.bias),
              _lengths(lengths, plan.desc.B, x), _p(dy), _p(state), _p(dstate), _p(ws), ws_bytes,
              _p(out["dx"]), _p(out["dweight"]), _p(out.get("dbias")), _p(out.get("dstate")))
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
        if not isinstance(A, torch.Tensor) or A.dim() != 1:
            raise SDMError(1, "A must be [H]")
        self.H = _param(A, "A", A.shape).shape[0]
        for t, name in ((D, "D"), (dt_bias, "dt_bias")):
            if t is not None:
                _param(t, name, (self.H,), A.device)
        self.A, self.D, self.dt_bias, self.softplus = A, D, dt_bias, bool(softplus)
        self._settings = ("scan", self.H, self.softplus, A.device)

    def _plan(self, x, dt, Bm, Cm):
        key = _key(self._settings, x, dt, Bm, Cm)
        plan = _plans.get(key)
        if plan is not None:
            return plan
        if x.dim() != 4 or x.shape[2] != self.H:
            raise SDMError(1, f"x must be [B, T, {self.H}, P]")
        if Bm.dim() != 4:
            raise SDMError(1, "Bm must be [B, T, G, N]")
        B, T, H, P = x.shape
        G, N = Bm.shape[2:]
        _view(x, "x", x, (B, T, H, P), 2)
        _view(Bm, "Bm", x, (B, T, G, N), 2)
        _view(Cm, "Cm", x, (B, T, G, N), 2)
        _out_tensor(dt, "dt", (B, T, H), x.dtype, x)
        _same_device(self.A, x, "A")
        d = _ScanDesc(B, T, H, P, N, G, int(self.softplus), _dtype(x, "x"), *_strides(x, 2),
                      *_strides(Bm, 2), *_strides(Cm, 2))
        return _keep(key, _Plan(d, (B, H, P, N)))

    def workspace_size(self, x, dt, Bm, Cm) -> int:
        """Bytes of workspace forward needs for inputs like these."""
        return _bytes(lib().sdm_scan_workspace_size, self._plan(x, dt, Bm, Cm).ref)

    def backward_workspace_size(self, x, dt, Bm, Cm) -> int:
        """Bytes of workspace backward needs for inputs like these."""
        return _bytes(lib().sdm_scan_backward_workspace_size, self._plan(x, dt, Bm, Cm).ref)

    def forward(self, x, dt, Bm, Cm, state=None, cont: bool = False, lengths=None, y=None,
                workspace=None):
        """(y, state): y [B, T, H, P] and the last state [B, H, P, N] (float32).

        x [B, T, H, P], dt [B, T, H], Bm and Cm [B, T, G, N].  With cont=True
        the scan starts from `state`, which is updated in place; otherwise from
        zero (a given `state` is overwritten).  lengths [B] int32: tokens of
        each sequence.
        """
        plan = self._plan(x, dt, Bm, Cm)
        if state is not None:
            _dense(state, "state", plan.shape, _F32, x)
        elif cont:
            raise SDMError(1, "cont=True needs the state")
        else:
            state = x.new_empty(plan.shape, dtype=_F32)
        y = x.new_empty(x.shape) if y is None else _dense(y, "y", x.shape, x.dtype, x)
        ws, ws_bytes = plan.workspace(lib().sdm_scan_workspace_size, workspace, x)
        _call(lib().sdm_scan_forward, x.device, plan.ref, x.data_ptr(), dt.data_ptr(),
              Bm.data_ptr(), Cm.data_ptr(), self.A.data_ptr(), _p(self.D), _p(self.dt_bias),
              _lengths(lengths, plan.desc.B, x), FLAG_CONTINUE if cont else 0, _p(ws), ws_bytes,
              y.data_ptr(), state.data_ptr())
        return y, state

    def backward(self, x, dt, Bm, Cm, dy, state=None, dstate=None, lengths=None,
                 workspace=None) -> dict:
        """Gradients for dy [B, T, H, P] (and dstate, that of the final state,
        or None for zero): dx, ddt, dB, dC, float32 dA, dD and ddt_bias (where
        given), and, for a forward that started from `state`, dstate."""
        plan = self._plan(x, dt, Bm, Cm)
        _dense(dy, "dy", x.shape, x.dtype, x)
        for t, name in ((state, "state"), (dstate, "dstate")):
            if t is not None:
                _dense(t, name, plan.shape, _F32, x)
        ws, ws_bytes = plan.workspace(lib().sdm_scan_backward_workspace_size, workspace, x)
        out = dict(dx=x.new_empty(x.shape), ddt=x.new_empty(dt.shape), dB=x.new_empty(Bm.shape),
                   dC=x.new_empty(Cm.shape), dA=torch.empty_like(self.A))
        if self.D is not None:
            out["dD"] = torch.empty_like(self.D)
        if self.dt_bias is not None:
            out["ddt_bias"] = torch.empty_like(self.dt_bias)
        if state is not None:
            out["dstate"] = x.new_empty(plan.shape, dtype=_F32)
        _call(lib().sdm_scan_backward, x.device, plan.ref, _p(x), _p(dt), _p(Bm), _p(Cm),
              _p(self.A), _p(self.D), _p(self.dt_bias), _lengths(lengths, plan.desc.B, x), _p(dy),
              _p(state), _p(dstate), _p(ws), ws_bytes, _p(out["dx"]), _p(out["ddt"]),
              _p(out["dB"]), _p(out["dC"]), _p(out["dA"]), _p(out.get("dD")),
              _p(out.get("ddt_bias")), _p(out.get("dstate")))
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
        self._settings = ("window", self.Hq, self.Hk, self.D, self.window, self.sinks, self.scale)

    def new_cache(self, B: int, dtype=_BF16, device="cuda"):
        """An empty rolling cache for B streams: (keys, values), each
        [B, sinks + window, Hk, D]."""
        shape = (B, self.sinks + self.window, self.Hk, self.D)
        return (torch.zeros(shape, dtype=dtype, device=device),
                torch.zeros(shape, dtype=dtype, device=device))

    def _plan(self, q, k, v):
        key = _key(self._settings, q, k, v)
        plan = _plans.get(key)
        if plan is not None:
            return plan
        if q.dim() != 4:
            raise SDMError(1, f"q must be [B, T, {self.Hq}, {self.D}]")
        B, T = q.shape[:2]
        _view(q, "q", q, (B, T, self.Hq, self.D), 1)
        _view(k, "k", q, (B, T, self.Hk, self.D), 1)
        _view(v, "v", q, (B, T, self.Hk, self.D), 1)
        d = _WindowDesc(B, T, self.Hq, self.Hk, self.D, self.window, self.sinks, self.scale,
                        _dtype(q, "q"), *_strides(q, 3), *_strides(k, 3), *_strides(v, 3))
        return _keep(key, _Plan(d, (B, self.sinks + self.window, self.Hk, self.D)))

    def workspace_size(self, q, k, v, cont: bool = False) -> int:
        """Bytes of workspace forward needs for inputs like these."""
        return _bytes(lib().sdm_window_workspace_size, self._plan(q, k, v).ref,
                      FLAG_CONTINUE if cont else 0)

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
        plan = self._plan(q, k, v)
        ck = cv = None
        if cache is not None:
            ck, cv = cache
            _dense(ck, "the cache's keys", plan.shape, q.dtype, q)
            _dense(cv, "the cache's values", plan.shape, q.dtype, q)
        if cont and (cache is None or pos is None):
            raise SDMError(1, "cont=True needs the cache and pos")
        if pos is not None:
            _dense(pos, "pos", (plan.desc.B,), torch.int64, q)
        o = q.new_empty(q.shape) if o is None else _dense(o, "o", q.shape, q.dtype, q)
        rows = q.shape[:3]
        lse = q.new_empty(rows, dtype=_F32) if lse is None else _dense(lse, "lse", rows, _F32, q)
        flags = FLAG_CONTINUE if cont else 0
        ws, ws_bytes = plan.workspace(lib().sdm_window_workspace_size, workspace, q, flags)
        _call(lib().sdm_window_forward, q.device, plan.ref, q.data_ptr(), k.data_ptr(),
              v.data_ptr(), _lengths(lengths, plan.desc.B, q), flags, _p(ck), _p(cv), _p(pos),
              _p(ws), ws_bytes, o.data_ptr(), lse.data_ptr())
        return o, lse

    def backward_workspace_size(self, q, k, v) -> int:
        """Bytes of workspace backward needs for inputs like these."""
        return _bytes(lib().sdm_window_backward_workspace_size, self._plan(q, k, v).ref)

    def backward(self, q, k, v, o, lse, do, lengths=None, workspace=None) -> dict:
        """Gradients dq, dk, dv for do [B, T, Hq, D], with the o and lse that a
        forward without a cache returned."""
        plan = self._plan(q, k, v)
        _dense(o, "o", q.shape, q.dtype, q)
        _dense(do, "do", q.shape, q.dtype, q)
        _dense(lse, "lse", q.shape[:3], _F32, q)
        ws, ws_bytes = plan.workspace(lib().sdm_window_backward_workspace_size, workspace, q)
        out = dict(dq=q.new_empty(q.shape), dk=k.new_empty(k.shape), dv=v.new_empty(v.shape))
        _call(lib().sdm_window_backward, q.device, plan.ref, _p(q), _p(k), _p(v), _p(o), _p(lse),
              _p(do), _lengths(lengths, plan.desc.B, q), _p(ws), ws_bytes, _p(out["dq"]),
              _p(out["dk"]), _p(out["dv"]))
        return out
