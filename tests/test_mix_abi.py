"""The C calls of the sequence mixers without a GPU: every refusal comes
before the first HIP call."""
import ctypes

import pytest

import sparse_memory_linear_select_amd as sdm
from sparse_memory_linear_select_amd import mixers

FAKE = 0x100000  # 16-byte aligned, never dereferenced: the checks come first


def conv_desc(**kw):
    d = dict(B=2, T=8, C=16, K=4, silu=1, dtype=sdm.BF16, x_batch=128, x_token=16)
    d.update(kw)
    return mixers._ConvDesc(**d)


def conv_forward(desc, flags=0, **ptr):
    p = dict(x=FAKE, weight=FAKE, bias=None, lengths=None, y=FAKE, state=FAKE)
    p.update(ptr)
    return sdm.lib().sdm_conv_forward(ctypes.byref(desc) if desc else None, p["x"], p["weight"],
                                      p["bias"], p["lengths"], flags, p["y"], p["state"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=0), 1), (dict(C=0), 1), (dict(K=0), 1), (dict(silu=2), 1),
    (dict(dtype=2), 1), (dict(x_batch=-1), 1), (dict(x_token=-1), 1), (dict(K=1), 2), (dict(K=9), 2),
    (dict(B=1 << 20, T=1 << 30), 2), (dict(T=1 << 31), 2),
])
def test_conv_descriptor_refusals(kw, status):
    assert conv_forward(conv_desc(**kw)) == status
    n = ctypes.c_size_t()
    assert sdm.lib().sdm_conv_backward_workspace_size(ctypes.byref(conv_desc(**kw)),
                                                      ctypes.byref(n)) == status
    assert n.value == 0 and sdm.lib().sdm_last_error()


def test_conv_pointer_refusals():
    assert conv_forward(None) == 1
    assert conv_forward(conv_desc(), flags=2) == 1
    for name in ("x", "weight", "y", "state"):
        assert conv_forward(conv_desc(), **{name: None}) == 1, name
    for name in ("weight", "bias", "y", "state"):
        assert conv_forward(conv_desc(), **{name: FAKE + 4}) == 1, name
    assert conv_forward(conv_desc(), x=FAKE + 1) == 1
    assert conv_forward(conv_desc(dtype=sdm.F32), x=FAKE + 2) == 1
    assert conv_forward(conv_desc(), lengths=FAKE + 2) == 1


def test_conv_backward_refusals():
    L, n = sdm.lib(), ctypes.c_size_t()
    d = conv_desc()
    assert L.sdm_conv_backward_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value
    assert L.sdm_conv_backward_workspace_size(ctypes.byref(d), None) == 1

    def call(ws_bytes=n.value, **ptr):
        p = dict(x=FAKE, weight=FAKE, dy=FAKE, ws=FAKE, dx=FAKE, dweight=FAKE, bias=None, state=None,
                 dstateT=None, dbias=None, dstate=None)
        p.update(ptr)
        return L.sdm_conv_backward(ctypes.byref(d), p["x"], p["weight"], p["bias"], None, p["dy"],
                                   p["state"], p["dstateT"], p["ws"], ws_bytes, p["dx"],
                                   p["dweight"], p["dbias"], p["dstate"], None)

    assert call(ws_bytes=n.value - 1) == 3
    for name in ("x", "weight", "dy", "ws", "dx", "dweight"):
        assert call(**{name: None}) == 1, name
    for name in ("dy", "ws", "dx", "dweight", "bias", "state", "dstateT", "dbias", "dstate"):
        assert call(**{name: FAKE + 4}) == 1, name
