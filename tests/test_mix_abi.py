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


def scan_desc(**kw):
    d = dict(B=2, T=100, H=4, P=16, N=8, G=2, softplus=1, dtype=sdm.BF16, x_batch=6400, x_token=64,
             B_batch=1600, B_token=16, C_batch=1600, C_token=16)
    d.update(kw)
    return mixers._ScanDesc(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1), (dict(P=0), 1), (dict(N=0), 1), (dict(G=0), 1),
    (dict(G=3), 1), (dict(softplus=2), 1), (dict(dtype=2), 1), (dict(x_token=-1), 1),
    (dict(B_batch=-1), 1), (dict(C_token=-1), 1), (dict(N=129), 2), (dict(P=65537), 2),
    (dict(B=65536, H=1, G=1), 2), (dict(T=1 << 31), 2), (dict(T=1 << 30), 2),
])
def test_scan_descriptor_refusals(kw, status):
    L, n = sdm.lib(), ctypes.c_size_t()
    d = ctypes.byref(scan_desc(**kw))
    assert L.sdm_scan_workspace_size(d, ctypes.byref(n)) == status and n.value == 0
    assert L.sdm_scan_backward_workspace_size(d, ctypes.byref(n)) == status
    assert L.sdm_scan_forward(d, *[FAKE] * 8, 0, FAKE, 1 << 40, FAKE, FAKE, None) == status
    assert L.sdm_scan_backward(d, *[FAKE] * 12, 1 << 40, *[FAKE] * 8, None) == status
    assert L.sdm_last_error()


def test_scan_pointer_refusals():
    L, n = sdm.lib(), ctypes.c_size_t()
    d = ctypes.byref(scan_desc())
    assert L.sdm_scan_workspace_size(d, None) == 1
    assert L.sdm_scan_workspace_size(None, ctypes.byref(n)) == 1
    assert L.sdm_scan_workspace_size(d, ctypes.byref(n)) == 0 and n.value > 0
    # forward: x dt Bm Cm A D bias lengths | flags ws bytes | y state
    need = n.value

    def fwd(at=None, value=None, flags=0, ws=FAKE, size=need, y=FAKE, state=FAKE):
        p = [FAKE] * 8
        if at is not None:
            p[at] = value
        return L.sdm_scan_forward(d, *p, flags, ws, size, y, state, None)

    for at in (0, 1, 2, 3, 4):
        assert fwd(at, None) == 1, at
    for at in (0, 2, 3):
        assert fwd(at, FAKE + 1) == 1, at
    for at in (1, 4, 5, 6):
        assert fwd(at, FAKE + 4) == 1, at
    assert fwd(7, FAKE + 2) == 1
    assert fwd(flags=8) == 1 and fwd(ws=None) == 1 and fwd(ws=FAKE + 8) == 1
    assert fwd(size=need - 1) == 3 and fwd(y=None) == 1 and fwd(state=FAKE + 4) == 1
    assert L.sdm_scan_backward_workspace_size(d, ctypes.byref(n)) == 0 and n.value > need
    # backward: x dt Bm Cm A D bias lengths dy state dstateT ws | bytes | 8 outputs
    for at in (0, 1, 2, 3, 4, 8, 11):
        p = [FAKE] * 12
        p[at] = None
        assert L.sdm_scan_backward(d, *p, n.value, *[FAKE] * 8, None) == 1, at
    for at in range(5):  # dx ddt dB dC dA
        q = [FAKE] * 8
        q[at] = None
        assert L.sdm_scan_backward(d, *[FAKE] * 12, n.value, *q, None) == 1, at
    for at in range(8):
        q = [FAKE] * 8
        q[at] = FAKE + 4
        assert L.sdm_scan_backward(d, *[FAKE] * 12, n.value, *q, None) == 1, at
    assert L.sdm_scan_backward(d, *[FAKE] * 12, n.value - 1, *[FAKE] * 8, None) == 3


def window_desc(**kw):
    d = dict(B=2, T=100, Hq=4, Hk=2, D=16, window=8, sinks=2, scale=0.25, dtype=sdm.BF16,
             q_batch=6400, q_token=64, q_head=16, k_batch=3200, k_token=32, k_head=16, v_batch=3200,
             v_token=32, v_head=16)
    d.update(kw)
    return mixers._WindowDesc(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=0), 1), (dict(Hq=0), 1), (dict(Hk=0), 1), (dict(Hk=3), 1), (dict(D=0), 1),
    (dict(window=0), 1), (dict(sinks=-1), 1), (dict(scale=float("nan")), 1), (dict(dtype=2), 1),
    (dict(q_token=-1), 1), (dict(k_head=-1), 1), (dict(v_batch=-1), 1), (dict(D=257), 2),
    (dict(sinks=1025), 2), (dict(window=1 << 30), 2), (dict(T=1 << 31), 2),
    (dict(B=1 << 15, T=1 << 20), 2),
])
def test_window_descriptor_refusals(kw, status):
    L, n = sdm.lib(), ctypes.c_size_t()
    d = ctypes.byref(window_desc(**kw))
    assert L.sdm_window_workspace_size(d, 0, ctypes.byref(n)) == status and n.value == 0
    assert L.sdm_window_backward_workspace_size(d, ctypes.byref(n)) == status
    assert L.sdm_window_forward(d, *[FAKE] * 4, 1, *[FAKE] * 4, 1 << 40, FAKE, FAKE, None) == status
    assert L.sdm_window_backward(d, *[FAKE] * 8, 1 << 40, FAKE, FAKE, FAKE, None) == status
    assert L.sdm_last_error()


def test_window_pointer_refusals():
    L, n = sdm.lib(), ctypes.c_size_t()
    d = ctypes.byref(window_desc())
    assert L.sdm_window_workspace_size(None, 0, ctypes.byref(n)) == 1
    assert L.sdm_window_workspace_size(d, 0, None) == 1
    assert L.sdm_window_workspace_size(d, 4, ctypes.byref(n)) == 1

    def fwd(flags=1, **kw):
        p = dict(q=FAKE, k=FAKE, v=FAKE, lengths=None, ck=FAKE, cv=FAKE, pos=FAKE, ws=FAKE, o=FAKE,
                 lse=FAKE)
        p.update(kw)
        return L.sdm_window_forward(d, p["q"], p["k"], p["v"], p["lengths"], flags, p["ck"], p["cv"],
                                    p["pos"], p["ws"], 1 << 40, p["o"], p["lse"], None)

    for name in ("q", "k", "v", "ck", "cv", "pos", "o", "lse"):
        assert fwd(**{name: None}) == 1, name
    for name in ("q", "k", "v"):
        assert fwd(**{name: FAKE + 1}) == 1, name
    for name in ("ck", "cv", "o", "lse", "ws"):
        assert fwd(**{name: FAKE + 8}) == 1, name
    assert fwd(pos=FAKE + 4) == 1 and fwd(lengths=FAKE + 2) == 1
    assert fwd(flags=0) == 1                      # pos without the flag
    assert fwd(flags=0, pos=None, cv=None) == 1   # half a cache
    assert fwd(flags=2) == 1
    assert L.sdm_window_backward_workspace_size(d, ctypes.byref(n)) == 0 and n.value > 0
    for at in (0, 1, 2, 3, 4, 5, 7):
        p = [FAKE] * 8
        p[at] = None
        assert L.sdm_window_backward(d, *p, n.value, FAKE, FAKE, FAKE, None) == 1, at
    assert L.sdm_window_backward(d, *[FAKE] * 8, n.value - 1, FAKE, FAKE, FAKE, None) == 3
    for at in range(3):
        q = [FAKE] * 3
        q[at] = None
        assert L.sdm_window_backward(d, *[FAKE] * 8, n.value, *q, None) == 1, at
