"""The short causal convolution against its definition in 64 bits: forward,
continuation, single tokens, backward (against autograd of the definition and
against differences), padded batches, strided views, refusals."""
import pytest
import torch

import sparse_memory_linear_select_amd as sdm
from mix_util import DTYPES, check, gen, leaf, normal

pytestmark = pytest.mark.gpu


def definition(x, w, b, state, lens, silu):
    """(y, new state) in 64 bits; rows behind a sequence's length give zeros."""
    B, T, C = x.shape
    K = w.shape[1]
    ys, states = [], []
    for s in range(B):
        n = T if lens is None else max(0, min(T, int(lens[s])))
        before = torch.zeros(K - 1, C, dtype=torch.float64) if state is None else state[s]
        xe = torch.cat([before, x[s, :n]])
        z = sum(xe[k:k + n] * w[:, k] for k in range(K)) + (0 if b is None else b)
        y = z * torch.sigmoid(z) if silu else z
        ys.append(torch.cat([y, torch.zeros(T - n, C, dtype=torch.float64)]))
        states.append(xe[n:n + K - 1])
    return torch.stack(ys), torch.stack(states)


def case(seed, B, T, C, K, dtype, bias=True, lens=None, with_state=False):
    g, dt = gen(seed), DTYPES[dtype]
    x = normal(g, B, T, C, dtype=dt)
    w = normal(g, C, K, scale=K ** -0.5)
    b = normal(g, C, scale=0.3) if bias else None
    st = normal(g, B, K - 1, C, dtype=dt) if with_state else None
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    return x, w, b, st, ln


def cpu(t):
    return None if t is None else t.cpu().double()


# B, T, C, K, dtype, bias, silu, lengths, state before
SHAPES = [
    (2, 1, 8, 4, "bf16", True, True, None, False),          # one token
    (3, 2, 16, 4, "f32", True, True, [2, 0, 1], True),      # shorter than the taps, an empty row
    (2, 65, 24, 4, "bf16", True, True, None, True),         # one token past a workgroup's run
    (2, 131, 520, 4, "bf16", False, False, [131, 77], False),
    (1, 200, 33, 3, "bf16", True, True, None, True),        # odd channels: scalar accesses
    (2, 150, 30, 5, "f32", True, True, [150, 149], True),   # channels in pairs
    (1, 64, 4, 8, "f32", False, True, None, True),
    (5, 17, 12, 2, "bf16", True, False, [17, 3, 0, 16, 1], True),
    (1, 300, 36, 7, "bf16", True, True, None, False),
    (2, 40, 10, 6, "f32", True, True, None, True),
    (1024, 5, 8, 4, "bf16", True, True, None, False),       # many short sequences: long runs
]
IDS = [f"B{s[0]}-T{s[1]}-C{s[2]}-K{s[3]}-{s[4]}" for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape):
    B, T, C, K, dt, bias, silu, lens, with_state = shape
    x, w, b, st, ln = case(7 * T + C, B, T, C, K, dt, bias, lens, with_state)
    ref, rs = definition(cpu(x), cpu(w), cpu(b), cpu(st), lens, silu)
    mag, _ = definition(cpu(x).abs(), cpu(w).abs(), None if b is None else cpu(b).abs(),
                        None if st is None else cpu(st).abs(), lens, False)
    conv = sdm.CausalConv(w, b, silu=silu)
    got = None if st is None else st.clone()
    y, s = conv.forward(x, state=got, cont=st is not None, lengths=ln)
    assert y.dtype == x.dtype
    check(y, ref, mag, "y")
    assert torch.equal(s.cpu().double(), rs)  # rows of the input, moved
    if got is not None:
        assert s is got


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape):
    B, T, C, K, dt, bias, silu, lens, with_state = shape
    x, w, b, st, ln = case(11 * T + C, B, T, C, K, dt, bias, lens, with_state)
    g = gen(5)
    dy, ds = normal(g, B, T, C, dtype=x.dtype), normal(g, B, K - 1, C, dtype=x.dtype)
    lx, lw, lb, ls = leaf(x), leaf(w), leaf(b), leaf(st)
    ref, rs = definition(lx, lw, lb, ls, lens, silu)
    loss = (ref * cpu(dy)).sum() + (rs * cpu(ds)).sum()
    leaves = [t for t in (lx, lw, lb, ls) if t is not None]
    grads = dict(zip([i for i, t in enumerate((lx, lw, lb, ls)) if t is not None],
                     torch.autograd.grad(loss, leaves)))
    # magnitudes: |silu'| < 1.1, so the sums of absolute terms of the linear form
    ax, aw, asx = (t.detach().abs().requires_grad_(True) if t is not None else None for t in (lx, lw, ls))
    m, ms = definition(ax, aw, None, asx, lens, False)
    ml = (m * 1.1 * cpu(dy).abs()).sum() + (ms * cpu(ds).abs()).sum()
    mx, mw = torch.autograd.grad(ml, (ax, aw), retain_graph=True)
    out = sdm.CausalConv(w, b, silu=silu).backward(x, dy, state=st, dstate=ds, lengths=ln)
    # z carries errors of |w||x|, which silu' passes on: a few steps of a magnitude below 8
    check(out["dx"], grads[0], 8 * mx, "dx")
    n = B * T
    check(out["dweight"], grads[1], mw, "dweight", steps=64 + n ** 0.5)
    if b is not None:
        lim = 1.1 * cpu(dy).abs().sum((0, 1))
        check(out["dbias"], grads[2], lim, "dbias", steps=64 + n ** 0.5)
    if st is not None:
        mst = torch.autograd.grad(ml, asx)[0]
        check(out["dstate"], grads[3], 8 * mst, "dstate")


def test_gradient_against_differences():
    x, w, b, st, _ = case(3, 1, 9, 4, 3, "f32", True, None, True)
    dy = normal(gen(4), 1, 9, 4)
    conv = sdm.CausalConv(w, b)
    out = conv.backward(x, dy, state=st)
    cx, cw, cb, cs = cpu(x), cpu(w), cpu(b), cpu(st)

    def loss(x_, w_):
        return float((definition(x_, w_, cb, cs, None, True)[0] * cpu(dy)).sum())

    h = 1e-5  # central differences: truncation ~h^2, rounding ~1e-16 / h
    for (t, i) in ((0, 0), (4, 2), (8, 3)):
        e = torch.zeros_like(cx)
        e[0, t, i] = h
        d = (loss(cx + e, cw) - loss(cx - e, cw)) / (2 * h)
        assert abs(float(out["dx"][0, t, i]) - d) <= 1e-5 * (1 + abs(d))
    for (i, k) in ((0, 0), (2, 1), (3, 2)):
        e = torch.zeros_like(cw)
        e[i, k] = h
        d = (loss(cx, cw + e) - loss(cx, cw - e)) / (2 * h)
        assert abs(float(out["dweight"][i, k]) - d) <= 1e-5 * (1 + abs(d))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_split_calls_equal_one_call(dt):
    """A sequence in one call, in two uneven parts and token by token: the same bits."""
    x, w, b, _, _ = case(21, 2, 70, 40, 4, dt)
    conv = sdm.CausalConv(w, b)
    y, s = conv.forward(x)
    for cuts in ((0, 33, 70), tuple(range(71))):
        st, parts = None, []
        for a, e in zip(cuts, cuts[1:]):
            part, st = conv.forward(x[:, a:e], state=st, cont=a > 0)  # strided views
            parts.append(part)
        assert torch.equal(torch.cat(parts, 1), y) and torch.equal(st, s)


@pytest.mark.parametrize("off", [0, 1, 3, 8])
def test_views(off):
    """x as a slice of a wider tensor, at any channel offset; an expanded batch."""
    g = gen(off)
    wide = normal(g, 2, 50, 64, dtype=torch.bfloat16)
    w, b = normal(g, 24, 4, scale=0.5), normal(g, 24)
    x = wide[:, :, off:off + 24]
    conv = sdm.CausalConv(w, b)
    y, s = conv.forward(x)
    y2, s2 = conv.forward(x.contiguous())
    assert torch.equal(y, y2) and torch.equal(s, s2)
    one = x[:1].expand(3, -1, -1)
    assert torch.equal(conv.forward(one)[0], y[:1].expand(3, -1, -1))
    dy = normal(g, 2, 50, 24, dtype=torch.bfloat16)
    a, c = conv.backward(x, dy), conv.backward(x.contiguous(), dy)
    # other accesses, the same sums
    for k in a:
        assert torch.equal(a[k], c[k]), k


def test_rows_behind_the_length_are_not_read():
    x, w, b, st, ln = case(31, 3, 40, 16, 4, "bf16", True, [40, 13, 0], True)
    conv = sdm.CausalConv(w, b)
    y, s = conv.forward(x, state=st.clone(), cont=True, lengths=ln)
    dy = normal(gen(1), 3, 40, 16, dtype=x.dtype)
    g = conv.backward(x, dy, state=st, lengths=ln)
    bad, bdy = x.clone(), dy.clone()
    for b_, n in enumerate((40, 13, 0)):
        bad[b_, n:] = float("nan")
        bdy[b_, n:] = float("inf")
    y2, s2 = conv.forward(bad, state=st.clone(), cont=True, lengths=ln)
    g2 = conv.backward(bad, bdy, state=st, lengths=ln)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    assert all(torch.equal(g[k], g2[k]) for k in g)
    assert (y[1, 13:] == 0).all() and (g["dx"][1, 13:] == 0).all()
    # lengths outside [0, T] act as the nearest bound
    wild = torch.tensor([99, 13, -5], dtype=torch.int32).cuda()
    y3, _ = conv.forward(x, state=st.clone(), cont=True, lengths=wild)
    assert torch.equal(y3, y)


def test_deterministic_and_graph_replay():
    x, w, b, st, _ = case(41, 2, 200, 48, 4, "bf16", True, None, True)
    dy = normal(gen(2), 2, 200, 48, dtype=x.dtype)
    conv = sdm.CausalConv(w, b)
    g1, g2 = conv.backward(x, dy), conv.backward(x, dy)
    assert all(torch.equal(g1[k], g2[k]) for k in g1)
    y = torch.empty_like(x[:, :1])
    step = x[:, :1].clone()
    s = st.clone()
    conv.forward(step, state=s.clone(), cont=True, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        conv.forward(step, state=s, cont=True, y=y)
    ref = st.clone()
    s.copy_(st)
    for t in range(5):
        step.copy_(x[:, t:t + 1])
        graph.replay()
        torch.cuda.synchronize()
        want, _ = conv.forward(x[:, t:t + 1], state=ref, cont=True)
        assert torch.equal(y, want) and torch.equal(s, ref), t


def test_refusals():
    x, w, b, st, ln = case(51, 2, 8, 16, 4, "bf16", True, [8, 8], True)
    conv = sdm.CausalConv(w, b)
    for call in (
        lambda: conv.forward(x, cont=True),                             # no state
        lambda: conv.forward(x.half()),                                 # another type
        lambda: conv.forward(x.transpose(1, 2).contiguous().transpose(1, 2)),  # channels not dense
        lambda: conv.forward(x[..., :15]),                              # another width
        lambda: conv.forward(x, state=st.float()),
        lambda: conv.forward(x, state=st[:, :2]),
        lambda: conv.forward(x, lengths=ln.long()),
        lambda: conv.forward(x, lengths=ln[:1]),
        lambda: conv.forward(x.cpu()),
        lambda: conv.forward(x, y=torch.empty(2, 8, 16, device="cuda")),
        lambda: conv.forward(x[:, :0]),                                 # no token
        lambda: conv.backward(x, x.float()),
        lambda: conv.backward(x, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: sdm.CausalConv(w.bfloat16(), b),
        lambda: sdm.CausalConv(w, b[:4]),
        lambda: sdm.CausalConv(normal(gen(0), 16, 9)).forward(x),       # too many taps
        lambda: sdm.CausalConv(normal(gen(0), 16, 1)).forward(x),
    ):
        with pytest.raises(sdm.SDMError):
            call()
