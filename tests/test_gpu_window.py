"""Sliding-window attention with sinks against its definition in 64 bits:
forward, rolling cache, single tokens, backward, padded batches, views,
refusals."""
import math

import pytest
import torch

import sparse_memory_linear_select_amd as sdm
from mix_util import DTYPES, check, gen, leaf, normal

pytestmark = pytest.mark.gpu


def cpu(t):
    return None if t is None else t.detach().cpu().double()


def definition(q, k, v, W, S, lens, scale):
    """(o, lse, weights) over whole sequences, in 64 bits; rows behind a length are zero."""
    B, T, Hq, D = q.shape
    r = Hq // k.shape[2]
    i, j = torch.arange(T)[:, None], torch.arange(T)[None]
    see = (j <= i) & ((i - j < W) | (j < S))
    on = torch.ones(B, T, dtype=torch.bool) if lens is None else \
        torch.arange(T)[None] < torch.tensor(lens)[:, None]
    kh, vh = k.repeat_interleave(r, 2), v.repeat_interleave(r, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, kh) * scale
    m = see[None, None] & on[:, None, :, None] & on[:, None, None, :]
    s = s.masked_fill(~m, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[..., None])
    o = torch.einsum("bhij,bjhd->bihd", p, vh)
    lse = torch.where(on[:, None], lse, 0.0).transpose(1, 2)
    return o, lse, p


def inputs(seed, B, T, Hq, Hk, D, dtype, lens):
    g, dt = gen(seed), DTYPES[dtype]
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    return (normal(g, B, T, Hq, D, dtype=dt), normal(g, B, T, Hk, D, dtype=dt),
            normal(g, B, T, Hk, D, dtype=dt), ln)


# B, T, Hq, Hk, D, window, sinks, dtype, lengths
SHAPES = [
    (2, 1, 2, 1, 32, 4, 2, "bf16", None),
    (1, 63, 2, 2, 64, 1, 0, "f32", None),              # each token sees itself alone
    (2, 65, 4, 2, 128, 16, 4, "bf16", [65, 30]),
    (2, 130, 4, 1, 40, 200, 3, "bf16", [130, 0]),      # window longer than the sequence
    (1, 257, 3, 3, 17, 33, 1, "f32", None),            # odd head columns
    (1, 300, 8, 2, 72, 100, 70, "bf16", [299]),        # sinks over a tile
    (3, 200, 2, 1, 256, 64, 5, "bf16", [200, 64, 1]),
    (1, 200, 2, 2, 130, 50, 2, "f32", None),
    (1, 1200, 2, 1, 64, 128, 4, "bf16", None),         # parts of the sinks' gradients
    (1, 150, 1, 1, 128, 1, 150, "f32", None),          # all tokens are sinks
    (1, 90, 6, 2, 8, 30, 100, "bf16", None),           # more sinks than tokens
    (1, 400, 8, 2, 64, 40, 6, "bf16", None),           # few sinks, two pairs of heads a key head
    (2, 300, 4, 1, 64, 30, 16, "f32", [300, 120]),     # as many as are summed apart
    (1, 300, 2, 2, 20, 50, 3, "bf16", None),           # scalar accesses
    (1, 260, 3, 1, 128, 60, 17, "bf16", [260]),        # one sink more
]
IDS = ["-".join(map(str, s[:8])) for s in SHAPES]


def mags(q, k, v, p, W, scale):
    """The magnitudes that scores are sums of, per query: errors of a score pass into weights."""
    r = q.shape[2] // k.shape[2]
    s = torch.einsum("bihd,bjhd->bhij", q.abs(), k.abs().repeat_interleave(r, 2)) * abs(scale)
    return s


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape):
    B, T, Hq, Hk, D, W, S, dt, lens = shape
    q, k, v, ln = inputs(7 * T + D, B, T, Hq, Hk, D, dt, lens)
    att = sdm.WindowAttention(Hq, Hk, D, W, S)
    o, lse = att.forward(q, k, v, lengths=ln)
    rq, rk, rv = cpu(q), cpu(k), cpu(v)
    ref, rl, p = definition(rq, rk, rv, W, S, lens, att.scale)
    # A score is off by D + 4 float32 half steps of its absolute sum sm; a weight
    # by that relative error, the exponent's few, and one rounding to bfloat16.
    sm = mags(rq, rk, rv, p, W, att.scale).masked_fill(p == 0, 0).amax(-1).transpose(1, 2)
    rel = (2 * (D + 4) * sm + T + 32) * 2.0 ** -24 + (0 if dt == "f32" else 2.0 ** -8)
    mag = torch.einsum("bhij,bjhd->bihd", p, rv.abs().repeat_interleave(Hq // Hk, 2))
    check(o, ref, mag * rel[..., None], "o", steps=0, weights=1.0)
    check(lse, rl, ((D + 4) * sm + T + 32) * 2.0 ** -24 + rl.abs() * 2.0 ** -22, "lse", steps=0, weights=1.0)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape):
    B, T, Hq, Hk, D, W, S, dt, lens = shape
    q, k, v, ln = inputs(11 * T + D, B, T, Hq, Hk, D, dt, lens)
    do = normal(gen(2), B, T, Hq, D, dtype=q.dtype)
    att = sdm.WindowAttention(Hq, Hk, D, W, S)
    o, lse = att.forward(q, k, v, lengths=ln)
    out = att.backward(q, k, v, o, lse, do, lengths=ln)
    lq, lk, lv = leaf(q), leaf(k), leaf(v)
    ro, _, p = definition(lq, lk, lv, W, S, lens, att.scale)
    ref = torch.autograd.grad((ro * cpu(do)).sum(), (lq, lk, lv))
    r = Hq // Hk
    aq, ak, av, ado = (cpu(t).abs() for t in (q, k, v, do))
    on = torch.ones(B, T) if lens is None else (torch.arange(T)[None] < torch.tensor(lens)[:, None])
    ado = ado * on.double()[..., None, None]
    p = p.detach()
    vr = av.repeat_interleave(r, 2)
    # ds = p (do.v - do.o) scale: the absolute terms, where o is what it was rounded to
    dp = torch.einsum("bihd,bjhd->bhij", ado, vr)
    oo = (ado * ro.detach().abs()).sum(-1).transpose(1, 2)[..., None]
    sm = (mags(aq, ak, av, p, W, att.scale) * (p > 0)).amax(-1, keepdim=True)
    one = 0 if dt == "f32" else 2.0 ** -8           # one rounding of o, and one of a weight
    rel = (2 * (D + 4) * sm + 2 * T + 64) * 2.0 ** -24
    ds = p * att.scale * ((dp + oo) * rel + oo * one)        # error of ds
    w = p * att.scale * (torch.einsum("bihd,bjhd->bhij", cpu(do), cpu(v).repeat_interleave(r, 2))
                         - (cpu(do) * ro.detach()).sum(-1).transpose(1, 2)[..., None]).abs() * one
    e = ds + w
    heads = lambda t: t.unflatten(2, (Hk, r)).sum(3)  # noqa: E731
    check(out["dq"], ref[0], torch.einsum("bhij,bjhd->bihd", e, ak.repeat_interleave(r, 2)), "dq", 0, 1.0)
    check(out["dk"], ref[1], heads(torch.einsum("bhij,bihd->bjhd", e, aq)), "dk", 0, 1.0)
    check(out["dv"], ref[2], heads(torch.einsum("bhij,bihd->bjhd", p * (rel + one), ado)), "dv", 0, 1.0)
    if lens is not None:
        for b, n in enumerate(lens):
            assert all((out[x][b, n:] == 0).all() for x in out)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_one_visible_key_has_no_score_gradient(dt):
    """A softmax over one key is 1: dq and dk are exactly zero, and dv is do."""
    for T, W, S in ((1, 5, 3), (150, 1, 0)):
        q, k, v, _ = inputs(T, 2, T, 4, 2, 64, dt, None)
        do = normal(gen(1), 2, T, 4, 64, dtype=q.dtype)
        att = sdm.WindowAttention(4, 2, 64, W, S)
        o, lse = att.forward(q, k, v)
        out = att.backward(q, k, v, o, lse, do)
        assert (out["dq"] == 0).all() and (out["dk"] == 0).all()
        both = do.float().unflatten(2, (2, 2)).sum(3)
        # the weight exp(s - lse) is off by the rounding of lse: |lse| 2^-22
        lim = (lse.abs().amax() + 1) * 2.0 ** -21 + torch.finfo(q.dtype).eps
        assert float(((out["dv"].float() - both).abs() / (1 + both.abs())).max()) <= float(lim)


@pytest.mark.parametrize("T,D,W,S", [(34, 64, 1235, 4), (300, 64, 2, 0), (300, 64, 3, 1), (300, 128, 8, 4),
                                     (300, 64, 40, 20), (500, 256, 20, 4)])
def test_few_visible_keys_lose_no_precision(T, D, W, S):
    """bfloat16 dq and dk carry two roundings, dS's for the products and their own, which
    add up in squares: sqrt(2) = 1.41 times the error of rounding the exact result (and
    dv, with its weights' rounding, too).  The rounding of o would be a third one, above 2
    times at two visible keys; 1.55 leaves 10% for the scatter of sums over 10^4 elements."""
    q, k, v, do = (normal(gen(11 + n), 2, T, h, D, dtype=torch.bfloat16) for n, h in enumerate((4, 2, 2, 4)))
    att = sdm.WindowAttention(4, 2, D, W, S)
    o, lse = att.forward(q, k, v)
    out = att.backward(q, k, v, o, lse, do)
    x = [leaf(cpu(t)) for t in (q, k, v)]
    (definition(*x, W, S, None, D ** -0.5)[0] * cpu(do)).sum().backward()
    for n, t in zip("qkv", x):
        one = (t.grad.bfloat16().double() - t.grad).norm()
        assert float((cpu(out["d" + n]) - t.grad).norm() / one) <= 1.55, n


def test_gradient_against_differences():
    q, k, v, _ = inputs(5, 1, 70, 2, 1, 8, "f32", None)
    do = normal(gen(6), 1, 70, 2, 8)
    att = sdm.WindowAttention(2, 1, 8, 20, 2, scale=0.7)
    o, lse = att.forward(q, k, v)
    out = att.backward(q, k, v, o, lse, do)
    c = dict(q=cpu(q), k=cpu(k), v=cpu(v))

    def loss(**kw):
        x = {**c, **kw}
        return float((definition(x["q"], x["k"], x["v"], 20, 2, None, 0.7)[0] * cpu(do)).sum())

    h = 1e-5
    for n, at in (("q", (0, 69, 1, 3)), ("k", (0, 0, 0, 0)), ("k", (0, 40, 0, 7)), ("v", (0, 1, 0, 5)),
                  ("v", (0, 69, 0, 2))):
        e = torch.zeros_like(c[n])
        e[at] = h
        d = (loss(**{n: c[n] + e}) - loss(**{n: c[n] - e})) / (2 * h)
        assert abs(float(out["d" + n][at]) - d) <= 1e-4 * (1 + abs(d)), (n, at)


@pytest.mark.parametrize("dt,Hq,Hk,D,W,S", [("bf16", 4, 2, 64, 24, 3), ("f32", 2, 2, 20, 70, 0),
                                            ("bf16", 8, 1, 128, 1, 5), ("bf16", 2, 1, 33, 9, 80)])
def test_stream_equals_whole_sequence(dt, Hq, Hk, D, W, S):
    """A prompt, parts of several lengths and single tokens through the rolling
    cache, sequences at different positions, against the whole sequence."""
    B, T = 2, 230
    q, k, v, _ = inputs(31, B, T, Hq, Hk, D, dt, None)
    att = sdm.WindowAttention(Hq, Hk, D, W, S)
    ref, rl, p = definition(cpu(q), cpu(k), cpu(v), W, S, None, att.scale)
    cache = att.new_cache(B, q.dtype)
    for c in cache:
        c.fill_(float("nan"))  # rows of tokens that have not come are not read
    at = [0, 0]
    got, gl = torch.zeros_like(ref), torch.zeros_like(rl)
    parts = [(70, 13)] + [(1, 1)] * 5 + [(0, 40), (30, 1), (1, 0)] + [(65, 66)] + [(1, 1)] * 20
    for n, ns in enumerate(parts):
        m = max(ns)
        sel = [torch.stack([t[b, at[b]:at[b] + m] if at[b] + m <= T else
                            torch.cat([t[b, at[b]:], t.new_full((m - T + at[b], *t.shape[2:]), math.nan)])
                            for b in range(B)]) for t in (q, k, v)]
        pos = torch.tensor(at, dtype=torch.int64).cuda()
        ln = torch.tensor(ns, dtype=torch.int32).cuda()
        o, lse = att.forward(*sel, cache=cache, pos=pos if n else None, cont=n > 0, lengths=ln)
        for b in range(B):
            got[b, at[b]:at[b] + ns[b]] = cpu(o[b, :ns[b]])
            gl[b, at[b]:at[b] + ns[b]] = cpu(lse[b, :ns[b]])
            assert (o[b, ns[b]:] == 0).all() and (lse[b, ns[b]:] == 0).all()
            at[b] += ns[b]
    sm = (mags(cpu(q), cpu(k), None, p, W, att.scale) * (p > 0)).amax(-1).transpose(1, 2)
    rel = (2 * (D + 4) * sm + T + 32) * 2.0 ** -24 + (0 if dt == "f32" else 2.0 ** -8)
    mag = torch.einsum("bhij,bjhd->bihd", p, cpu(v).abs().repeat_interleave(Hq // Hk, 2)) * rel[..., None]
    for b in range(B):
        n = at[b]
        check(got[b, :n].to(q.dtype), ref[b, :n], mag[b, :n], "o", 0, 1.0)
        check(gl[b, :n].float(), rl[b, :n], ((D + 4) * sm + T + 32)[b, :n] * 2.0 ** -24 +
              rl[b, :n].abs() * 2.0 ** -22, "lse", 0, 1.0)
        # the cache: the sinks and the last `window` tokens, bit for bit
        for t in list(range(min(S, n))) + list(range(max(S, n - W), n)):
            slot = t if t < S else S + (t - S) % W
            assert torch.equal(cache[0][b, slot], k[b, t]) and torch.equal(cache[1][b, slot], v[b, t])


# B, Hq, Hk, D, window, sinks, dtype, positions
STEPS = [
    (3, 2, 1, 64, 2000, 3, "bf16", [0, 700, 5000]),        # a cache shared among workgroups
    (2, 12, 1, 128, 300, 0, "bf16", [299, 300]),           # two groups of heads
    (2, 3, 3, 256, 70, 5, "f32", [74, 1000]),
    (1, 8, 2, 33, 1100, 80, "f32", [40000]),               # scalar accesses
    (2, 4, 1, 8, 1, 0, "bf16", [0, 9]),                    # the token sees itself alone
    (4, 5, 1, 96, 130, 4, "bf16", [0, 3, 133, 134]),
]


@pytest.mark.parametrize("case", STEPS, ids=["-".join(map(str, c[:7])) for c in STEPS])
def test_step(case):
    """One token against a rolling cache of any age; rows that no token has filled hold NaN."""
    B, Hq, Hk, D, W, S, dt, at = case
    q, k, v, _ = inputs(W + D, B, 1, Hq, Hk, D, dt, None)
    g = gen(9)
    R = S + W
    ck, cv = (normal(g, B, R, Hk, D, dtype=q.dtype) for _ in range(2))
    for b, p in enumerate(at):
        ck[b, p:], cv[b, p:] = math.nan, math.nan
    ek, ev = ck.clone(), cv.clone()
    att = sdm.WindowAttention(Hq, Hk, D, W, S)
    pos = torch.tensor(at, dtype=torch.int64).cuda()
    on = torch.tensor([1] * (B - 1) + [0 if B > 3 else 1], dtype=torch.int32).cuda()
    o, lse = att.forward(q, k, v, cache=(ck, cv), pos=pos, cont=True, lengths=on)
    r = Hq // Hk
    for b, p in enumerate(at):
        if on[b] == 0:
            assert (o[b] == 0).all() and (lse[b] == 0).all()
            continue
        slot = p if p < S else S + (p - S) % W
        ek[b, slot], ev[b, slot] = k[b, 0], v[b, 0]
        n = min(p + 1, R)
        kk = cpu(ek[b, :n]).repeat_interleave(r, 1)
        vv = cpu(ev[b, :n]).repeat_interleave(r, 1)
        s = torch.einsum("hd,nhd->hn", cpu(q[b, 0]), kk) * att.scale
        w = torch.softmax(s, -1)
        ref = torch.einsum("hn,nhd->hd", w, vv)
        sm = (torch.einsum("hd,nhd->hn", cpu(q[b, 0]).abs(), kk.abs()) * att.scale).amax(-1)
        rel = (2 * (D + 4) * sm + n + 32) * 2.0 ** -24   # float32 weights throughout
        check(o[b, 0], ref, torch.einsum("hn,nhd->hd", w, vv.abs()) * rel[:, None], "o", 0, 1.0)
        check(lse[b, 0], torch.logsumexp(s, -1), rel + s.abs().amax(-1) * 2.0 ** -22, "lse", 0, 1.0)
    # only the token's row changed
    assert torch.equal(ck.nan_to_num(7.0), ek.nan_to_num(7.0))
    assert torch.equal(cv.nan_to_num(7.0), ev.nan_to_num(7.0))


def test_far_position():
    """Positions beyond 32 bits: only their order and slots matter."""
    Hq, Hk, D, W, S = 2, 1, 64, 16, 2
    att = sdm.WindowAttention(Hq, Hk, D, W, S)
    q, k, v, _ = inputs(3, 1, 60, Hq, Hk, D, "f32", None)
    ref, _, _ = definition(cpu(q), cpu(k), cpu(v), W, S, None, att.scale)
    cache = att.new_cache(1, torch.float32)
    att.forward(q[:, :40], k[:, :40], v[:, :40], cache=cache)
    shift = W * (1 << 34)  # a multiple of the ring: the same slots
    for t in range(40, 60):
        pos = torch.tensor([t + shift], dtype=torch.int64).cuda()
        o, _ = att.forward(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], cache=cache, pos=pos, cont=True)
        assert float((cpu(o)[:, 0] - ref[:, t]).abs().max()) < 1e-4


@pytest.mark.parametrize("off", [0, 1, 8])
def test_views(off):
    """q, k, v as slices of one projection, and as [B, H, T, D] tensors: the same bits."""
    g = gen(off)
    wide = normal(g, 2, 100, off + 8 * 24, dtype=torch.bfloat16)[..., off:].unflatten(-1, (8, 24))
    q, k, v = wide[:, :, :4], wide[:, :, 4:6], wide[:, :, 6:]
    att = sdm.WindowAttention(4, 2, 24, 30, 2)
    dense = [t.contiguous() for t in (q, k, v)]
    heads = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    o, lse = att.forward(*dense)
    do = normal(g, 2, 100, 4, 24, dtype=torch.bfloat16)
    grads = att.backward(*dense, o, lse, do)
    for other in ((q, k, v), heads):
        o2, l2 = att.forward(*other)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
        g2 = att.backward(*other, o, lse, do)
        assert all(torch.equal(grads[n], g2[n]) for n in grads)


def test_rows_behind_the_length_are_not_read():
    lens = [150, 40, 0]
    q, k, v, ln = inputs(41, 3, 150, 2, 1, 64, "bf16", lens)
    do = normal(gen(1), 3, 150, 2, 64, dtype=q.dtype)
    att = sdm.WindowAttention(2, 1, 64, 60, 3)
    o, lse = att.forward(q, k, v, lengths=ln)
    g = att.backward(q, k, v, o, lse, do, lengths=ln)
    bad = [t.clone() for t in (q, k, v, do, o, lse)]
    for b, n in enumerate(lens):
        for t in bad:
            t[b, n:] = math.nan
    o2, l2 = att.forward(*bad[:3], lengths=ln)
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    g2 = att.backward(*bad[:3], bad[4], bad[5], bad[3], lengths=ln)
    assert all(torch.equal(g[n], g2[n]) for n in g)
    assert (o[1, 40:] == 0).all() and (lse[2] == 0).all()


def test_large_scores():
    """Scores far apart: the running maximum keeps every weight finite."""
    q, k, v, _ = inputs(8, 1, 200, 2, 2, 64, "f32", None)
    att = sdm.WindowAttention(2, 2, 64, 90, 2, scale=300.0)
    o, lse = att.forward(q, k, v)
    ref, rl, p = definition(cpu(q), cpu(k), cpu(v), 90, 2, None, 300.0)
    sm = (mags(cpu(q), cpu(k), None, p, 90, 300.0)).amax(-1).transpose(1, 2)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    check(lse, rl, (68 * sm + 232) * 2.0 ** -24 + rl.abs() * 2.0 ** -22, "lse", 0, 1.0)


def test_deterministic_and_graph_replay():
    q, k, v, _ = inputs(51, 2, 1200, 4, 2, 64, "bf16", None)
    do = normal(gen(2), 2, 1200, 4, 64, dtype=q.dtype)
    att = sdm.WindowAttention(4, 2, 64, 128, 4)
    o, lse = att.forward(q, k, v)
    g1, g2 = (att.backward(q, k, v, o, lse, do) for _ in range(2))
    assert all(torch.equal(g1[n], g2[n]) for n in g1)
    # a captured decode step: tokens and positions copied into static buffers
    cache, ref = att.new_cache(2), att.new_cache(2)
    for c in (cache, ref):
        att.forward(q[:, :300], k[:, :300], v[:, :300], cache=c)
    step = [t[:, :1].clone() for t in (q, k, v)]
    pos = torch.full((2,), 300, dtype=torch.int64, device="cuda")
    so, sl = torch.empty_like(step[0]), torch.empty(2, 1, 4, device="cuda")
    ws = torch.empty(max(16, att.workspace_size(*step, cont=True)), dtype=torch.uint8, device="cuda")
    scratch = tuple(c.clone() for c in cache)
    att.forward(*step, cache=scratch, pos=pos, cont=True, o=so, lse=sl, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att.forward(*step, cache=cache, pos=pos, cont=True, o=so, lse=sl, workspace=ws)
        pos += 1
    pos.fill_(300)
    for t in range(300, 306):
        for s, x in zip(step, (q, k, v)):
            s.copy_(x[:, t:t + 1])
        graph.replay()
        torch.cuda.synchronize()
        want, wl = att.forward(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], cache=ref,
                               pos=torch.full((2,), t, dtype=torch.int64, device="cuda"), cont=True)
        assert torch.equal(so, want) and torch.equal(sl, wl), t
        assert torch.equal(cache[0], ref[0]) and torch.equal(cache[1], ref[1]), t


def test_refusals():
    q, k, v, ln = inputs(61, 2, 8, 4, 2, 16, "bf16", [8, 8])
    att = sdm.WindowAttention(4, 2, 16, 8, 2)
    cache = att.new_cache(2)
    pos = torch.zeros(2, dtype=torch.int64, device="cuda")
    o, lse = att.forward(q, k, v)
    for call in (
        lambda: att.forward(q, k, v, cont=True),
        lambda: att.forward(q, k, v, cache=cache, cont=True),
        lambda: att.forward(q, k, v, cache=cache, pos=pos),
        lambda: att.forward(q, k, v, cache=cache, pos=pos.int(), cont=True),
        lambda: att.forward(q, k, v, cache=(cache[0], cache[1][:, :9])),
        lambda: att.forward(q, k, v, cache=tuple(c.float() for c in cache)),
        lambda: att.forward(q.half(), k.half(), v.half()),
        lambda: att.forward(q, k.float(), v),
        lambda: att.forward(q, k[:, :4], v),
        lambda: att.forward(q[..., ::2], k, v),
        lambda: att.forward(q, k, v, lengths=ln.long()),
        lambda: att.forward(q[:, :0], k[:, :0], v[:, :0]),
        lambda: att.forward(q.cpu(), k, v),
        lambda: att.forward(q, k, v, lse=lse.bfloat16()),
        lambda: att.backward(q, k, v, o, lse, q.float()),
        lambda: att.backward(q, k, v, o, lse[:1], q),
        lambda: att.backward(q, k, v, o, lse, q, workspace=torch.empty(4, dtype=torch.uint8, device="cuda")),
        lambda: sdm.WindowAttention(4, 2, 16, 0),
        lambda: sdm.WindowAttention(4, 2, 16, 8, -1),
        lambda: sdm.WindowAttention(4, 3, 16, 8).forward(q, k[:, :, :1].expand(-1, -1, 3, -1),
                                                         v[:, :, :1].expand(-1, -1, 3, -1)),
        lambda: sdm.WindowAttention(4, 2, 16, 8, scale=math.inf).forward(q, k, v),
        lambda: sdm.WindowAttention(4, 2, 16, 8, 1025).forward(q, k, v),
        lambda: sdm.WindowAttention(1, 1, 257, 8).forward(*(normal(gen(0), 1, 2, 1, 257),) * 3),
    ):
        with pytest.raises(sdm.SDMError):
            call()
