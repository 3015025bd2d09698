"""The selective scan against its definition in 64 bits (token by token):
forward, continuation, single tokens, backward, padded batches, views, split
calls, refusals."""
import math

import pytest
import torch

import sparse_memory_linear_select_amd as sdm
from mix_util import DTYPES, check, gen, leaf, normal

pytestmark = pytest.mark.gpu


def cpu(t):
    return None if t is None else t.detach().cpu().double()


def recurrence(x, delta, logs, Bm, Cm, D, S0, lens):
    """(y, last state) from D_t and log a_t, token by token."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    Bh, Ch = Bm.repeat_interleave(H // G, 2), Cm.repeat_interleave(H // G, 2)
    S = torch.zeros(B, H, P, N, dtype=torch.float64) if S0 is None else S0
    on = torch.ones(B, T, dtype=torch.float64)
    if lens is not None:
        on = (torch.arange(T)[None] < torch.tensor(lens)[:, None]).double()
    ys = []
    for t in range(T):
        new = torch.exp(logs[:, t])[..., None, None] * S + \
            (delta[:, t, :, None] * x[:, t])[..., None] * Bh[:, t, :, None]
        m = on[:, t, None, None, None]
        S = m * new + (1 - m) * S
        y = (S * Ch[:, t, :, None]).sum(-1)
        if D is not None:
            y = y + D[:, None] * x[:, t]
        ys.append(y * on[:, t, None, None])
    return torch.stack(ys, 1), S


def inputs(seed, B, T, H, P, N, G, dtype, opts, lens, with_state):
    g, dt = gen(seed), DTYPES[dtype]
    d = dict(x=normal(g, B, T, H, P, dtype=dt), dt=normal(g, B, T, H, dtype=dt, shift=-2.0),
             Bm=normal(g, B, T, G, N, dtype=dt), Cm=normal(g, B, T, G, N, dtype=dt),
             A=-(0.2 + 8 * torch.rand(H, generator=g)).cuda(),
             D=normal(g, H) if "D" in opts else None,
             bias=normal(g, H, scale=0.3) if "b" in opts else None)
    if "s" not in opts:
        d["dt"] = d["dt"].abs()  # softplus off: steps as given
    if "z" in opts:
        d["A"].zero_()  # nothing is forgotten
    if "h" in opts:
        d["A"] *= 300.0  # hardly anything is kept
    d["S0"] = normal(g, B, H, P, N, scale=0.5) if with_state else None
    d["lengths"] = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    d["scan"] = sdm.SelectiveScan(d["A"], d["D"], d["bias"], softplus="s" in opts)
    return d


def steps_of(d, dt, bias, soft):
    z = dt if bias is None else dt + bias
    return torch.nn.functional.softplus(z, threshold=40) if soft else z


# B, T, H, P, N, G, dtype, options (s softplus, b bias, D skip, z A = 0, h A large), lengths, state before
SHAPES = [
    (1, 1, 2, 8, 4, 1, "f32", "sbD", None, True),              # one token
    (2, 1, 4, 64, 64, 2, "bf16", "sbD", [1, 0], True),         # an inactive sequence
    (2, 5, 2, 17, 3, 1, "f32", "s", [5, 0], True),             # odd sizes, an empty sequence
    (1, 64, 2, 64, 128, 2, "bf16", "sbD", None, False),        # one full chunk
    (1, 65, 3, 64, 128, 1, "bf16", "sbD", None, True),         # one token into the next
    (2, 130, 4, 40, 33, 2, "f32", "sbD", [130, 63], True),
    (2, 200, 4, 130, 20, 4, "bf16", "bD", [199, 128], False),  # three slices of columns
    (1, 1100, 2, 16, 64, 1, "f32", "sbD", None, True),         # segments of the time axis
    (2, 1200, 1, 70, 16, 1, "bf16", "sD", [1200, 700], True),
    (1, 150, 2, 32, 32, 1, "f32", "sbDz", None, True),
    (1, 150, 2, 32, 32, 1, "f32", "sbDh", None, True),
    (1, 90, 6, 24, 100, 3, "bf16", "sbD", None, True),
]
IDS = ["-".join(map(str, s[:8])) for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape):
    B, T, H, P, N, G, dt, opts, lens, with_state = shape
    d = inputs(13 * T + P, *shape)
    x, Bm, Cm, A, D, S0 = (cpu(d[k]) for k in ("x", "Bm", "Cm", "A", "D", "S0"))
    delta = steps_of(d, cpu(d["dt"]), cpu(d["bias"]), "s" in opts)
    ref, rs = recurrence(x, delta, delta * A, Bm, Cm, D, S0, lens)
    mag, ms = recurrence(x.abs(), delta, delta * A, Bm.abs(), Cm.abs(), None if D is None else D.abs(),
                         None if S0 is None else S0.abs(), lens)
    st = None if S0 is None else d["S0"].clone()
    y, s = d["scan"].forward(d["x"], d["dt"], d["Bm"], d["Cm"], state=st, cont=st is not None,
                             lengths=d["lengths"])
    # T terms a sum, plus the exponents and weights; bfloat16 rounds the decayed
    # scores and the state that y is made of to bfloat16 once
    n = 64 + T
    check(y, ref, mag, "y", steps=n, weights=0.0 if dt == "f32" else 2.0 ** -8)
    check(s, rs, ms, "state", steps=n)
    if st is not None:
        assert s is st


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape):
    B, T, H, P, N, G, dt, opts, lens, with_state = shape
    d = inputs(17 * T + P, *shape)
    g = gen(3)
    dy = normal(g, B, T, H, P, dtype=DTYPES[dt])
    dS = normal(g, B, H, P, N, scale=0.5)
    soft = "s" in opts
    L = {k: leaf(d[k]) for k in ("x", "dt", "Bm", "Cm", "A", "D", "bias", "S0")}
    delta = steps_of(d, L["dt"], L["bias"], soft)
    y, s = recurrence(L["x"], delta, delta * L["A"], L["Bm"], L["Cm"], L["D"], L["S0"], lens)
    loss = (y * cpu(dy)).sum() + (s * cpu(dS)).sum()
    names = [k for k in L if L[k] is not None]
    ref = dict(zip(names, torch.autograd.grad(loss, [L[k] for k in names])))
    # magnitudes: the same sums of absolute terms, with D_t and log a_t apart
    M = {k: None if d[k] is None else cpu(d[k]).abs().requires_grad_(True)
         for k in ("x", "Bm", "Cm", "D", "S0")}
    md = steps_of(d, cpu(d["dt"]), cpu(d["bias"]), soft).abs().requires_grad_(True)
    ml = (md.detach() * cpu(d["A"])).requires_grad_(True)
    y, s = recurrence(M["x"], md, ml, M["Bm"], M["Cm"], M["D"], M["S0"], lens)
    mloss = (y * cpu(dy).abs()).sum() + (s * cpu(dS).abs()).sum()
    mn = [k for k in M if M[k] is not None]
    mag = dict(zip(mn + ["d", "l"], torch.autograd.grad(mloss, [M[k] for k in mn] + [md, ml])))
    slope = 1 - torch.exp(-md.detach()) if soft else 1.0
    mag["dt"] = (mag["d"] + cpu(d["A"]).abs() * mag["l"]) * slope
    out = d["scan"].backward(d["x"], d["dt"], d["Bm"], d["Cm"], dy, state=d["S0"], dstate=dS,
                             lengths=d["lengths"])
    n, w = 64 + 2 * T, 0.0 if dt == "f32" else 2.0 ** -8
    check(out["dx"], ref["x"], mag["x"], "dx", steps=n, weights=w)
    check(out["dB"], ref["Bm"], mag["Bm"], "dB", steps=n, weights=w)
    check(out["dC"], ref["Cm"], mag["Cm"], "dC", steps=n, weights=w)
    check(out["ddt"], ref["dt"], mag["dt"], "ddt", steps=n)
    check(out["dA"], ref["A"], (mag["l"] * md.detach()).sum((0, 1)), "dA", steps=n)
    if d["D"] is not None:
        check(out["dD"], ref["D"], mag["D"], "dD", steps=n)
    if d["bias"] is not None:
        check(out["ddt_bias"], ref["bias"], mag["dt"].sum((0, 1)), "ddt_bias", steps=n)
    if d["S0"] is not None:
        check(out["dstate"], ref["S0"], mag["S0"], "dstate", steps=n)
    if lens is not None:
        for b, k in enumerate(lens):
            assert all((out[o][b, k:] == 0).all() for o in ("dx", "ddt", "dB", "dC"))


def test_gradient_against_differences():
    d = inputs(5, 1, 70, 2, 5, 4, 1, "f32", "sbD", None, True)
    dy = normal(gen(6), 1, 70, 2, 5)
    out = d["scan"].backward(d["x"], d["dt"], d["Bm"], d["Cm"], dy, state=d["S0"])
    c = {k: cpu(d[k]) for k in ("x", "dt", "Bm", "Cm", "A", "D", "bias", "S0")}

    def loss(**kw):
        v = {**c, **kw}
        delta = steps_of(d, v["dt"], v["bias"], True)
        y, _ = recurrence(v["x"], delta, delta * v["A"], v["Bm"], v["Cm"], v["D"], v["S0"], None)
        return float((y * cpu(dy)).sum())

    h = 1e-5  # central differences in 64 bits: truncation ~h^2
    for name, key, at in (("dt", "ddt", (0, 0, 1)), ("dt", "ddt", (0, 66, 0)), ("x", "dx", (0, 63, 1, 2)),
                          ("Bm", "dB", (0, 10, 0, 3)), ("Cm", "dC", (0, 69, 0, 0)), ("A", "dA", (1,)),
                          ("bias", "ddt_bias", (0,)), ("S0", "dstate", (0, 1, 4, 2))):
        e = torch.zeros_like(c[name])
        e[at] = h
        diff = (loss(**{name: c[name] + e}) - loss(**{name: c[name] - e})) / (2 * h)
        assert abs(float(out[key][at]) - diff) <= 1e-4 * (1 + abs(diff)), (name, at)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_prompt_then_tokens(dt):
    """A prompt, then single tokens that continue its state, against one long call."""
    B, T, H, P, N, G = 2, 150, 4, 64, 64, 1
    d = inputs(31, B, T, H, P, N, G, dt, "sbD", None, False)
    x, Bm, Cm, A, D = (cpu(d[k]) for k in ("x", "Bm", "Cm", "A", "D"))
    delta = steps_of(d, cpu(d["dt"]), cpu(d["bias"]), True)
    ref, rs = recurrence(x, delta, delta * A, Bm, Cm, D, None, None)
    mag, ms = recurrence(x.abs(), delta, delta * A, Bm.abs(), Cm.abs(), D.abs(), None, None)
    parts, st = [], None
    cuts = [0, 70] + list(range(71, 80)) + [150]
    for a, e in zip(cuts, cuts[1:]):
        y, st = d["scan"].forward(d["x"][:, a:e], d["dt"][:, a:e].contiguous(), d["Bm"][:, a:e],
                                  d["Cm"][:, a:e], state=st, cont=a > 0)
        parts.append(y)
    w = 0.0 if dt == "f32" else 2.0 ** -8
    check(torch.cat(parts, 1), ref, mag, "y", steps=64 + T, weights=w)
    check(st, rs, ms, "state", steps=64 + T)


@pytest.mark.parametrize("off", [0, 1, 8])
def test_views(off):
    """x, B and C as slices of one tensor at any offset: the same bits."""
    g = gen(off)
    B, T, H, P, G, N = 2, 70, 2, 24, 1, 16
    wide = normal(g, B, T, off + H * P + 2 * G * N + 7, dtype=torch.bfloat16)
    x = wide[..., off:off + H * P].unflatten(-1, (H, P))
    Bm = wide[..., off + H * P:off + H * P + G * N].unflatten(-1, (G, N))
    Cm = wide[..., off + H * P + G * N:off + H * P + 2 * G * N].unflatten(-1, (G, N))
    dt = normal(g, B, T, H, dtype=torch.bfloat16, shift=-2.0)
    scan = sdm.SelectiveScan(-torch.ones(H).cuda())
    args, dense = (x, dt, Bm, Cm), (x.contiguous(), dt, Bm.contiguous(), Cm.contiguous())
    for a, c in zip(scan.forward(*args), scan.forward(*dense)):
        assert torch.equal(a, c)
    dy = normal(g, B, T, H, P, dtype=torch.bfloat16)
    a, c = scan.backward(*args, dy), scan.backward(*dense, dy)
    assert all(torch.equal(a[k], c[k]) for k in a)


def test_strides_of_single_dimensions_say_nothing():
    """One token of one sequence, with strides that no row uses."""
    d = inputs(71, 1, 1, 2, 16, 8, 1, "bf16", "sbD", None, True)
    odd = {k: torch.as_strided(d[k], d[k].shape, (1 << 40, 1 << 30, *d[k].stride()[2:]))
           for k in ("x", "Bm", "Cm")}
    y, s = d["scan"].forward(d["x"], d["dt"], d["Bm"], d["Cm"], state=d["S0"].clone(), cont=True)
    y2, s2 = d["scan"].forward(odd["x"], d["dt"], odd["Bm"], odd["Cm"], state=d["S0"].clone(), cont=True)
    assert torch.equal(y, y2) and torch.equal(s, s2)


def test_token_stride_limit():
    """Rows of a tile lie within 31 bits of each other, or the call is refused."""
    d = inputs(72, 1, 2, 2, 16, 8, 1, "bf16", "s", None, False)
    far = torch.empty((1 << 22) + 64, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(far, (1, 2, 2, 16), (1 << 22, 1 << 22, 16, 1))
    with pytest.raises(sdm.SDMError, match="stride"):
        d["scan"].forward(x, d["dt"], d["Bm"], d["Cm"])


def test_rows_behind_the_length_are_not_read():
    lens = [150, 40, 0]
    d = inputs(41, 3, 150, 2, 20, 16, 1, "bf16", "sbD", lens, True)
    dy = normal(gen(1), 3, 150, 2, 20, dtype=torch.bfloat16)
    names = ("x", "dt", "Bm", "Cm")
    y, s = d["scan"].forward(*(d[k] for k in names), state=d["S0"].clone(), cont=True, lengths=d["lengths"])
    g = d["scan"].backward(*(d[k] for k in names), dy, state=d["S0"], lengths=d["lengths"])
    bad = {k: d[k].clone() for k in names}
    bdy = dy.clone()
    for b, n in enumerate(lens):
        for k, v in zip(names, (math.nan, math.inf, math.nan, -math.inf)):
            bad[k][b, n:] = v
        bdy[b, n:] = math.nan
    y2, s2 = d["scan"].forward(*(bad[k] for k in names), state=d["S0"].clone(), cont=True,
                               lengths=d["lengths"])
    g2 = d["scan"].backward(*(bad[k] for k in names), bdy, state=d["S0"], lengths=d["lengths"])
    assert torch.equal(y, y2) and torch.equal(s, s2)
    assert all(torch.equal(g[k], g2[k]) for k in g)
    assert (y[1, 40:] == 0).all() and torch.equal(s[2], d["S0"][2])


def test_deterministic_and_graph_replay():
    d = inputs(51, 2, 1100, 2, 32, 32, 1, "bf16", "sbD", None, True)
    a = [d[k] for k in ("x", "dt", "Bm", "Cm")]
    dy = normal(gen(2), 2, 1100, 2, 32, dtype=torch.bfloat16)
    scan = d["scan"]
    g1, g2 = scan.backward(*a, dy, state=d["S0"]), scan.backward(*a, dy, state=d["S0"])
    assert all(torch.equal(g1[k], g2[k]) for k in g1)
    ws = torch.empty(scan.workspace_size(*a), dtype=torch.uint8, device="cuda")
    y, s = torch.empty_like(d["x"]), torch.empty_like(d["S0"])
    scan.forward(*a, state=s, y=y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        scan.forward(*a, state=s, cont=True, y=y, workspace=ws)
    ref = d["S0"].clone()
    s.copy_(d["S0"])
    for n in range(3):
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = scan.forward(*a, state=ref, cont=True)
        assert torch.equal(y, want) and torch.equal(s, ref), n


def test_refusals():
    d = inputs(61, 2, 8, 4, 16, 8, 2, "bf16", "sbD", [8, 8], True)
    scan, x, dt, Bm, Cm, S0 = (d[k] for k in ("scan", "x", "dt", "Bm", "Cm", "S0"))
    for call in (
        lambda: scan.forward(x, dt, Bm, Cm, cont=True),
        lambda: scan.forward(x.half(), dt.half(), Bm.half(), Cm.half()),
        lambda: scan.forward(x, dt.float(), Bm, Cm),
        lambda: scan.forward(x, dt, Bm, Cm.float()),
        lambda: scan.forward(x, dt, Bm, Cm[..., :4]),
        lambda: scan.forward(x[:, :, :2], dt, Bm, Cm),
        lambda: scan.forward(x, dt[:, :4], Bm, Cm),
        lambda: scan.forward(x[..., ::2], dt, Bm, Cm),
        lambda: scan.forward(x, dt, Bm, Cm, state=S0.bfloat16(), cont=True),
        lambda: scan.forward(x, dt, Bm, Cm, lengths=d["lengths"].long()),
        lambda: scan.forward(x, dt, Bm.repeat(1, 1, 2, 1)[:, :, :3], Cm.repeat(1, 1, 2, 1)[:, :, :3]),
        lambda: scan.forward(x, dt, normal(gen(0), 2, 8, 1, 129, dtype=x.dtype),
                             normal(gen(0), 2, 8, 1, 129, dtype=x.dtype)),
        lambda: scan.forward(x, dt, Bm, Cm, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: scan.forward(x[:, :0], dt[:, :0].contiguous(), Bm[:, :0], Cm[:, :0]),
        lambda: scan.forward(x.cpu(), dt, Bm, Cm),
        lambda: scan.backward(x, dt, Bm, Cm, x.float()),
        lambda: scan.backward(x, dt, Bm, Cm, x, state=S0[:1]),
        lambda: sdm.SelectiveScan(d["A"].double()),
        lambda: sdm.SelectiveScan(d["A"], D=d["D"][:2]),
    ):
        with pytest.raises(sdm.SDMError):
            call()
