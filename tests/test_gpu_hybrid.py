"""The sequence mixers and the SDM core together, as a hybrid stack uses them: a
recurrent block (short convolution, selective scan), a local block
(sliding-window attention) and an SDM block, over a prompt and then token by
token, eager, on a stream of its own and from a captured graph; and the
gradients of the recurrent block chained by hand."""
import pytest
import torch

import sparse_memory_linear_select_amd as sdm
from mix_util import check, gen, leaf, normal

pytestmark = pytest.mark.gpu

B, T, H, P, N, G = 2, 140, 4, 32, 16, 1
D = H * P                     # width of the stream between the blocks
HQ, HK, HD = 4, 2, 32
W, S = 48, 2
SQ, WR = 16, 8                # SDM: 256 slots, 8 written and read


class Stack:
    """Projections are plain matrix products; the mixers are the library's."""

    def __init__(self, dtype):
        g = gen(7)
        C = D + 2 * G * N

        def proj(i, o):
            return normal(g, i, o, dtype=dtype, scale=i ** -0.5)

        self.dtype = dtype
        self.w_in, self.w_dt = proj(D, C), proj(D, H)
        self.w_qkv = proj(D, (HQ + 2 * HK) * HD)
        self.w_k, self.w_q, self.w_v = proj(D, 2 * SQ), proj(D, 2 * SQ), proj(D, D)
        self.w_a = proj(D, 2)
        self.conv = sdm.CausalConv(normal(g, C, 4, scale=0.5), normal(g, C, scale=0.1))
        self.scan = sdm.SelectiveScan(-(0.5 + torch.rand(H, generator=g)).cuda(), D=normal(g, H),
                                      dt_bias=normal(g, H, shift=-2.0))
        self.att = sdm.WindowAttention(HQ, HK, HD, W, S)
        self.core = sdm.SDM(normal(g, 1, SQ * SQ, D, scale=0.02), WR, WR)

    def new_state(self):
        return dict(conv=torch.zeros(B, 3, D + 2 * G * N, dtype=self.dtype, device="cuda"),
                    scan=torch.zeros(B, H, P, N, device="cuda"),
                    cache=self.att.new_cache(B, self.dtype),
                    pos=torch.zeros(B, dtype=torch.int64, device="cuda"),
                    M=torch.empty(B, 1, SQ * SQ, D, device="cuda"))

    def __call__(self, x, st, cont):
        n = x.shape[1]
        xbc, _ = self.conv.forward(x @ self.w_in, state=st["conv"], cont=cont)
        xs = xbc[..., :D].unflatten(-1, (H, P))
        bm = xbc[..., D:D + G * N].unflatten(-1, (G, N))
        cm = xbc[..., D + G * N:].unflatten(-1, (G, N))
        y, _ = self.scan.forward(xs, x @ self.w_dt, bm, cm, state=st["scan"], cont=cont)
        x = x + y.flatten(2)
        qkv = (x @ self.w_qkv).unflatten(-1, (HQ + 2 * HK, HD))
        o, _ = self.att.forward(qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HK], qkv[:, :, HQ + HK:],
                                cache=st["cache"], pos=st["pos"] if cont else None, cont=cont)
        st["pos"] += n
        x = x + o.flatten(2)
        gates = (x @ self.w_a).float()
        y, _ = self.core.forward((x @ self.w_k)[:, :, None].contiguous(),
                                 (x @ self.w_q)[:, :, None].contiguous(),
                                 (x @ self.w_v)[:, :, None].contiguous(),
                                 torch.exp(-torch.nn.functional.softplus(gates[..., :1])),
                                 torch.sigmoid(gates[..., 1:]), M=st["M"], cont=cont)
        return x + y[:, :, 0].to(x.dtype)


def run(stack, x, cuts):
    st, parts = stack.new_state(), []
    for a, e in zip(cuts, cuts[1:]):
        parts.append(stack(x[:, a:e].contiguous(), st, a > 0))
    return torch.cat(parts, 1), st


def test_prompt_then_tokens():
    """float32: a prompt and single tokens give what one pass over everything gives.

    The mixers differ by their order of summing (some 1e-6 of the values here);
    SDM's selection of slots is discrete, so a near tie may fall the other way:
    nearly all outputs agree closely."""
    stack = Stack(torch.float32)
    x = normal(gen(1), B, T, D)
    y, st = run(stack, x, (0, T))
    y2, st2 = run(stack, x, [0, 100] + list(range(101, T + 1)))
    err = (y - y2).abs() / (1 + y.abs())
    assert float((err < 1e-3).float().mean()) > 0.97
    for n in ("conv", "scan"):  # the first block holds no discrete choice
        assert float((st[n] - st2[n]).abs().max()) < 1e-4
    assert torch.equal(st["pos"], st2["pos"]) and torch.isfinite(y2).all()


def test_other_stream_and_graph():
    """bfloat16: on a stream of its own the same bits; a captured step replayed token by token
    gives the eager steps' bits, with both states living side by side."""
    stack = Stack(torch.bfloat16)
    x = normal(gen(2), B, T, D, dtype=torch.bfloat16)
    y, st = run(stack, x, [0, 90] + list(range(91, 110)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, st2 = run(stack, x, [0, 90] + list(range(91, 110)))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and torch.equal(st["scan"], st2["scan"])

    _, sg = run(stack, x, (0, 90))
    step = x[:, 90:91].clone()
    warm = {k: (tuple(c.clone() for c in v) if k == "cache" else v.clone()) for k, v in sg.items()}
    stack(step, warm, True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = stack(step, sg, True)
    for t in range(90, 109):
        step.copy_(x[:, t:t + 1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y[:, t:t + 1]), t
        _ = (y.float() * 2).sum().item()  # eager work between replays
    assert torch.equal(sg["scan"], st["scan"]) and torch.equal(sg["cache"][0], st["cache"][0])


def test_gradients_chain():
    """conv -> scan -> attention, backward by hand, against autograd in 64 bits."""
    stack = Stack(torch.float32)
    g = gen(3)
    n, C = 100, D + 2 * G * N
    u, dt = normal(g, 1, n, C), normal(g, 1, n, H, shift=-1.0)
    do = normal(g, 1, n, HQ, HD)
    # forward: the scan's output is the attention's queries, B and C padded into keys and values
    xbc, _ = stack.conv.forward(u)
    cut = lambda t: (t[..., :D].unflatten(-1, (H, P)), t[..., D:D + N].unflatten(-1, (G, N)),  # noqa: E731
                     t[..., D + N:].unflatten(-1, (G, N)))
    xs, bm, cm = cut(xbc)
    y, _ = stack.scan.forward(xs, dt, bm, cm)
    k = y[:, :, :HK] * 0.5
    v = y[:, :, HK:]
    o, lse = stack.att.forward(y, k, v)
    ga = stack.att.backward(y, k, v, o, lse, do)
    dy = ga["dq"].clone()
    dy[:, :, :HK] += 0.5 * ga["dk"]
    dy[:, :, HK:] += ga["dv"]
    gs = stack.scan.backward(xs, dt, bm, cm, dy)
    dxbc = torch.cat([gs["dx"].flatten(2), gs["dB"].flatten(2), gs["dC"].flatten(2)], -1)
    gc = stack.conv.backward(u, dxbc)

    lu, ldt, lw, lA = leaf(u), leaf(dt), leaf(stack.conv.weight), leaf(stack.scan.A)
    lb, lD, lbias = (t.cpu().double() for t in (stack.conv.bias, stack.scan.D, stack.scan.dt_bias))
    ue = torch.cat([torch.zeros(1, 3, C, dtype=torch.float64), lu], 1)
    z = sum(ue[:, i:i + n] * lw[:, i] for i in range(4)) + lb
    rx, rb, rc = cut(z * torch.sigmoid(z))
    delta = torch.nn.functional.softplus(ldt + lbias, threshold=40)
    st, ys = torch.zeros(1, H, P, N, dtype=torch.float64), []
    for t in range(n):
        st = torch.exp(delta[:, t] * lA)[..., None, None] * st + \
            (delta[:, t, :, None] * rx[:, t])[..., None] * rb[:, t, :, None]
        ys.append((st * rc[:, t, :, None]).sum(-1) + lD[:, None] * rx[:, t])
    ry = torch.stack(ys, 1)
    i, j = torch.arange(n)[:, None], torch.arange(n)[None]
    see = (j <= i) & ((i - j < W) | (j < S))
    kh, vh = (t.repeat_interleave(HQ // HK, 2) for t in (ry[:, :, :HK] * 0.5, ry[:, :, HK:]))
    s = torch.einsum("bihd,bjhd->bhij", ry, kh) * HD ** -0.5
    ro = torch.einsum("bhij,bjhd->bihd", torch.softmax(s.masked_fill(~see, float("-inf")), -1), vh)
    ref = torch.autograd.grad((ro * do.cpu().double()).sum(), (lu, ldt, lw, lA))
    # three float32 operators in a row: 2^-24 times a few thousand operations of the largest values
    for got, r, name in ((gc["dx"], ref[0], "du"), (gs["ddt"], ref[1], "ddt"),
                         (gc["dweight"], ref[2], "dweight"), (gs["dA"], ref[3], "dA")):
        check(got, r, r.abs().max(), name, steps=4000)
