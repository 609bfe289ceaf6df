"""GPU tests of the mixer operators where calls meet: streams, captured graphs,
memory that held something else, rows and states past 32 bits, many short
sequences, and shapes drawn at random. What has been checked value by value
elsewhere serves as the expected result here, bit for bit."""
import random

import pytest
import torch

import mixer_ref as R
from block_ref import assert_within, rounded
from selective_state_space_56_amd import (linear_attn_bwd, linear_attn_fwd, linear_attn_update, qk_norm_rope_bwd,
                                          qk_norm_rope_fwd)
from test_mixer_gpu import BF, F32, check, gen, make, normal, turn_case

pytestmark = pytest.mark.gpu
ARGS = ("q", "k", "v", "g")


def run(s, off=None):
    """Both directions, as a flat list of tensors."""
    args = [s[n] for n in ARGS]
    d = linear_attn_bwd(*args, s["dout"], h0=s.get("h0"), dlast=s.get("dlast"), offsets=off)
    return [*linear_attn_fwd(*args, h0=s.get("h0"), offsets=off), *d.values()]


def same(xs, ys):
    return len(xs) == len(ys) and all(torch.equal(x, y) for x, y in zip(xs, ys))


def dirty(n=1 << 27):
    """Memory that the next calls are given holds NaN."""
    x = torch.full((n // 4,), float("nan"), device="cuda")
    del x


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("K,V,G", [(64, 40, 1), (128, 128, 2), (200, 136, 1)])
def test_workspace_holds_nothing_on_entry(K, V, G, io):
    s = make(50, (1, 2177), 2, G, K, V, io, states=1)
    off = torch.tensor([1, 1, 1100, 1103, 2177], device="cuda")
    p = {n: t[0] if n in (*ARGS, "dout") else t.expand(4, -1, -1, -1).contiguous() for n, t in s.items()}
    first, packed = run(s), run(p, off)
    for _ in range(2):
        dirty()
        assert same(run(s), first)
        dirty()
        assert same(run(p, off), packed)


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("K,V", [(256, 256), (200, 136), (24, 256), (256, 24), (64, 64)])
def test_segments_of_every_layout(K, V, io):
    check(make(K + V, (1, 1090), 2, 1, K, V, io, states=1))


@pytest.mark.parametrize("io", [F32, BF])
def test_many_short_sequences(io):
    rnd = random.Random(3)
    lens = [rnd.choice((0, 1, 2, 7, 31, 33, 64, 65)) for _ in range(300)]
    off = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda")
    check(make(51, (sum(lens),), 2, 1, 24, 16, io, states=len(lens)), offsets=off)


@pytest.mark.parametrize("io", [F32, BF])
def test_long_packed_sequences(io):
    # several with states between stretches of 1024 steps, ends on both sides of a stretch's
    lens = [1030, 1024, 2049, 1025, 5]
    off = torch.tensor([3 + sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda")
    check(make(58, (int(off[-1]) + 2,), 2, 1, 16, 24, io, states=len(lens)), offsets=off)


@pytest.mark.parametrize("seed", range(16))
def test_drawn_shapes(seed):
    rnd = random.Random(seed)
    K, V = 8 * rnd.randint(1, 32), 8 * rnd.randint(1, 32)
    G = rnd.randint(1, 3)
    H, io = G * rnd.randint(1, 3), rnd.choice((F32, BF))
    kw = dict(fixed=rnd.random() < 0.4, strided=rnd.random() < 0.5)
    if rnd.random() < 0.5:
        lens = [rnd.choice((0, 1, 5, 63, 64, 130)) for _ in range(rnd.randint(1, 4))]
        first = rnd.randint(0, 3)
        off = torch.tensor([first + sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda")
        s = make(seed, (int(off[-1]) + rnd.randint(0, 3),), H, G, K, V, io, states=rnd.choice((0, len(lens))), **kw)
        check(s, offsets=off)
    else:
        B = rnd.randint(1, 2)
        s = make(seed, (B, rnd.randint(1, 150)), H, G, K, V, io, states=rnd.choice((0, B)), **kw)
        check(s, scale=rnd.choice((None, 0.5, -1.0)))


def test_scale_of_zero():
    s = make(52, (1, 70), 2, 1, 16, 16, BF, states=1)
    out, last = linear_attn_fwd(*(s[n] for n in ARGS), scale=0.0, h0=s["h0"])
    d = linear_attn_bwd(*(s[n] for n in ARGS), s["dout"], scale=0.0, h0=s["h0"])
    assert not out.any() and torch.equal(last, linear_attn_fwd(*(s[n] for n in ARGS), h0=s["h0"])[1])
    for n in ("dq", "dk", "dv", "dg", "dh0"):
        assert not d[n].any(), n


@pytest.mark.parametrize("io", [F32, BF])
def test_one_tensor_for_several_operands(io):
    s = make(53, (2, 100), 2, 2, 64, 64, io)
    x, y, z = s["q"], s["q"].clone(), s["q"].clone()
    assert same(run({**s, "q": x, "k": x, "v": x, "dout": x}), run({**s, "q": x, "k": y, "v": z, "dout": z}))
    one = [t[:, 0].contiguous() for t in (x, s["g"])]
    a, b = normal(gen(1), 2, 2, 64, 64), None
    b = a.clone()
    assert torch.equal(linear_attn_update(a, one[0], one[0], one[0], one[1]),
                       linear_attn_update(b, one[0], one[0].clone(), one[0].clone(), one[1]))


@pytest.mark.parametrize("io", [F32, BF])
def test_outputs_as_columns(io):
    s = make(54, (2, 70), 2, 2, 32, 24, io)
    out, _ = linear_attn_fwd(*(s[n] for n in ARGS))
    wide = torch.full((2, 70, 60), 7.0, dtype=io, device="cuda")
    linear_attn_fwd(*(s[n] for n in ARGS), out=wide[..., 5:53].unflatten(-1, (2, 24)))
    assert torch.equal(wide[..., 5:53].reshape(out.shape), out)
    assert (wide[..., :5] == 7).all() and (wide[..., 53:] == 7).all()
    tok = [s[n][:, 0].contiguous() for n in ARGS]
    a = normal(gen(2), 2, 2, 32, 24)
    b = a.clone()
    wide.fill_(7.0)
    linear_attn_update(b, *tok, out=wide[:, 0, 5:53].unflatten(-1, (2, 24)))
    assert torch.equal(wide[:, 0, 5:53].reshape(2, 2, 24), linear_attn_update(a, *tok)) and torch.equal(a, b)
    assert (wide[:, 0, :5] == 7).all() and (wide[:, 0, 53:] == 7).all() and (wide[:, 1:] == 7).all()


def test_rows_past_32_bits():
    # 40 000 rows 65 536 elements apart: the last lie beyond 2^31 elements and 2^32 bytes
    n, H, K, V = 40000, 1, 16, 24
    rows = torch.empty((n, 1 << 16), dtype=BF, device="cuda")
    ends = (0, 16, 32, 56, 80, 96, 112, 136, 152, 168)
    q, k, v, do, dq, dk, dv, qn, kn = (rows[:, a:b].unflatten(1, (1, b - a)) for a, b in zip(ends[:-1], ends[1:]))
    gn = gen(55)
    for t in (q, k, v, do):
        t.copy_(normal(gn, *t.shape, io=BF))
    g = -torch.rand(n, H, generator=gn, device="cuda")
    off = torch.tensor([0, 39000, 39990, n], device="cuda")
    near = [t.contiguous() for t in (q, k, v)]
    out, last = linear_attn_fwd(*near, g, offsets=off)
    d = linear_attn_bwd(*near, g, do.contiguous(), offsets=off)
    assert same(linear_attn_fwd(q, k, v, g, offsets=off, out=dv), (out, last)) and torch.equal(dv, out)
    e = linear_attn_bwd(q, k, v, g, do, offsets=off, dq=dq, dk=dk, dv=dv)
    assert same(list(d.values()), list(e.values()))
    pos, freqs, w = torch.arange(n, device="cuda"), torch.full((4,), 0.01, device="cuda"), torch.ones(16, device="cuda")
    y, z = qk_norm_rope_fwd(near[0], near[1], pos, freqs, w, w)
    qk_norm_rope_fwd(q, k, pos, freqs, w, w, q_out=qn, k_out=kn)
    assert torch.equal(qn, y) and torch.equal(kn, z)
    a = qk_norm_rope_bwd(near[0], near[1], pos, freqs, w, w, y, z)
    b = qk_norm_rope_bwd(q, k, pos, freqs, w, w, qn, kn, dq=dq, dk=dk)
    assert same(list(a.values()), list(b.values()))


def test_states_past_32_bits():
    n, K, V = 33000, 256, 256     # 2.16e9 elements of state
    gn = gen(56)
    q, k, v = normal(gn, n, 1, K, io=BF), normal(gn, n, 1, K, io=BF), normal(gn, n, 1, V, io=BF)
    g = -torch.rand(n, 1, generator=gn, device="cuda")
    state = torch.zeros((n, 1, K, V), device="cuda")
    some = torch.tensor([0, 1, 16383, 16384, 32767, 32768, n - 1])
    at = some.cuda()
    state[at] = normal(gn, len(some), 1, K, V)
    before = state[at]
    # a prompt of one token each, and a token more
    out, last = linear_attn_fwd(q[:, None], k[:, None], v[:, None], g[:, None], h0=state)
    ref = R.linattn(*(t[at][:, None] for t in (q, k, v, g)), K ** -0.5, before)
    assert_within("out", out[at], rounded(ref["out"], BF))
    assert_within("last_state", last[at], rounded(ref["last_state"], F32))
    del last
    ref = R.update(before, q[at], k[at], v[at], g[at], K ** -0.5)
    out = linear_attn_update(state, q, k, v, g)
    assert_within("state", state[at], rounded(ref["state"], F32))
    assert_within("out", out[at], rounded(ref["out"], BF))


def test_streams():
    """Calls on several streams at once, each on tensors that its own stream has
    made, give what they give alone."""
    cases = [make(57 + i, (1, 1500 + 100 * i), 4, 2, 64, 64, BF, states=1) for i in range(3)]
    turns = [turn_case(60 + i, 700, 4, 2, 64, 32, None, BF) for i in range(3)]

    def both(i, s):
        q, k, pos, freqs, wq, wk, dy, dz = turns[i]
        e = qk_norm_rope_bwd(q, k, pos, freqs, wq, wk, dy, dz)
        return run(s) + [*qk_norm_rope_fwd(q, k, pos, freqs, wq, wk), *e.values()]
    alone = [both(i, s) for i, s in enumerate(cases)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None] * 3
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                later = {n: t * 1 if n != "h0" else t.clone() for n, t in cases[i].items()}  # made on this stream
                got[i] = both(i, later)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(alone, got))


@pytest.mark.parametrize("io", [F32, BF])
def test_in_graphs(io):
    """A layer's calls in both directions and a decode token, captured into two graphs
    that share their memory, replayed with new inputs, eager calls and
    synchronizations between: every replay is the eager result."""
    sizes = [((1, 1300), 4, 2, 64, 64, False), ((1, 1300), 2, 1, 40, 64, True)]
    sets = []
    for i, (lead, H, G, K, V, fixed) in enumerate(sizes):
        s = make(70 + i, lead, H, G, K, V, io, fixed=fixed, states=1)
        s["pos"] = torch.arange(1300, device="cuda") * (i + 1)
        s["freqs"] = torch.full((K // 8 * 4,), 0.01, device="cuda")
        s["w"] = 1 + 0.1 * normal(gen(80 + i), K)
        sets.append(s)

    def layer(s):
        y, z = qk_norm_rope_fwd(s["q"][0], s["k"][0], s["pos"], s["freqs"], s["w"], s["w"])
        t = {**s, "q": y[None], "k": z[None]}
        outs = run(t)
        back = qk_norm_rope_bwd(s["q"][0], s["k"][0], s["pos"], s["freqs"], s["w"], s["w"], outs[2][0], outs[3][0])
        state = outs[1].clone()
        g = s["g"] if s["g"].dim() == 1 else s["g"][:, -1]
        token = linear_attn_update(state, y[-1:], z[-1:], s["v"][:, -1], g.contiguous())
        return outs + list(back.values()) + [state, token]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            layer(s)
    torch.cuda.current_stream().wait_stream(side)
    graphs, held, pool = [], [], None
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            held.append(layer(s))
        pool = pool or graph.pool()
        graphs.append(graph)
    for turn in range(4):
        for s in sets:
            for n in ("q", "k", "v", "dout", "h0", "dlast"):
                s[n].copy_(normal(gen(90 + turn), *s[n].shape, io=s[n].dtype))
        dirty()
        for i in (0, 1, 1, 0)[turn], (1, 0, 0, 1)[turn]:
            want = layer(sets[i])
            graphs[i].replay()
            torch.cuda.synchronize()
            assert same(held[i], want), (turn, i, [torch.equal(a, b) for a, b in zip(held[i], want)])
    graphs[0].replay()
    graphs[1].replay()       # back to back
    torch.cuda.synchronize()
    assert same(held[0], layer(sets[0])) and same(held[1], layer(sets[1]))


@pytest.mark.parametrize("bad", ["K", "heads", "g shape", "g type", "h0", "offsets", "out", "device", "broadcast"])
def test_refusals_by_name(bad):
    s = make(99, (1, 8), 4, 2, 16, 16, BF)
    q, k, v, g = (s[n] for n in ARGS)
    kw = {}
    if bad == "K":
        q = k = normal(gen(1), 1, 8, 2, 12, io=BF)
    elif bad == "heads":
        q = k = normal(gen(1), 1, 8, 3, 16, io=BF)
    elif bad == "g shape":
        g = g[:, :4]
    elif bad == "g type":
        g = g.to(BF)
    elif bad == "h0":
        kw["h0"] = torch.zeros((1, 4, 16, 8), device="cuda")
    elif bad == "offsets":
        kw["offsets"] = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
        q, k, v, g = (t[0] for t in (q, k, v, g))
    elif bad == "out":
        kw["out"] = v
    elif bad == "device":
        k = k.cpu()
    elif bad == "broadcast":
        v = v[:, :1].expand(1, 8, 4, 16)
    with pytest.raises((ValueError, TypeError, RuntimeError)):
        linear_attn_fwd(q, k, v, g, **kw)
    torch.cuda.synchronize()
