"""GPU tests of the gradients of linear attention's decays: every value within a bound
from its own token's terms (decay_ref)."""
import math

import pytest
import torch

import decay_ref as D
import mixer_ref as R
from block_ref import assert_within, rounded
from decay_cases import CASES, arguments, case
from selective_state_space_56_amd import linear_attn_bwd, linear_attn_fwd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
CPU = torch.device("cpu")


def gradients(s, off=None):
    return linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], h0=s.get("h0"), dlast=s.get("dlast"), offsets=off)


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("name", list(CASES))
def test_decays(name, io):
    s, off = case(name, io, CPU)
    want = rounded(D.dg(*arguments(s), offsets=off), F32)
    s, off = case(name, io, "cuda")
    assert_within(name, gradients(s, off)["dg"], want)


@pytest.mark.parametrize("io", [F32, BF])
def test_no_gradient_without_a_state(io):
    """The first step's decay multiplies no state without h0, nor does one that follows rows of zeros."""
    s, _ = case("padded rows", io, "cuda")
    dg = gradients(s)["dg"]
    assert not dg[:, :76].any() and dg[:, 76:170].any(1).all()


@pytest.mark.parametrize("io", [F32, BF])
def test_what_a_cut_drops_reaches_no_later_gradient(io):
    s, _ = case("strong steps", io, CPU)
    cut = 90
    s["g"][0, cut] = -math.inf
    clean = {n: t.clone() for n, t in s.items()}
    for n in ("q", "k", "v", "dout"):
        s[n][0, 80:cut] = math.nan
    want = rounded(D.dg(*arguments(clean)), F32)
    d = gradients({n: t.cuda() for n, t in s.items()})
    assert_within("dg", d["dg"][:, cut:], tuple(x[:, cut:] for x in want))
    for n in ("dq", "dk", "dv"):
        assert d[n][:, cut:].isfinite().all(), n
    # and what comes behind it reaches no earlier one
    s = {n: t.clone() for n, t in clean.items()}
    for n in ("q", "k", "v", "dout"):
        s[n][0, cut:cut + 5] = math.nan
    d = gradients({n: t.cuda() for n, t in s.items()})
    assert_within("dg", d["dg"][:, :cut + 1], tuple(x[:, :cut + 1] for x in want))
    for n in ("dq", "dk", "dv"):
        assert d[n][:, :cut].isfinite().all(), n


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("K,V", [(64, 64), (200, 136), (24, 256)])
def test_strided_rows(K, V, io):
    """Column slices of one projection's rows give the bits of contiguous tensors."""
    n, H, G = 200, 2, 1
    gen = torch.Generator().manual_seed(9)
    rows = torch.randn((1, n, 2 * G * K + H * V + 3), generator=gen).to(io).cuda()
    s = {"q": rows[..., 1:1 + G * K].unflatten(-1, (G, K)), "k": rows[..., 1 + G * K:1 + 2 * G * K].unflatten(-1, (G, K)),
         "v": rows[..., 1 + 2 * G * K:1 + 2 * G * K + H * V].unflatten(-1, (H, V)),
         "g": -torch.rand((1, n, H), generator=gen).cuda(), "dout": torch.randn((1, n, H, V), generator=gen).to(io).cuda()}
    near = {m: t.contiguous() for m, t in s.items()}
    assert torch.equal(gradients(s)["dg"], gradients(near)["dg"])
    assert_within("dg", gradients(s)["dg"], rounded(D.dg(*arguments({m: t.cpu() for m, t in near.items()})), F32))


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("fixed", [False, True])
def test_many_chunks_and_heads(fixed, io):
    """More of them than a launch has workgroups (65536): the first heads and the last ones."""
    B, n, H, K = (1, 1000, 2100, 8) if io == F32 else (2, 1030, 2000, 8)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(io)
    s = {m: normal(B, n, H, K) for m in ("q", "k", "v", "dout")}
    s["g"] = -0.1 * torch.rand((H,) if fixed else (B, n, H), generator=gen, device="cuda")
    got = gradients(s)["dg"]
    for at in (slice(0, 3), slice(H - 3, H)):
        part = {m: (t[at] if m == "g" and fixed else t[..., at] if m == "g" else t[:, :, at]).cpu() for m, t in s.items()}
        assert_within("dg", got[..., at], rounded(D.dg(*arguments(part)), F32))


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("name", ["40 x 72, shared keys, states", "65 steps", "packed", "one step"])
def test_a_state_on_one_side_only(name, io):
    s, off = case(name, io, CPU)
    h0, dlast, zeros = s["h0"], s["dlast"], torch.zeros_like(s["h0"])
    args, dev = arguments(s), {n: t.cuda() for n, t in s.items()}
    off_d = None if off is None else off.cuda()
    for mine, theirs in (((h0, zeros), (dev["h0"], None)), ((zeros, dlast), (None, dev["dlast"])), ((zeros, zeros), (None, None))):
        got = linear_attn_bwd(*(dev[n] for n in "qkvg"), dev["dout"], h0=theirs[0], dlast=theirs[1], offsets=off_d)["dg"]
        assert_within(name, got, rounded(D.dg(*args[:6], *mine, offsets=off), F32))


@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("K,V,n", [(16, 24, 40), (64, 64, 70), (136, 32, 33)])
def test_decays_against_differences(K, V, n, fixed):
    """dg of one step (or head) against (loss(g + h) - loss(g - h)) / 2 h there, the loss from the forward's
    outputs and states. Values are positive, so that the loss is the sum of its terms' magnitudes. A term
    holds the step's decay once (a fixed one n times at most): the central difference is off by h^2 / 6 of the
    loss (n^3 h^2 / 6). The forward rounds each term n + K + V + 64 times at most."""
    gen = torch.Generator().manual_seed(3)

    def values(*shape):
        return torch.rand(shape, generator=gen).cuda()
    q, k, v, dout = values(2, n, 1, K), values(2, n, 1, K), values(2, n, 2, V), values(2, n, 2, V)
    h0, dlast = values(2, 2, K, V), values(2, 2, K, V)
    g = -0.2 * values(2) if fixed else -0.2 * values(2, n, 2)
    d = linear_attn_bwd(q, k, v, g, dout, h0=h0, dlast=dlast)["dg"]
    h = 2.0 ** -9 if fixed else 2.0 ** -5

    def loss(g):
        out, last = linear_attn_fwd(q, k, v, g, h0=h0)
        return (out.double() * dout.double()).sum() + (last.double() * dlast.double()).sum()
    for at in ((0,), (1,)) if fixed else ((0, 0, 0), (1, 5, 1), (0, n // 2, 1), (1, n - 1, 0)):
        up, down = g.clone(), g.clone()
        up[at] += h
        down[at] -= h
        a, b, step = loss(up), loss(down), float(up[at].double() - down[at].double())
        off = float(a) * (((n * h) ** 3 if fixed else h ** 3) / 6 + 2 * (2 * (n + K + V) + 128) * 2.0 ** -24)
        assert abs(float(d[at]) * step - float(a - b)) <= 2 * off, at
        assert off < 0.25 * abs(float(a - b))     # the difference says something


@pytest.mark.parametrize("packed", [False, True])
def test_heads_in_turn(packed):
    """Chunks' states of more than 8 GiB: the backward goes through the heads in turn. Its first and last
    groups in the first and last sequences, and one decay for each head as the sum over all tokens."""
    B, n, H, G, K = 2048, 128, 32, 16, 128
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)

    def normal(*shape, io=BF):
        return torch.randn(shape, generator=gen, device="cuda").to(io)
    s = {"q": normal(B, n, G, K), "k": normal(B, n, G, K), "v": normal(B, n, H, K), "dout": normal(B, n, H, K),
         "h0": normal(B, H, K, K, io=F32), "g": -0.2 * torch.rand((B, n, H), generator=gen, device="cuda")}
    rows = {m: t.flatten(0, 1) if packed and m != "h0" else t for m, t in s.items()}
    off = torch.arange(0, B * n + 1, n, device="cuda") if packed else None
    d = gradients(rows, off)
    for i in (0, B - 1):
        for h in (0, H - 2):
            heads, group = slice(h, h + 2), slice(h // 2, h // 2 + 1)
            part = {m: t[i:i + 1, :, group if m in "qk" else heads].cpu() for m, t in s.items() if m != "h0"}
            part["h0"] = s["h0"][i:i + 1, heads].cpu()
            ref = R.linattn(*(part[m] for m in ("q", "k", "v", "g")), K ** -0.5, part["h0"], None, part["dout"])
            for m in ("dq", "dk", "dv"):
                got = d[m].view(s[m[1:]].shape)[i:i + 1, :, heads if m == "dv" else group]
                assert_within(m, got, rounded(ref[m], BF))
            assert_within("dh0", d["dh0"][i:i + 1, heads], rounded(ref["dh0"], F32))
            args = [part[m] for m in ("q", "k", "v", "g")]
            want = D.dg(*args, K ** -0.5, part["dout"], part["h0"])
            assert_within("dg", d["dg"].view(B, n, H)[i:i + 1, :, heads], rounded(want, F32))
    del d
    fixed = -0.1 * torch.rand(H, generator=gen, device="cuda")
    rows["g"] = fixed.expand(B, n, H).contiguous().view(-1, H) if packed else fixed.expand(B, n, H).contiguous()
    each = gradients(rows, off)["dg"].double().view(-1, H)
    rows["g"] = fixed
    one = gradients(rows, off)["dg"].double()
    # the same values but for the order: a float32 sum for each chunk, and of these
    parts = 3 * B + 4
    assert ((one - each.sum(0)).abs() <= (2 * parts + 4) * 2.0 ** -24 * each.abs().sum(0)).all() and one.all()

