"""GPU tests of the gradients of linear attention's decays: every value within a bound
from its own token's terms (decay_ref)."""
import math

import pytest
import torch

import decay_ref as D
from block_ref import assert_within, rounded
from decay_cases import CASES, arguments, case
from selective_state_space_56_amd import linear_attn_bwd

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
