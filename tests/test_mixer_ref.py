"""CPU tests of the mixer's plain implementations themselves: the forward
against the matrix form, the gradients against automatic ones and against
differences."""
import pytest
import torch

import mixer_ref as R


def inputs(seed, lead, H, G, K, V, fixed=False):
    gen = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=gen, dtype=torch.float64)
    g = -torch.rand((H,) if fixed else lead + (H,), generator=gen, dtype=torch.float64)
    return r(*lead, G, K), r(*lead, G, K), r(*lead, H, V), g


def matrix_form(q, k, v, g, scale, h0):
    """Every pair of steps at once, from the unrolled recurrence; batch form."""
    H = v.shape[2]
    q, k = (x.repeat_interleave(H // x.shape[2], 2) for x in (q, k))
    g = g.expand(v.shape[:3])
    L = v.shape[1]
    ell = g.cumsum(1).movedim(2, 1)
    d = (ell[..., :, None] - ell[..., None, :]).masked_fill(~torch.ones(L, L, dtype=torch.bool).tril(), float("-inf")).exp()
    out = torch.einsum("bhts,bthk,bshk,bshv->bthv", d, q, k, v)
    out = out + torch.einsum("bht,bthk,bhkv->bthv", ell.exp(), q, h0)
    end = (ell[..., -1:] - ell).exp()
    last = torch.einsum("bhs,bshk,bshv->bhkv", end, k, v) + ell[..., -1].exp()[..., None, None] * h0
    return scale * out, last


@pytest.mark.parametrize("fixed", [False, True])
def test_linattn_reference(fixed, monkeypatch):
    monkeypatch.setitem(R.SPLIT, torch.float64, 0.0)
    q, k, v, g = inputs(1, (2, 9), 4, 2, 8, 16, fixed)
    h0, dout, dlast = (torch.randn(2, 4, 8, 16, dtype=torch.float64), torch.randn(2, 9, 4, 16, dtype=torch.float64),
                       torch.randn(2, 4, 8, 16, dtype=torch.float64))
    leaves = [t.requires_grad_() for t in (q, k, v, g, h0)]
    out, last = matrix_form(*leaves[:4], 0.3, h0)
    grads = torch.autograd.grad((out * dout).sum() + (last * dlast).sum(), leaves)
    res = R.linattn(q, k, v, g, 0.3, h0, dout=dout, dlast=dlast)
    torch.testing.assert_close(res["out"][0], out.detach(), rtol=1e-10, atol=1e-10)
    torch.testing.assert_close(res["last_state"][0], last.detach(), rtol=1e-10, atol=1e-10)
    for n, want in zip(("dq", "dk", "dv", "dg", "dh0"), grads):
        torch.testing.assert_close(res[n][0], want, rtol=1e-9, atol=1e-9)


def test_linattn_reference_differences(monkeypatch):
    monkeypatch.setitem(R.SPLIT, torch.float64, 0.0)
    q, k, v, g = inputs(2, (1, 4), 2, 1, 8, 8)

    def f(*args):
        return matrix_form(*args, 0.5, torch.zeros(1, 2, 8, 8, dtype=torch.float64))[0]
    assert torch.autograd.gradcheck(f, [t.requires_grad_() for t in (q, k, v, g)])


def test_linattn_reference_packed(monkeypatch):
    monkeypatch.setitem(R.SPLIT, torch.float64, 0.0)
    q, k, v, g = inputs(3, (12,), 2, 2, 8, 8)
    off = torch.tensor([1, 5, 5, 11])
    res = R.linattn(q, k, v, g, 1.0, offsets=off)
    for a, b in ((1, 5), (5, 11)):
        want, last = matrix_form(q[None, a:b], k[None, a:b], v[None, a:b], g[None, a:b], 1.0,
                                 torch.zeros(1, 2, 8, 8, dtype=torch.float64))
        torch.testing.assert_close(res["out"][0][a:b], want[0], rtol=1e-10, atol=1e-10)
    torch.testing.assert_close(res["last_state"][0][2], last[0], rtol=1e-10, atol=1e-10)
    assert not res["out"][0][[0, 11]].any() and not res["last_state"][0][1].any()


def test_a_decay_of_zero_starts_anew(monkeypatch):
    monkeypatch.setitem(R.SPLIT, torch.float64, 0.0)
    q, k, v, g = inputs(4, (1, 7), 2, 1, 8, 8)
    g[:, 3] = float("-inf")
    res = R.linattn(q, k, v, g, 1.0, h0=torch.full((1, 2, 8, 8), float("nan"), dtype=torch.float64))
    want, _ = matrix_form(q[:, 3:], k[:, 3:], v[:, 3:], g[:, 3:].clamp(min=-700), 1.0,
                          torch.zeros(1, 2, 8, 8, dtype=torch.float64))
    torch.testing.assert_close(res["out"][0][:, 3:], want, rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("interleaved", [False, True])
def test_qknorm_reference(interleaved):
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(3, 2, 24, generator=gen, dtype=torch.float64, requires_grad=True)
    w = torch.randn(24, generator=gen, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(3, 2, 24, generator=gen, dtype=torch.float64)
    pos, freqs = torch.tensor([[0, 5, 900], [7, 1, 3]]), torch.rand(8, generator=gen)
    angle = R.angles(pos, freqs, (3, 5))
    a, b = (slice(0, 16, 2), slice(1, 16, 2)) if interleaved else (slice(0, 8), slice(8, 16))

    def f(x, w):
        n = x / (x.square().mean(-1, keepdim=True) + 1e-3).sqrt() * w
        z = torch.complex(n[..., a], n[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        pairs = torch.stack([z.real, z.imag], -1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
        return torch.cat([pairs, n[..., 16:]], -1)
    res = R.qknorm(x, w, pos, freqs, 1e-3, (3, 5), interleaved, dy)
    y = f(x, w)
    dx, dw = torch.autograd.grad((y * dy).sum(), (x, w))
    torch.testing.assert_close(res["y"][0], y.detach(), rtol=1e-10, atol=1e-10)
    torch.testing.assert_close(res["dx"][0], dx, rtol=1e-10, atol=1e-10)
    torch.testing.assert_close(res["dweight"][0], dw, rtol=1e-10, atol=1e-10)
    assert torch.autograd.gradcheck(f, (x, w))
