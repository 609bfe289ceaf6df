"""CPU tests of decay_ref: its values against automatic gradients, and that its
bound tells a right gradient of the decays from a wrong one at the sizes, masks and scales of the
GPU tests."""
import pytest
import torch

import decay_ref as D
from decay_cases import CASES, arguments, case

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("fixed", [False, True])
def test_values(fixed):
    gen = torch.Generator().manual_seed(1)

    def r(*s):
        return torch.randn(s, generator=gen, dtype=torch.float64)
    q, k, v, dout = r(2, 9, 2, 8), r(2, 9, 2, 8), r(2, 9, 4, 16), r(2, 9, 4, 16)
    h0, dlast = r(2, 4, 8, 16), r(2, 4, 8, 16)
    g = (-torch.rand((4,) if fixed else (2, 9, 4), generator=gen, dtype=torch.float64)).requires_grad_()
    S, loss = h0, 0.0
    pick = torch.arange(4) // 2
    for t in range(9):
        e = g.expand(2, 9, 4)[:, t].exp()[..., None, None]
        S = e * S + k[:, t, pick][..., None] * v[:, t][..., None, :]
        loss = loss + (0.3 * (q[:, t, pick][..., None] * S).sum(-2) * dout[:, t]).sum()
    want, = torch.autograd.grad(loss + (S * dlast).sum(), g)
    for chunk in (4, 32):
        parts = {}
        value, bound = D.dg(q, k, v, g.detach(), 0.3, dout, h0, dlast, chunk=chunk, parts=parts)
        torch.testing.assert_close(value, want, rtol=1e-11, atol=1e-11)
        torch.testing.assert_close(sum(parts.values()), want, rtol=1e-11, atol=1e-11)
        assert (bound > 0).all()


def outside(got, value, bound):
    return float(((got - value).abs() > bound).double().mean())


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("name", list(CASES))
def test_the_bound_tells_wrong_from_right(name, io):
    s, off = case(name, io, "cpu")
    parts = {}
    value, bound = D.dg(*arguments(s), offsets=off, parts=parts)
    some = value.abs() > 1e-24  # (below it the range of float32's factors bounds)
    assert some.any()

    def told(got):
        return outside(got[some], value[some], bound[some])
    few = 0.7 if s["g"].dim() == 1 else 0.8  # values near 0 may pass, whole tensors may not
    assert told(torch.zeros_like(value)) > few and told(-value) > few
    assert told(1.5 * value) > (0.4 if s["g"].dim() == 1 else 0.7) and told(value.roll(1, -1)) > 0.7
    for n, x in parts.items():  # a term left out, where it makes half of the value
        part = (x.abs() > value.abs() * 0.5) & some
        if int(part.sum()) >= 30:
            assert outside((value - x)[part], value[part], bound[part]) > 0.7, n
    assert told(value + 0.99 * bound) == 0.0


@pytest.mark.parametrize("name", ["late gradients", "a late burst", "strong steps"])
def test_a_product_carried_on_by_differences_is_outside(name):
    """What a float32 sum over other tokens leaves by cancellation does not pass: <S, dS> at the
    sequence's end less what crosses no longer, every term rounded to float32 and added in 64 bits."""
    s, off = case(name, F32, "cpu")
    value, bound = D.dg(*arguments(s), offsets=off)
    q, k, v, g, scale, dout = arguments(s)
    H = v.shape[2]
    zero = torch.zeros(H, q.shape[-1], v.shape[-1], dtype=torch.float64)
    x = [D._expand(D.d64(t)[0], H) for t in (q, k, v, dout)]
    gs = D.d64(g)[0]
    fwd = D.states(x[1], x[2], gs, zero, 1 << 20)
    bwd = D.states(scale * x[0], x[3], gs, zero, 1 << 20, reverse=True)
    got, rest = torch.zeros_like(value), torch.zeros(H, dtype=torch.float64)
    for t in range(len(fwd) - 1, -1, -1):
        S, dS = fwd[t][0], bwd[t][0]
        own = x[1][t][:, :, None] * x[2][t][:, None, :]
        after = gs[t].exp()[:, None, None] * S + own
        # + q . dq of this step - k . dk
        rest = rest + (scale * (x[0][t][:, :, None] * x[3][t][:, None, :] * after).sum((1, 2))).float().double()
        rest = rest - (dS * own).sum((1, 2)).float().double()
        got[0, t] = rest
    some = value.abs() > 1e-24
    assert outside(got[some], value[some], bound[some]) > 0.02
