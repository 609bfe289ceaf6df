"""The plain implementations that the block operators are tested against,
checked on the CPU: their gradients against differences of their values and
against automatic differentiation of separately written forms."""
import torch

import block_ref as ref


def _inputs(batch, L, dim, seed):
    g = torch.Generator().manual_seed(seed)
    n = [torch.randn((batch, L, dim), generator=g, dtype=torch.float64) for _ in range(4)]
    A = -0.01 - torch.rand(dim, generator=g, dtype=torch.float64)
    h0, dlast = (torch.randn((batch, dim), generator=g, dtype=torch.float64) for _ in range(2))
    reset = torch.rand((batch, L), generator=g) < 0.15
    return n, A, h0, dlast, reset


def test_gated_gradients_are_those_of_the_recurrence():
    (x, r, g, dout), A, h0, dlast, reset = _inputs(2, 23, 5, 1)
    leaves = [t.clone().requires_grad_() for t in (x, r, g, A, h0)]
    xx, rr, gg, AA, h = leaves
    loss = 0.0
    for t in range(x.shape[1]):
        a = torch.exp(AA * torch.sigmoid(rr[:, t]))
        fresh = torch.sigmoid(gg[:, t]) * xx[:, t]
        h = torch.where(reset[:, t, None], fresh, a * h + torch.sqrt(1 - a * a) * fresh)
        loss = loss + (h * dout[:, t]).sum()
    loss = loss + (h * dlast).sum()
    want = torch.autograd.grad(loss, leaves)
    got = ref.gated(x, r, g, A, h0, reset, dout, dlast)
    for name, w in zip(("dx", "dr", "dg", "dA", "dh0"), want):
        torch.testing.assert_close(got[name][0], w, rtol=1e-10, atol=1e-11)


def test_gated_gradients_are_differences():
    (x, r, g, dout), A, h0, dlast, reset = _inputs(1, 7, 3, 2)

    def loss(x, r, g, A, h0):
        v = ref.gated(x, r, g, A, h0, reset)
        return float((v["out"][0] * dout).sum() + (v["last_state"][0] * dlast).sum())

    got = ref.gated(x, r, g, A, h0, reset, dout, dlast)
    base, step = [x, r, g, A, h0], 1e-6
    for i, name in enumerate(("dx", "dr", "dg", "dA", "dh0")):
        for at in range(base[i].numel()):
            ends = []
            for s in (step, -step):
                moved = [t.clone() for t in base]
                moved[i].view(-1)[at] += s
                ends.append(loss(*moved))
            d = (ends[0] - ends[1]) / (2 * step)
            assert abs(d - float(got[name][0].reshape(-1)[at])) <= 1e-7 * (1 + abs(d)), (name, at)


def test_norm_gradients_are_those_of_the_norm():
    g = torch.Generator().manual_seed(3)
    s = torch.randn((6, 11), generator=g).requires_grad_()
    w = torch.randn(11, generator=g).requires_grad_()
    dout, ds = torch.randn((6, 11), generator=g), torch.randn((6, 11), generator=g)
    s64, w64 = s.double(), w.double()
    y = s64 / torch.sqrt(s64.square().mean(-1, keepdim=True) + 1e-5) * w64
    want = torch.autograd.grad((y * dout).sum() + (s64 * ds).sum(), [s64, w64])
    got = ref.norm(s, w, None, 1e-5, dout, ds)
    torch.testing.assert_close(got["out"][0], y.detach(), rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(got["dresidual"][0], want[0], rtol=1e-10, atol=1e-11)
    torch.testing.assert_close(got["dweight"][0], want[1], rtol=1e-10, atol=1e-11)


def test_conv_gradients_are_those_of_the_convolution():
    g = torch.Generator().manual_seed(4)
    for W, L in [(1, 5), (2, 6), (3, 1), (4, 9), (4, 2)]:
        x = torch.randn((2, L, 3), generator=g, dtype=torch.float64).requires_grad_()
        st = torch.randn((2, 3, W - 1), generator=g, dtype=torch.float64).requires_grad_()
        w = torch.randn((3, W), generator=g, dtype=torch.float64).requires_grad_()
        b = torch.randn(3, generator=g, dtype=torch.float64).requires_grad_()
        dout = torch.randn((2, L, 3), generator=g, dtype=torch.float64)
        dst = torch.randn((2, 3, W - 1), generator=g, dtype=torch.float64)
        seen = torch.cat([st.transpose(1, 2), x], 1)
        v = torch.nn.functional.conv1d(seen.transpose(1, 2), w[:, None], b, groups=3).transpose(1, 2)
        loss = (torch.nn.functional.silu(v) * dout).sum() + (seen[:, L:].transpose(1, 2) * dst).sum()
        want = torch.autograd.grad(loss, [x, w, b, st])
        got = ref.conv_bwd(x, w, dout, b, st, dst)
        for name, t in zip(("dxin", "dweight", "dbias", "dstate_in"), want):
            torch.testing.assert_close(got[name][0], t, rtol=1e-10, atol=1e-11)
