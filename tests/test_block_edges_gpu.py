"""GPU tests of the block operators where single values decide: 8-bit values at
the borders of their roundings."""
import pytest
import torch

from selective_state_space_56_amd import rmsnorm_fwd, rmsnorm_quant_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", torch.cuda.current_device())


def _ties(n, g):
    """n values midway between two neighbouring e4m3 values, both normal and below."""
    e = torch.randint(-7, 9, (n,), generator=g)
    m = torch.randint(0, 8, (n,), generator=g)
    m = torch.where(e == 8, m % 6, m)                        # at most 432: 448 is the largest value
    normal = (8.0 + m + 0.5) / 8.0 * torch.exp2(e.float())
    return torch.where(e == -7, (m + 0.5) * 2.0 ** -9, normal)


@pytest.mark.parametrize("dim", [128, 2560, 8192, 20000])
@pytest.mark.parametrize("group", [0, 128])
def test_8_bit_values_are_the_rounded_quotient(dev, dim, group):
    """q is e4m3 of the float32 quotient y / scale by the scale that is returned,
    also where that lies at or next to the middle between two 8-bit values.

    y is what rmsnorm_fwd gives in float32 (the same sums and products). Its
    weights are chosen so that y lands within a few steps of such middles; the
    first channel of each group holds the largest value."""
    g = torch.Generator().manual_seed(dim + group)
    span = group or dim
    first = torch.arange(dim) % span == 0
    hits = 0
    for _ in range(4):
        x = torch.rand((1, dim), generator=g) * 0.5 + 0.5
        x[0, first] = 4.0
        x *= torch.where(torch.rand((1, dim), generator=g) < 0.5, -1.0, 1.0)
        n = rmsnorm_fwd(x.to(dev), torch.ones(dim, device=dev), eps=1e-5)[0].cpu()
        top = n[0, first].abs().repeat_interleave(span)[:dim]
        w = _ties(dim, g) * (top / 448.0) / n[0].abs()
        step = torch.randint(-2, 3, (dim,), generator=g).float()
        w = torch.where(first, torch.ones(dim), w * (1.0 + step * 2.0 ** -23))
        y = rmsnorm_fwd(x.to(dev), w.to(dev), eps=1e-5)[0].cpu()
        q, scale, _ = rmsnorm_quant_fwd(x.to(dev), w.to(dev), eps=1e-5, group=group)
        torch.cuda.synchronize()
        scale = scale.cpu()
        assert torch.equal(scale, y[:, first].abs() / 448.0)
        ratio = y / scale.repeat_interleave(span, 1)[:, :dim]
        want = ratio.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        hits += int((q.cpu().view(torch.uint8) != want.view(torch.uint8)).sum())
    assert hits == 0, f"{hits} of {4 * dim} values are not the rounded quotient"


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("size", [2.0 ** -99, 2.0 ** -60, 2.0 ** -45, 2.0 ** 70, 2.0 ** 108, 2.0 ** 120])
def test_8_bit_values_at_every_size(dev, size, group):
    """The same quotient for rows of weights near the ends of float32's range."""
    g = torch.Generator().manual_seed(7)
    dim = 1000
    x = torch.randn((5, dim), generator=g).to(dev)
    w = (torch.rand(dim, generator=g) + 0.5).to(dev) * size
    y = rmsnorm_fwd(x, w)[0].cpu()
    q, scale, _ = rmsnorm_quant_fwd(x, w, group=group)
    torch.cuda.synchronize()
    per = scale.cpu().repeat_interleave(group or dim, 1)[:, :dim]
    want = (y / per).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("group", [0, 128])
def test_8_bit_values_of_an_infinite_maximum(dev, group):
    """Where y itself is infinite, its scale is too: that value is NaN, the
    others of the scale's run are 0."""
    x = torch.ones((2, 300), device=dev)
    w = torch.ones(300, device=dev)
    w[7] = float("inf")
    q, scale, _ = rmsnorm_quant_fwd(x, w, group=group)
    torch.cuda.synchronize()
    f = q.float().cpu()
    assert bool(f[:, 7].isnan().all()) and bool((scale[:, 0] == float("inf")).all())
    run = f[:, :group or 300]
    assert int(run.isnan().sum()) == 2 and float(run.nan_to_num(0.0).abs().max()) == 0.0
    assert bool(f[:, 128:].isfinite().all())
