"""Inputs for the tests of the decays' gradients, the same on the CPU and the GPU: sizes
of every class, packed sequences, and values that a sum over other tokens would drown."""
import torch

F32 = torch.float32


def _make(seed, lead, H, G, K, V, io, fixed=False, states=0):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape, io=F32):
        return torch.randn(shape, generator=gen).to(io)
    s = {"q": normal(*lead, G, K, io=io), "k": normal(*lead, G, K, io=io), "v": normal(*lead, H, V, io=io)}
    rate = torch.exp(torch.rand(H, generator=gen) * 6.0 - 5.0)
    s["g"] = -rate if fixed else -rate * torch.rand(lead + (H,), generator=gen)
    s["dout"] = normal(*lead, H, V, io=io)
    if states:
        s["h0"], s["dlast"] = normal(states, H, K, V), normal(states, H, K, V)
    return s


def _late(s):        # only the last outputs have a gradient, and the decays are strong
    s["g"].fill_(-1.0)
    s["dout"][:, :-32] = 0


def _burst(s):       # the last outputs' gradients are larger by far
    s["g"].fill_(-0.5)
    s["dout"][:, -64:] *= 1e6


def _strong(s):      # single strong steps among weak ones
    s["g"] *= 0.01
    s["g"][:, 17::64] = -20.0
    s["g"][:, 40::128] = -30.0
    s["g"][:, 100] = -90.0


def _small(s):       # keys grow along the sequence
    n = s["k"].shape[1]
    s["k"] *= torch.logspace(-6, 0, n)[:, None, None].to(s["k"].dtype)


def _padded(s):      # rows of zeros before the first token and behind the last
    for n in ("q", "k", "v", "dout"):
        s[n][:, :75] = 0
        s[n][:, -20:] = 0


def _cuts(s):
    s["g"][0, 70], s["g"][0, 71, 0], s["g"][1, 0], s["g"][1, 149] = float("-inf"), -104.0, torch.finfo(F32).min, -1e4
    s["g"][1, 64] = float("-inf")


def _grows(s):
    s["g"] *= -0.02


# name: (lead, H, G, K, V, fixed, states, lengths of packed sequences or None, what is done to the values)
CASES = {
    "128 x 128": ((2, 150), 2, 2, 128, 128, False, 0, None, None),
    "40 x 72, shared keys, states": ((1, 67), 3, 1, 40, 72, False, 1, None, None),
    "136 x 24": ((1, 150), 2, 1, 136, 24, False, 1, None, None),
    "24 x 200": ((1, 150), 2, 2, 24, 200, False, 1, None, None),
    "256 x 256": ((1, 67), 2, 1, 256, 256, False, 1, None, None),
    "200 x 136, several chunks": ((1, 330), 2, 1, 200, 136, False, 0, None, None),
    "long": ((1, 2177), 2, 1, 64, 40, False, 1, None, None),
    "long, one decay for each head": ((1, 450), 4, 2, 64, 40, True, 1, None, None),
    "one decay for each head": ((2, 130), 6, 2, 32, 64, True, 2, None, None),
    "one step": ((2, 1), 2, 1, 64, 64, False, 2, None, None),
    "33 steps": ((2, 33), 2, 1, 64, 64, False, 2, None, None),
    "65 steps": ((2, 65), 2, 1, 64, 64, False, 2, None, None),
    "packed": (None, 2, 1, 64, 32, False, 5, (65, 1, 0, 130, 63), None),
    "packed, long": (None, 2, 1, 16, 24, False, 5, (1030, 1024, 700, 0, 5), None),
    "packed, one decay for each head": (None, 2, 2, 32, 32, True, 3, (100, 1, 333), None),
    "late gradients": ((1, 512), 2, 2, 64, 64, False, 0, None, _late),
    "a late burst": ((1, 512), 2, 2, 64, 64, False, 0, None, _burst),
    "strong steps": ((1, 512), 2, 2, 64, 64, False, 0, None, _strong),
    "strong steps, states": ((1, 300), 2, 2, 128, 128, False, 1, None, _strong),
    "small keys first": ((1, 400), 2, 2, 64, 64, False, 0, None, _small),
    "padded rows": ((2, 200), 2, 2, 64, 64, False, 0, None, _padded),
    "cuts": ((2, 150), 2, 1, 32, 40, False, 2, None, _cuts),
    "growing": ((1, 140), 2, 1, 32, 32, False, 1, None, _grows),
}


def case(name, io, device):
    """(tensors by name, offsets or None)."""
    lead, H, G, K, V, fixed, states, lens, then = CASES[name]
    off = None
    if lens is not None:  # rows of no sequence on both sides
        off = torch.tensor([2 + sum(lens[:i]) for i in range(len(lens) + 1)], device=device)
        lead = (int(off[-1]) + 3,)
    s = _make(len(name) + K + V, lead, H, G, K, V, io, fixed, states)
    if then:
        then(s)
    return {n: t.to(device) for n, t in s.items()}, off


def arguments(s):
    """decay_ref.dg's."""
    return (*(s[n] for n in ("q", "k", "v", "g")), s["q"].shape[-1] ** -0.5, s["dout"],
            *((s["h0"], s["dlast"]) if "h0" in s else ()))
