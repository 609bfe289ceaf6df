"""GPU tests of the mixer operators on float32 tensors that lie at 4 bytes only:
contiguous views one element into a buffer give the same bits as tensors that
lie at the start of an allocation."""
import pytest
import torch

from selective_state_space_56_amd import (linear_attn_bwd, linear_attn_fwd, linear_attn_update, qk_norm_rope_bwd,
                                          qk_norm_rope_fwd)
from test_mixer_gpu import BF, F32, make, turn_case

pytestmark = pytest.mark.gpu


def odd(t):
    """t's values as a contiguous view one element into a buffer."""
    x = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape).copy_(t)
    assert x.is_contiguous() and x.data_ptr() % 16 == t.element_size()
    return x


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("lead,K,V,fixed", [((2, 70), 64, 64, False), ((1, 1300), 40, 72, True), ((1, 2100), 128, 128, False)])
def test_sequences(lead, K, V, fixed, io):
    s = make(K + V, lead, 2, 1, K, V, io, fixed=fixed, states=lead[0])
    t = {n: odd(x) for n, x in s.items()}
    for x, y in zip(linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"]),
                    linear_attn_fwd(t["q"], t["k"], t["v"], t["g"], h0=t["h0"], out=odd(torch.zeros_like(s["v"])),
                                    last_state=odd(torch.zeros_like(s["h0"])))):
        assert torch.equal(x, y)
    a = linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], h0=s["h0"], dlast=s["dlast"])
    b = linear_attn_bwd(t["q"], t["k"], t["v"], t["g"], t["dout"], h0=t["h0"], dlast=t["dlast"],
                        dq=odd(torch.zeros_like(s["q"])), dk=odd(torch.zeros_like(s["k"])), dv=odd(torch.zeros_like(s["v"])))
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("io", [F32, BF])
def test_update(io):
    s = make(3, (3,), 4, 2, 40, 24, io, states=3)
    t = {n: odd(x) for n, x in s.items()}
    x = linear_attn_update(s["h0"], s["q"], s["k"], s["v"], s["g"])
    y = linear_attn_update(t["h0"], t["q"], t["k"], t["v"], t["g"], out=odd(torch.zeros_like(s["v"])))
    assert torch.equal(x, y) and torch.equal(s["h0"], t["h0"])


@pytest.mark.parametrize("io", [F32, BF])
def test_norm_and_rotation(io):
    q, k, pos, freqs, wq, wk, dy, dz = turn_case(4, 50, 3, 2, 64, 32, None, io, strided=False)
    args = (q, k, pos, freqs, wq, wk)
    far = (odd(q), odd(k), odd(pos), odd(freqs), odd(wq), odd(wk))
    for x, y in zip(qk_norm_rope_fwd(*args), qk_norm_rope_fwd(*far, q_out=odd(q), k_out=odd(k))):
        assert torch.equal(x, y)
    a = qk_norm_rope_bwd(*args, dy, dz)
    b = qk_norm_rope_bwd(*far, odd(dy), odd(dz), dq=odd(q), dk=odd(k))
    for n in a:
        assert torch.equal(a[n], b[n]), n
