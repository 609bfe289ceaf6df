"""GPU tests of linear attention on values that are not finite: they reach the outputs
and the states of later tokens however small the score or the decay between has become, until a
decay of 0 (g <= -104), and no others."""
import math

import pytest
import torch

import mixer_ref as R
from block_ref import assert_within, rounded
from selective_state_space_56_amd import linear_attn_fwd
from test_mixer_gpu import BF, F32, make

pytestmark = pytest.mark.gpu


def forward(s):
    return linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], h0=s.get("h0"))


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("K,V", [(32, 64), (128, 128)])
def test_a_value_reaches_outputs_whose_score_underflows(K, V, sign, io):
    # 30 steps of a chunk, scores of +-1e-12 with decays down to e^-95
    s = make(60, (1, 30), 1, 1, K, V, io)
    at = 2
    s["g"].fill_(-3.5)
    s["q"].fill_(1.0)
    s["k"][0, at] = sign * 1e-12 / K
    clean = {n: t.clone() for n, t in s.items()}
    s["v"][0, at, 0, 5] = math.inf
    out, last = forward(s)
    assert not out[0, at:, 0, 5].isfinite().any() and not last[0, 0, :, 5].isfinite().any()
    ref = R.linattn(*(clean[n] for n in "qkvg"), K ** -0.5)
    keep = [c for c in range(V) if c != 5]
    assert_within("others", out[..., keep], tuple(x[..., keep] for x in rounded(ref["out"], io)))
    assert_within("before", out[:, :at], tuple(x[:, :at] for x in rounded(ref["out"], io)))
