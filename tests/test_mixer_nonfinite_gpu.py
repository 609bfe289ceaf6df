"""GPU tests of linear attention on values that are not finite: they reach the outputs
and the states of later tokens however small the score or the decay between has become, until a
decay of 0 (g <= -104), and no others."""
import math

import pytest
import torch

import mixer_ref as R
from block_ref import assert_within, rounded
from selective_state_space_56_amd import linear_attn_bwd, linear_attn_fwd
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


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("lead", [(1, 200), (1, 1300)])  # (the longer one in segments)
@pytest.mark.parametrize("K,V", [(64, 64), (40, 136)])
def test_decays_that_only_underflow_drop_nothing(K, V, lead, io):
    s = make(61, lead, 2, 1, K, V, io, states=1)
    s["g"].fill_(-4.0)      # e^-128 over 32 steps: 0 in float32
    clean = {n: t.clone() for n, t in s.items()}
    s["v"][0, 3, 0, 5] = math.nan
    s["h0"][0, 1, 2, 7] = math.inf
    out, last = forward(s)
    assert not out[0, 3:, 0, 5].isfinite().any() and not last[0, 0, :, 5].isfinite().any()
    assert not out[0, :, 1, 7].isfinite().any() and not last[0, 1, 2, 7].isfinite()
    ref = R.linattn(*(clean[n] for n in "qkvg"), K ** -0.5, clean["h0"])
    for h, c in ((0, 5), (1, 7)):
        keep = [i for i in range(V) if i != c]
        assert_within("others", out[:, :, h, keep], tuple(x[:, :, h, keep] for x in rounded(ref["out"], io)))
        assert_within("states", last[:, h][..., keep], tuple(x[:, h][..., keep] for x in rounded(ref["last_state"], F32)))
    # and behind a decay of 0 everything is as without them
    for x in (s, clean):
        x["g"][0, 150] = -math.inf
    (out, last), ref = forward(s), R.linattn(*(clean[n] for n in "qkvg"), K ** -0.5, clean["h0"])
    assert_within("behind a cut", out[:, 150:], tuple(x[:, 150:] for x in rounded(ref["out"], io)))
    assert_within("last state", last, rounded(ref["last_state"], F32))


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("lead", [(1, 200), (1, 1300)])
def test_nor_do_they_in_the_gradients(lead, io):
    s = make(62, lead, 2, 1, 64, 64, io, states=1)
    s["g"].fill_(-4.0)
    s["dlast"][0, 1, 2, 7] = math.nan
    d = linear_attn_bwd(*(s[n] for n in "qkvg"), s["dout"], h0=s["h0"], dlast=s["dlast"])
    assert not d["dv"][0, :, 1, 7].isfinite().any() and not d["dk"][0, :, 0, 2].isfinite().any()
    assert not d["dh0"][0, 1, 2, 7].isfinite() and d["dh0"][0, 0].isfinite().all() and d["dv"][0, :, 0].isfinite().all()
    assert d["dq"].isfinite().all()


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_decay_that_is_not_a_number(bad, io):
    """Reaches its own and later tokens, segments behind it among them, and no earlier one."""
    s = make(63, (1, 1300), 2, 1, 64, 64, io, states=1)
    ref = R.linattn(*(s[n] for n in "qkvg"), 64 ** -0.5, s["h0"])
    s["g"][0, 100, 0] = bad
    out, last = forward(s)
    assert not out[0, 100:, 0].isfinite().any() and not last[0, 0].isfinite().any()
    assert_within("before", out[:, :100], tuple(x[:, :100] for x in rounded(ref["out"], io)))
    assert_within("other head", out[:, :, 1], tuple(x[:, :, 1] for x in rounded(ref["out"], io)))
