"""GPU tests of linear attention with a decay for each head and of the norm and
rotation of its queries and keys: each value against the 64-bit definition
within the bound of mixer_ref."""
import math

import pytest
import torch

import mixer_ref as R
from block_ref import assert_within, rounded
from selective_state_space_56_amd import (linear_attn_bwd, linear_attn_fwd, linear_attn_update, qk_norm_rope_bwd,
                                          qk_norm_rope_fwd)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(gn, *shape, io=F32):
    return torch.randn(shape, generator=gn, device="cuda").to(io)


def make(seed, lead, H, G, K, V, io, fixed=False, strided=False, states=0):
    gn = gen(seed)
    if strided:  # column slices of one projection's rows, at an odd first column
        rows = normal(gn, *lead, 2 * G * K + H * V + 13, io=io)
        q = rows[..., 3:3 + G * K].unflatten(-1, (G, K))
        k = rows[..., 3 + G * K:3 + 2 * G * K].unflatten(-1, (G, K))
        v = rows[..., 3 + 2 * G * K:3 + 2 * G * K + H * V].unflatten(-1, (H, V))
    else:
        q, k, v = normal(gn, *lead, G, K, io=io), normal(gn, *lead, G, K, io=io), normal(gn, *lead, H, V, io=io)
    rate = torch.exp(torch.rand(H, generator=gn, device="cuda") * 6.0 - 5.0)
    g = -rate if fixed else -rate * torch.rand(lead + (H,), generator=gn, device="cuda")
    s = {"q": q, "k": k, "v": v, "g": g, "dout": normal(gn, *lead, H, V, io=io)}
    if states:
        s["h0"], s["dlast"] = normal(gn, states, H, K, V), normal(gn, states, H, K, V)
    return s


def check(s, scale=None, offsets=None, backward=True, **kw):
    q, k, v, g, io = s["q"], s["k"], s["v"], s["g"], s["v"].dtype
    sc = q.shape[-1] ** -0.5 if scale is None else scale
    h0, dlast = s.get("h0"), s.get("dlast")
    out, last = linear_attn_fwd(q, k, v, g, scale=scale, h0=h0, offsets=offsets, **kw)
    d = linear_attn_bwd(q, k, v, g, s["dout"], scale=scale, h0=h0, offsets=offsets, dlast=dlast) if backward else {}
    torch.cuda.synchronize()
    off = None if offsets is None else offsets.cpu()
    ref = R.linattn(q, k, v, g, sc, h0, off, s["dout"] if backward else None, dlast)
    assert_within("out", out, rounded(ref["out"], io))
    assert_within("last_state", last, rounded(ref["last_state"], F32))
    if backward:
        for n in ("dq", "dk", "dv"):
            assert_within(n, d[n], rounded(ref[n], io))
        for n in ("dg", "dh0"):
            assert_within(n, d[n], rounded(ref[n], F32))
    return out, last, d


SIZES = [(8, 8), (32, 64), (64, 32), (128, 128), (40, 72), (136, 24), (24, 200), (256, 256)]


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("K,V", SIZES)
def test_sequences(K, V, io):
    check(make(K * 3 + V, (2, 150), 2, 2, K, V, io))
    check(make(K * 3 + V + 1, (1, 67), 3, 1, K, V, io, strided=True, states=1))


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191])
def test_lengths(L, io):
    check(make(L, (2, L), 2, 1, 64, 64, io, states=2))


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("fixed", [False, True])
def test_many_segments(fixed, io):
    # few heads and a long way: more than one workgroup for each sequence, and states
    # between stretches of 1024 steps
    check(make(5, (1, 2177), 2, 1, 64, 40, io, fixed=fixed, states=1))


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("fixed", [False, True])
def test_shared_heads(fixed, io):
    check(make(6, (2, 130), 6, 2, 32, 64, io, fixed=fixed, states=2))
    check(make(7, (1, 90), 5, 1, 128, 64, io, fixed=fixed))


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 5], [64, 64], [65, 1, 0, 130, 63], [1500, 3, 700, 0]])
def test_packed(lens, io):
    first, rest = 2, 5
    off = torch.tensor([first + sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda")
    n = int(off[-1]) + rest
    s = make(sum(lens) + len(lens), (n,), 2, 1, 64, 32, io, states=len(lens))
    out, _, d = check(s, offsets=off)
    for t in (out, d["dq"], d["dk"], d["dv"], d["dg"]):  # zeros in what the call has made
        assert not t[:first].any() and not t[n - rest:].any()


def test_packed_rest_is_left():
    off = torch.tensor([3, 70], device="cuda")
    s = make(11, (80,), 2, 2, 32, 32, BF)
    out = torch.full_like(s["v"], 7.0)
    given = {n: torch.full_like(s[n[1:]], 7.0) for n in ("dq", "dk", "dv")}
    linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], offsets=off, out=out)
    linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], offsets=off, **given)
    for t in (out, *given.values()):
        assert (t[:3] == 7).all() and (t[70:] == 7).all() and not (t[3:70] == 7).all()
    # one given, the others made: zeros in those
    d = linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], offsets=off, dq=given["dq"])
    assert (d["dq"][:3] == 7).all() and not d["dk"][:3].any() and not d["dv"][70:].any() and not d["dg"][70:].any()


def test_packed_equals_separate():
    lens = [100, 1, 333]
    off = torch.tensor([0, 100, 101, 434], device="cuda")
    s = make(12, (434,), 2, 2, 64, 64, BF, states=3)
    out, last = linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"], offsets=off)
    for i in range(len(lens)):
        a, b = int(off[i]), int(off[i + 1])
        one, end = linear_attn_fwd(s["q"][None, a:b], s["k"][None, a:b], s["v"][None, a:b],
                                   s["g"][None, a:b].contiguous(), h0=s["h0"][i:i + 1])
        assert torch.equal(one[0], out[a:b]) and torch.equal(end[0], last[i])


def test_offsets_out_of_range_are_held_to_the_rows():
    s = make(13, (50,), 2, 2, 32, 32, F32)
    bad = torch.tensor([-5, 20, 1 << 40], device="cuda")
    good = torch.tensor([0, 20, 50], device="cuda")
    args = (s["q"], s["k"], s["v"], s["g"])
    for x, y in zip(linear_attn_fwd(*args, offsets=bad), linear_attn_fwd(*args, offsets=good)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("io", [F32, BF])
def test_no_tokens(io):
    s = make(14, (2, 0), 2, 1, 16, 24, io, fixed=True, states=2)
    out, last = linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"])
    assert out.shape == (2, 0, 2, 24) and torch.equal(last, s["h0"])
    d = linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], h0=s["h0"], dlast=s["dlast"])
    assert torch.equal(d["dh0"], s["dlast"]) and not d["dg"].any()
    s = make(15, (0, 4), 2, 1, 16, 24, io)
    assert linear_attn_fwd(s["q"], s["k"], s["v"], s["g"])[1].shape == (0, 2, 16, 24)
    # packed, with rows but no sequence
    s = make(16, (9,), 2, 1, 16, 24, io)
    out, last = linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], offsets=torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert not out.any() and last.shape[0] == 0


@pytest.mark.parametrize("io", [F32, BF])
def test_decays_of_zero(io):
    s = make(17, (2, 150), 2, 1, 32, 40, io, states=2)
    g = s["g"]
    g[0, 70], g[0, 71, 0], g[1, 0], g[1, 149] = -math.inf, -104.0, torch.finfo(F32).min, -1e4
    g[1, 64] = -math.inf
    _, _, d = check(s)
    assert not d["dg"][0, 70].any() and not d["dg"][1, 0].any()


@pytest.mark.parametrize("io", [F32, BF])
def test_no_gradient_of_decays_before_what_is_cut_off(io):
    # nothing before token 100 reaches a gradient: what later ones have may not leave a rest
    s = make(18, (1, 150), 2, 1, 32, 40, io, states=1)
    s["dout"][:, :100] = 0
    s["g"][:, 100], s["g"][0, 120, 0] = -math.inf, -1e4
    _, _, d = check(s)
    assert not d["dg"][:, :101].any() and not d["dg"][0, 120, 0].any()
    assert d["dg"][:, 101:120].all() and d["dg"][:, 121:].all()


def clean_ref(s, h0=None):
    """Beside values that are not finite the other outputs keep to the bound of
    the inputs without them, not to the same bits: where an output of a tile is
    not finite its steps' terms are added one by one, the same terms in another
    order, which the bound (additions in any order) covers."""
    return R.linattn(s["q"], s["k"], s["v"], s["g"], s["q"].shape[-1] ** -0.5, h0)


@pytest.mark.parametrize("io", [F32, BF])
def test_what_a_cut_drops_may_be_anything(io):
    s = make(18, (1, 200), 2, 1, 32, 64, io, states=1)
    clean = {k: v.clone() for k, v in s.items()}
    cut = 90
    s["g"][0, cut] = clean["g"][0, cut] = -math.inf
    for n in "qkv":
        s[n][0, 80:cut] = math.nan
    s["v"][0, 3] = math.inf
    s["h0"][:] = math.nan
    out, last = linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"])
    ref = clean_ref(clean, clean["h0"])
    assert_within("out", out[:, cut:], tuple(x[:, cut:] for x in rounded(ref["out"], io)))
    assert_within("last_state", last, rounded(ref["last_state"], F32))
    assert out[0, 80:cut].isnan().all()
    # a decay of 0 in the first step drops h0
    s["g"][0, 0] = -200.0
    a = linear_attn_fwd(*(s[n][:, :3].contiguous() for n in "qkvg"), h0=s["h0"])
    assert a[0].isfinite().all()


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_later_tokens_do_not_reach_earlier_outputs(bad, io):
    s = make(19, (1, 160), 2, 2, 32, 64, io)
    ref = rounded(clean_ref(s)["out"], io)
    for at, n in ((1, "v"), (40, "k"), (63, "v"), (64, "v"), (100, "q")):
        x = {m: t.clone() for m, t in s.items()}
        x[n][0, at, 1, 5] = bad
        out, _ = linear_attn_fwd(x["q"], x["k"], x["v"], x["g"])
        assert_within(f"before {n} {at}", out[:, :at], tuple(t[:, :at] for t in ref))
        assert_within(f"other head {n} {at}", out[:, :, 0], tuple(t[:, :, 0] for t in ref))
        assert not out[0, at, 1].isfinite().all()
        if n == "v":  # one value channel
            keep = [c for c in range(64) if c != 5]
            assert_within(f"other channels {n} {at}", out[..., keep], tuple(t[..., keep] for t in ref))


def test_padding_behind_the_tokens_may_be_anything():
    # a batch whose shorter sequences are padded: what stands there reaches no other rows
    s = make(20, (2, 100), 2, 1, 64, 64, BF)
    ref = rounded(clean_ref(s)["out"], BF)
    for n in "qkv":
        s[n][1, 37:] = math.nan
    s["g"][1, 37:] = math.nan
    out, _ = linear_attn_fwd(s["q"], s["k"], s["v"], s["g"])
    assert_within("whole", out[0], tuple(t[0] for t in ref))
    assert_within("padded", out[1, :37], tuple(t[1, :37] for t in ref))


@pytest.mark.parametrize("io", [F32, BF])
def test_strong_and_growing_decays(io):
    s = make(21, (1, 140), 2, 1, 32, 32, io)
    s["g"][:, ::3] = -60.0   # sums of thousands beside small ones
    check(s)
    s["g"] = 0.02 * torch.rand_like(s["g"])   # the state grows
    check(s)


def test_gradients_are_optional():
    # without dg the state goes into the products in two parts instead of three: the same
    # values to the bound that holds for two (2^-17 of each term), not the same bits
    s = make(22, (2, 130), 4, 2, 64, 64, BF, states=2)
    some = linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], h0=s["h0"], dlast=s["dlast"], want_dg=False,
                           want_dh0=False)
    assert some["dg"] is None and some["dh0"] is None
    ref = R.linattn(s["q"], s["k"], s["v"], s["g"], 64 ** -0.5, s["h0"], None, s["dout"], s["dlast"])
    for n in ("dq", "dk", "dv"):
        assert_within(n, some[n], rounded(ref[n], BF))


def test_gradients_into_one_buffer():
    s = make(23, (2, 70), 2, 2, 32, 40, BF, strided=True)
    ref = linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"])
    rows = torch.full((2, 70, 2 * 64 + 80 + 5), 7.0, dtype=BF, device="cuda")
    into = {"dq": rows[..., :64].unflatten(-1, (2, 32)), "dk": rows[..., 64:128].unflatten(-1, (2, 32)),
            "dv": rows[..., 128:208].unflatten(-1, (2, 40))}
    linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["dout"], **into)
    for n, t in into.items():
        assert torch.equal(t, ref[n])
    assert (rows[..., 208:] == 7).all()


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("K,V", [(8, 8), (128, 128), (40, 72), (256, 256), (64, 24)])
@pytest.mark.parametrize("fixed", [False, True])
def test_update(K, V, fixed, io):
    for batch, H, G in ((1, 2, 2), (3, 4, 2), (700, 2, 1)):
        s = make(K + V + batch, (batch,), H, G, K, V, io, fixed=fixed, strided=batch == 3, states=batch)
        if not fixed:
            s["g"][0, 0] = -math.inf
        state, before = s["h0"].clone(), s["h0"]
        if not fixed:
            state[0, 0] = math.nan
        out = linear_attn_update(state, s["q"], s["k"], s["v"], s["g"], scale=0.25)
        ref = R.update(before, s["q"], s["k"], s["v"], s["g"], 0.25)
        assert_within("state", state, rounded(ref["state"], F32))
        assert_within("out", out, rounded(ref["out"], io))


@pytest.mark.parametrize("io", [F32, BF])
def test_prompt_then_tokens(io):
    # a prompt in pieces, then single tokens: the same as in one go
    s = make(24, (2, 90), 4, 2, 64, 32, io, states=2)
    cut = lambda a, b: [s[n][:, a:b].contiguous() for n in "qkvg"]  # noqa: E731
    whole, last = linear_attn_fwd(*cut(0, 90), h0=s["h0"])
    ref = R.linattn(*cut(0, 90), 64 ** -0.5, s["h0"])
    first, state = linear_attn_fwd(*cut(0, 70), h0=s["h0"])
    _, state = linear_attn_fwd(*cut(70, 80), h0=state)
    outs = [linear_attn_update(state, *(t[:, 0].contiguous() for t in cut(i, i + 1))) for i in range(80, 90)]
    assert_within("state", state, rounded(ref["last_state"], F32))
    v, e = rounded(ref["out"], io)
    assert_within("out", torch.stack(outs, 1), (v[:, 80:], e[:, 80:]))
    assert_within("first", first, (v[:, :70], e[:, :70]))


TURN = [  # tokens, hq, hk, D, rotary, sections, interleaved
    (1, 1, 1, 8, 8, None, False), (5, 3, 2, 64, 64, None, True), (33, 5, 1, 128, 64, None, False),
    (7, 40, 40, 128, 128, None, False), (130, 2, 0, 256, 256, None, False), (9, 6, 2, 80, 80, (14, 13, 13), True),
    (11, 3, 3, 40, 16, (1, 0, 3, 4), False), (4, 2, 2, 96, 0, None, False), (300, 4, 2, 72, 24, (5, 7), True)]


def turn_case(seed, n, hq, hk, D, rot, sections, io, strided=True, far=1 << 20):
    gn = gen(seed)
    rows = normal(gn, n, (hq + hk) * D + 5, io=io) * 2
    q, k = rows[:, 3:3 + hq * D].unflatten(1, (hq, D)), rows[:, 3 + hq * D:3 + (hq + hk) * D].unflatten(1, (hk, D))
    if not strided:
        q, k = q.contiguous(), k.contiguous()
    axes = (n,) if sections is None else (len(sections), n)
    pos = torch.randint(-far, far, axes, generator=gn, device="cuda")
    freqs = 10000.0 ** (-torch.arange(rot // 2, device="cuda") / max(1, rot // 2))
    wq, wk = 1 + normal(gn, D) * 0.2, 1 + normal(gn, D) * 0.2
    return q, (k if hk else None), pos, freqs, wq, wk, normal(gn, n, hq, D, io=io), normal(gn, n, hk, D, io=io) if hk else None


@pytest.mark.parametrize("io", [F32, BF])
@pytest.mark.parametrize("case", TURN)
@pytest.mark.parametrize("weights", [True, False])
def test_norm_and_rotation(case, weights, io):
    n, hq, hk, D, rot, sections, inter = case
    q, k, pos, freqs, wq, wk, dy, dz = turn_case(n + D, n, hq, hk, D, rot, sections, io, strided=n != 7)
    if not weights:
        wq = wk = None
    more = {"eps": 1e-5, "sections": sections, "interleaved": inter}
    y, z = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk, **more)
    d = qk_norm_rope_bwd(q, k, pos, freqs, wq, wk, dy, dz, **more)
    torch.cuda.synchronize()
    for x, w, g, out, name in ((q, wq, dy, y, "q"), (k, wk, dz, z, "k")):
        if x is None:
            assert out is None and d["dk"] is None
            continue
        ref = R.qknorm(x, w, pos, freqs, 1e-5, sections, inter, g)
        assert_within(name, out, rounded(ref["y"], io))
        assert_within("d" + name, d["d" + name], rounded(ref["dx"], io))
        if weights:
            assert_within("dw" + name, d[f"d{name}_weight"], rounded(ref["dweight"], F32))
        else:
            assert d[f"d{name}_weight"] is None
    if weights and hk == 0:
        assert not d["dk_weight"].any()


def test_norm_and_rotation_far_positions():
    q, k, pos, freqs, wq, wk, *_ = turn_case(1, 40, 2, 1, 64, 64, None, F32, far=1 << 28)
    y, _ = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk)
    assert_within("q", y, rounded(R.qknorm(q, wq, pos, freqs, 1e-6)["y"], F32))


def test_norm_and_rotation_of_many_tokens():
    # more tokens than workgroups at a time
    for io in (F32, BF):
        q, k, pos, freqs, wq, wk, dy, dz = turn_case(2, 9001, 2, 1, 32, 32, None, io)
        y, z = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk)
        d = qk_norm_rope_bwd(q, k, pos, freqs, wq, wk, dy, dz)
        for x, w, g, out, n in ((q, wq, dy, y, "q"), (k, wk, dz, z, "k")):
            ref = R.qknorm(x, w, pos, freqs, 1e-6, dy=g)
            assert_within(n, out, rounded(ref["y"], io))
            assert_within("d" + n, d["d" + n], rounded(ref["dx"], io))
            assert_within("dw" + n, d[f"d{n}_weight"], rounded(ref["dweight"], F32))


def test_norm_and_rotation_in_place():
    q, k, pos, freqs, wq, wk, dy, dz = turn_case(3, 50, 4, 2, 64, 32, None, BF)
    y, z = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk)
    d = qk_norm_rope_bwd(q, k, pos, freqs, wq, wk, dy, dz)
    a, b = dy.clone(), dz.clone()
    e = qk_norm_rope_bwd(q, k, pos, freqs, wq, wk, a, b, dq=a, dk=b)
    assert e["dq"] is a and torch.equal(a, d["dq"]) and torch.equal(b, d["dk"]) and torch.equal(e["dq_weight"], d["dq_weight"])
    got = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, y) and torch.equal(k, z)


def test_norm_and_rotation_rows_that_are_not_finite():
    q, k, pos, freqs, wq, wk, dy, dz = turn_case(4, 6, 2, 2, 64, 64, None, F32)
    y, _ = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk)
    q[2, 1, 3] = math.nan
    q[4, 0, 7] = math.inf
    x, _ = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk)
    d = qk_norm_rope_bwd(q, k, pos, freqs, wq, wk, dy, dz)
    assert x[2, 1].isnan().all() and x[4, 0].isnan().any() and d["dq"][2, 1].isnan().all()
    keep = torch.ones(6, 2, dtype=torch.bool)
    keep[2, 1] = keep[4, 0] = False
    assert torch.equal(x[keep], y[keep]) and d["dq"][keep].isfinite().all()


def test_norm_and_rotation_rows_of_zeros():
    q, k, pos, freqs, wq, wk, dy, dz = turn_case(5, 3, 2, 1, 40, 16, None, F32)
    q[1] = 0
    y, _ = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk)
    assert not y[1].any()
    # with eps 0, heads that do not exist are not heads of zeros
    d = qk_norm_rope_bwd(q[:1], k[:1], pos[:1], freqs, wq, wk, dy[:1], dz[:1], eps=0.0)
    assert d["dq_weight"].isfinite().all() and d["dk_weight"].isfinite().all()


@pytest.mark.parametrize("io", [F32, BF])
def test_norm_and_rotation_ends_of_the_range(io):
    q, k, pos, freqs, wq, wk, dy, dz = turn_case(6, 3, 2, 1, 40, 16, None, io)
    q[0, 0], q[1, 0], q[2, 0] = 0.0, 1e-24, 1e20
    y, _ = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk, eps=0.0)
    assert y[0, 0].isnan().all() and y[1, 0].isinf().any() and not y[2, 0].any()
    assert y[:, 1].isfinite().all()
    y, _ = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk)
    assert not y[0, 0].any() and y[1, 0].isfinite().all()


def layer(rows, pos, freqs, wq, wk, g, dims, offsets=None, h0=None):
    H, K, V = dims
    q, k = rows[..., :H * K].unflatten(-1, (H, K)), rows[..., H * K:2 * H * K].unflatten(-1, (H, K))
    v = rows[..., 2 * H * K:].unflatten(-1, (H, V))
    qn, kn = qk_norm_rope_fwd(q, k, pos, freqs, wq, wk)
    return q, k, v, qn, kn, linear_attn_fwd(qn, kn, v, g, offsets=offsets, h0=h0)


@pytest.mark.parametrize("io", [F32, BF])
def test_layer(io):
    """The operators as a layer uses them: a projection's rows of packed
    prompts, normed and turned, mixed, their gradients back into one row
    gradient, and a token that goes on from the states."""
    H, K, V = 4, 64, 32
    lens = [70, 5, 133]
    off = torch.tensor([0, 70, 75, 208], device="cuda")
    gn = gen(40)
    rows = normal(gn, 208, H * (2 * K + V), io=io)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    freqs = 10000.0 ** (-torch.arange(K // 2, device="cuda") / (K // 2))
    wq, wk = 1 + 0.1 * normal(gn, K), 1 + 0.1 * normal(gn, K)
    g = -torch.rand(208, H, generator=gn, device="cuda")
    q, k, v, qn, kn, (out, last) = layer(rows, pos, freqs, wq, wk, g, (H, K, V), off)
    ref = R.linattn(qn, kn, v, g, K ** -0.5, offsets=off.cpu())
    assert_within("out", out, rounded(ref["out"], io))
    dout = normal(gn, 208, H, V, io=io)
    drows = torch.zeros_like(rows)
    dq, dk = drows[:, :H * K].unflatten(1, (H, K)), drows[:, H * K:2 * H * K].unflatten(1, (H, K))
    d = linear_attn_bwd(qn, kn, v, g, dout, offsets=off, dq=dq, dk=dk, dv=drows[:, 2 * H * K:].unflatten(1, (H, V)))
    dqn, dkn = dq.clone(), dk.clone()
    e = qk_norm_rope_bwd(q, k, pos, freqs, wq, wk, dq, dk, dq=dq, dk=dk)
    rq = R.qknorm(q, wq, pos, freqs, 1e-6, dy=dqn)
    rk = R.qknorm(k, wk, pos, freqs, 1e-6, dy=dkn)
    assert_within("dq", drows[:, :H * K].unflatten(1, (H, K)), rounded(rq["dx"], io))
    assert_within("dk", drows[:, H * K:2 * H * K].unflatten(1, (H, K)), rounded(rk["dx"], io))
    assert_within("dwq", e["dq_weight"], rounded(rq["dweight"], F32))
    assert torch.equal(d["dv"], drows[:, 2 * H * K:].unflatten(1, (H, V)))
    # the next token of each sequence
    new = normal(gn, 3, H * (2 * K + V), io=io)
    at = torch.tensor(lens, device="cuda")
    q1, k1 = new[:, :H * K].unflatten(1, (H, K)), new[:, H * K:2 * H * K].unflatten(1, (H, K))
    v1 = new[:, 2 * H * K:].unflatten(1, (H, V))
    qn1, kn1 = qk_norm_rope_fwd(q1, k1, at, freqs, wq, wk)
    g1 = -torch.rand(3, H, generator=gn, device="cuda")
    before = last.clone()
    o1 = linear_attn_update(last, qn1, kn1, v1, g1)
    ref = R.update(before, qn1, kn1, v1, g1, K ** -0.5)
    assert_within("token", o1, rounded(ref["out"], io))
    assert_within("state", last, rounded(ref["state"], F32))
