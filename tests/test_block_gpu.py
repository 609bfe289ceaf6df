"""GPU tests of the block operators (gated linear recurrence, RMS norm with
residual, convolution backward) against plain implementations in 64 bits.
Every value has its own bound, from the float32 operations that make it
(block_ref.py)."""
import pytest
import torch

import block_ref as ref
from block_ref import assert_within, rounded
from gpu_common import TOL, norm_err
from selective_state_space_56_amd import (conv1d_bwd, conv1d_fwd, conv1d_update, gated_scan_bwd, gated_scan_fwd,
                                          gated_update, rmsnorm_bwd, rmsnorm_fwd, rmsnorm_quant_fwd)
from selective_state_space_56_amd.block import CHECKPOINT

pytestmark = pytest.mark.gpu
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", torch.cuda.current_device())


def _gated_inputs(dev, batch, L, dim, io, halves=False, resets=0.0, seed=0):
    g = torch.Generator().manual_seed(1000 * L + dim + seed)

    def normal(*shape):
        return torch.randn(shape, generator=g)

    x = normal(batch, L, dim).to(io).to(dev)
    gates = normal(batch, L, 2 * dim).to(io).to(dev)
    r, i = gates[..., :dim], gates[..., dim:]
    if not halves:
        r, i = r.contiguous(), i.contiguous()
    A = (8.0 * torch.log(0.9 + 0.099 * torch.rand(dim, generator=g))).to(dev)
    reset = (torch.rand((batch, L), generator=g) < resets).to(dev) if resets else None
    return {"x": x, "r": r, "g": i, "A": A, "reset": reset, "h0": normal(batch, dim).to(dev),
            "dout": normal(batch, L, dim).to(io).to(dev), "dlast": normal(batch, dim).to(dev)}


def _check_gated(v, io, with_h0=True):
    h0, dlast = (v["h0"], v["dlast"]) if with_h0 else (None, None)
    out, last, marks = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], h0=h0, reset=v["reset"], return_checkpoints=True)
    d = gated_scan_bwd(v["x"], v["r"], v["g"], v["A"], v["dout"], marks, reset=v["reset"], dlast=dlast)
    torch.cuda.synchronize()
    want = ref.gated(v["x"], v["r"], v["g"], v["A"], h0, v["reset"], v["dout"], dlast)
    assert_within("out", out, rounded(want["out"], io))
    assert_within("last_state", last, rounded(want["last_state"], torch.float32))
    before = tuple(t[:, ::CHECKPOINT] for t in want["before"])
    assert_within("checkpoints", marks, rounded(before, torch.float32))
    for name in ("dx", "dr", "dg"):
        assert_within(name, d[name], rounded(want[name], io))
    for name in ("dA", "dh0"):
        assert_within(name, d[name], rounded(want[name], torch.float32))
    return out, last, marks, d


@pytest.mark.parametrize("batch,L,dim,io,halves,h0,resets", [
    (1, 1, 1, "bf16", False, True, 0.0),
    (2, 2, 3, "f32", True, True, 0.0),
    (3, 5, 64, "bf16", True, False, 0.3),
    (1, 16, 130, "bf16", False, True, 0.0),
    (2, 63, 65, "f32", True, True, 0.05),
    (1, 127, 128, "bf16", False, False, 0.0),
    (2, 128, 200, "bf16", True, True, 0.02),
    (2, 129, 256, "f32", False, True, 0.02),
    (1, 257, 771, "bf16", True, True, 0.01),
    (5, 300, 66, "f32", True, False, 0.0),
    (1, 1000, 127, "bf16", False, True, 0.0),
    (3, 1021, 71, "f32", False, True, 0.01),
    (2, 2049, 192, "bf16", True, True, 0.002),
    (1, 4500, 130, "bf16", True, False, 0.0),
    (1, 9001, 20, "f32", False, True, 0.001),
    (70, 40, 24, "bf16", True, True, 0.0),
])
def test_gated_vs_64_bits(dev, batch, L, dim, io, halves, h0, resets):
    print(f"gated {batch}x{L}x{dim} {io}", flush=True)
    _check_gated(_gated_inputs(dev, batch, L, dim, IO[io], halves, resets), IO[io], h0)


@pytest.mark.parametrize("L", [1, 130, 400])
@pytest.mark.parametrize("where", ["first", "last", "all", "none", "checkpoints"])
def test_gated_resets(dev, L, where):
    """Resets at the ends, at every step, on none, and right at the spans' edges."""
    v = _gated_inputs(dev, 2, L, 96, torch.float32)
    reset = torch.zeros((2, L), dtype=torch.uint8, device=dev)
    if where == "first":
        reset[:, 0] = 1
    elif where == "last":
        reset[0, -1] = 255
    elif where == "all":
        reset[:] = 1
    elif where == "checkpoints":
        reset[:, ::64] = 1
        reset[1, 63::64] = 1
    v["reset"] = reset
    _check_gated(v, torch.float32)


def test_gated_pieces(dev):
    """Pieces chained through the state are one sequence, and so are tokens."""
    v = _gated_inputs(dev, 2, 333, 70, torch.float32)
    want = ref.gated(v["x"], v["r"], v["g"], v["A"], v["h0"])
    h, outs = v["h0"], []
    for a, b in [(0, 1), (1, 140), (140, 140), (140, 300)]:
        o, h = gated_scan_fwd(v["x"][:, a:b].contiguous(), v["r"][:, a:b].contiguous(), v["g"][:, a:b].contiguous(),
                              v["A"], h0=h)
        outs.append(o)
    h = h.clone()
    for t in range(300, 333):
        outs.append(gated_update(h, v["x"][:, t].contiguous(), v["r"][:, t].contiguous(), v["g"][:, t].contiguous(),
                                 v["A"])[:, None])
    torch.cuda.synchronize()
    assert_within("out", torch.cat(outs, 1), rounded(want["out"], torch.float32))
    assert_within("state", h, rounded(want["last_state"], torch.float32))


@pytest.mark.parametrize("batch,dim,io,strided", [(1, 1, "f32", False), (1, 5120, "bf16", False), (3, 77, "bf16", True),
                                                  (130, 64, "bf16", True), (33, 100, "f32", True),
                                                  (1025, 129, "bf16", False)])
def test_gated_update(dev, batch, dim, io, strided):
    g = torch.Generator().manual_seed(batch + dim)
    wide = torch.randn((batch, 3 * dim + 1), generator=g).to(IO[io]).to(dev)
    x, r, i = wide[:, :dim], wide[:, dim:2 * dim], wide[:, 2 * dim:3 * dim]
    if not strided:
        x, r, i = x.contiguous(), r.contiguous(), i.contiguous()
    A = -torch.rand(dim, generator=g).to(dev)
    state = torch.randn((batch, dim), generator=g).to(dev)
    want = ref.gated(x[:, None], r[:, None], i[:, None], A, state)
    room = torch.full((batch, dim + 5), 7.0, dtype=IO[io], device=dev)
    out = gated_update(state, x, r, i, A, out=room[:, 2:dim + 2] if strided else None)
    torch.cuda.synchronize()
    assert_within("out", out, rounded((want["out"][0][:, 0], want["out"][1][:, 0]), IO[io]))
    assert_within("state", state, rounded(want["last_state"], torch.float32))
    if strided:
        assert bool((room[:, :2] == 7).all()) and bool((room[:, dim + 2:] == 7).all())


@pytest.mark.parametrize("io,dim", [("bf16", 33), ("bf16", 128), ("f32", 65)])
def test_gated_strided_outputs_touch_only_their_columns(dev, io, dim):
    v = _gated_inputs(dev, 2, 150, dim, IO[io], halves=True, resets=0.02)
    wide = torch.full((2, 150, 4 * dim + 3), 5.0, dtype=IO[io], device=dev)
    cols = [wide[..., 1 + k * dim:1 + (k + 1) * dim] for k in range(4)]
    _, last, marks = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], reset=v["reset"], out=cols[0], return_checkpoints=True)
    d = gated_scan_bwd(v["x"], v["r"], v["g"], v["A"], v["dout"], marks, reset=v["reset"], dx=cols[1], dr=cols[2],
                       dg=cols[3])
    torch.cuda.synchronize()
    want = ref.gated(v["x"], v["r"], v["g"], v["A"], None, v["reset"], v["dout"])
    for name, t in zip(("out", "dx", "dr", "dg"), cols):
        assert_within(name, t, rounded(want[name], IO[io]))
    assert bool((wide[..., 0] == 5).all()) and bool((wide[..., 4 * dim + 1:] == 5).all())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gated_at_the_gates_limits(dev, io):
    """Gates at +-infinity and decays of exactly 1 are limits, not NaN: closed
    recurrence gates and A = 0 hold the state, and their gradients are 0."""
    v = _gated_inputs(dev, 2, 300, 40, IO[io])
    v["r"][:, 10:200, 0] = -INF
    v["r"][:, ::3, 1] = INF
    v["g"][:, 20:60, 2] = -INF
    v["g"][:, ::2, 3] = INF
    v["A"][4] = 0.0
    out, last, marks = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], h0=v["h0"], return_checkpoints=True)
    d = gated_scan_bwd(v["x"], v["r"], v["g"], v["A"], v["dout"], marks, dlast=v["dlast"])
    torch.cuda.synchronize()
    want = ref.gated(v["x"], v["r"], v["g"], v["A"], v["h0"], None, v["dout"], v["dlast"])
    assert_within("out", out, rounded(want["out"], IO[io]))
    # held to rounding: where pieces of the sequence join, the state is A h + B
    # with the piece's map, two roundings away from the step-by-step one, and at
    # most 200 / 8 joins lie between
    torch.testing.assert_close(out[:, 10:200, 0].float(), out[:, 9:10, 0].float().expand(-1, 190),
                               rtol=50 * ref.U + (2 * ref.HALF[torch.bfloat16] if io == "bf16" else 0), atol=0)
    assert bool((out[:, :, 4] == v["h0"][:, None, 4].to(IO[io])).all())
    for t in list(d.values()):
        assert bool(torch.isfinite(t).all())
    for name in ("dx", "dr", "dg"):
        assert_within(name, d[name], rounded(want[name], IO[io]))
    assert float(d["dr"][:, 10:200, 0].abs().max()) == 0.0


@pytest.mark.parametrize("L,at", [(40, 3), (700, 130), (700, 255)])
def test_gated_non_finite_values_stay_in_their_channel_and_sequence(dev, L, at):
    """A NaN input makes its own channel NaN from there to the next reset; an
    infinite one stays infinite; a reset drops either."""
    v = _gated_inputs(dev, 2, L, 70, torch.float32)
    clean, _ = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], h0=v["h0"])
    stop = at + (L - at) // 2
    x = v["x"].clone()
    x[0, at, 5], x[1, at, 6] = NAN, INF
    reset = torch.zeros((2, L), dtype=torch.bool, device=dev)
    reset[:, stop] = True
    out, last = gated_scan_fwd(x, v["r"], v["g"], v["A"], h0=v["h0"], reset=reset)
    base, blast = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], h0=v["h0"], reset=reset)
    torch.cuda.synchronize()
    assert bool(out[0, at:stop, 5].isnan().all())
    assert bool((out[1, at:stop, 6] == INF).all())
    mask = torch.ones_like(out, dtype=torch.bool)
    mask[0, at:stop, 5] = mask[1, at:stop, 6] = False
    assert torch.equal(out[mask], base[mask])
    assert torch.equal(last, blast)
    assert bool(torch.isfinite(clean).all())
    bad = v["h0"].clone()
    bad[0, 1], bad[1, 2] = NAN, -INF
    first = torch.zeros_like(reset)
    first[:, 0] = True
    a, la = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], h0=bad, reset=first)
    assert bool(torch.isfinite(a).all()) and bool(torch.isfinite(la).all())
    a, la = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], h0=bad)
    torch.cuda.synchronize()
    assert bool(a[0, :, 1].isnan().all()) and bool((a[1, :, 2] == -INF).all())
    assert bool(la[0, 1].isnan()) and float(la[1, 2]) == -INF


def test_gated_empty(dev):
    A = -torch.ones(8, device=dev)
    z = torch.empty((2, 0, 8), device=dev)
    h0, dl = torch.randn((2, 8), device=dev), torch.randn((2, 8), device=dev)
    out, last, marks = gated_scan_fwd(z, z, z, A, h0=h0, return_checkpoints=True)
    assert out.shape == z.shape and torch.equal(last, h0) and marks.shape == (2, 0, 8)
    assert torch.equal(gated_scan_fwd(z, z, z, A)[1], torch.zeros_like(h0))
    d = gated_scan_bwd(z, z, z, A, z, marks, dlast=dl)
    assert torch.equal(d["dh0"], dl) and float(d["dA"].abs().max()) == 0.0
    d = gated_scan_bwd(z[:0], z[:0], z[:0], A, z[:0], marks[:0])
    assert float(d["dA"].abs().max()) == 0.0
    e = torch.empty((0, 8), device=dev)
    assert gated_update(e.clone(), e, e, e, A).shape == (0, 8)


def test_gated_is_deterministic(dev):
    v = _gated_inputs(dev, 3, 3000, 200, torch.bfloat16, resets=0.001)
    first = None
    for _ in range(4):
        out, last, marks = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], reset=v["reset"], return_checkpoints=True)
        d = gated_scan_bwd(v["x"], v["r"], v["g"], v["A"], v["dout"], marks, reset=v["reset"])
        now = [out, last, marks] + [d[k] for k in ("dx", "dr", "dg", "dA", "dh0")]
        torch.cuda.synchronize()
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def _norm_inputs(dev, rows, dim, io, res, seed=0):
    g = torch.Generator().manual_seed(rows * 7 + dim + seed)

    def normal(dtype, scale=1.0):
        return (torch.randn((rows, dim), generator=g) * scale).to(dtype).to(dev)

    w = (1.0 + 0.1 * torch.randn(dim, generator=g)).to(dev)
    stream = io if res is None else res
    return normal(io), None if res is None else normal(res, 2.0), w, normal(io), normal(stream)


NORM = [(1, 1, "f32", None), (3, 7, "bf16", None), (1, 64, "bf16", "bf16"), (5, 129, "bf16", "f32"),
        (257, 128, "f32", "f32"), (2, 511, "bf16", "bf16"), (600, 1541, "f32", "f32"), (37, 2560, "bf16", "f32"),
        (300, 2560, "bf16", "bf16"), (3, 8192, "bf16", "f32"), (2, 8197, "f32", None), (2, 20000, "bf16", "bf16"),
        (1, 65536, "bf16", "f32"), (1, 65533, "f32", "f32")]


@pytest.mark.parametrize("rows,dim,io,res", NORM)
def test_norm_vs_64_bits(dev, rows, dim, io, res):
    print(f"norm {rows}x{dim} {io} {res}", flush=True)
    x, residual, w, dout, ds = _norm_inputs(dev, rows, dim, IO[io], IO.get(res))
    y, total = rmsnorm_fwd(x, w, residual, eps=1e-5)
    stream = x if residual is None else total
    want = ref.norm(x, w, residual, 1e-5, dout, ds)
    torch.cuda.synchronize()
    assert torch.equal(stream.cpu(), want["sum"])
    assert_within("out", y, rounded(want["out"], IO[io]))
    d = rmsnorm_bwd(stream, w, dout, ds=ds, eps=1e-5)
    torch.cuda.synchronize()
    assert_within("dresidual", d["dresidual"], rounded(want["dresidual"], stream.dtype))
    assert_within("dx", d["dx"], rounded(want["dresidual"], IO[io]))
    assert_within("dweight", d["dweight"], rounded(want["dweight"], torch.float32))
    d = rmsnorm_bwd(stream, w, dout, eps=1e-5)
    want = ref.norm(x, w, residual, 1e-5, dout)
    assert_within("dresidual without ds", d["dresidual"], rounded(want["dresidual"], stream.dtype))


def _check_quant(q, scale, want, group):
    """Scales, and values within half an e4m3 step (2^-4 of the value, 2^-10 below the normal range) of y / scale."""
    (y, e), dim = want["out"], want["out"][0].shape[1]
    span = group or dim
    n = -(-dim // span)
    pad = torch.nn.functional.pad(y.abs(), (0, n * span - dim)).view(y.shape[0], n, span)
    epad = torch.nn.functional.pad(e, (0, n * span - dim)).view(y.shape[0], n, span)
    s = pad.amax(-1).clamp(min=2.0 ** -100) / 448
    assert_within("scale", scale, (s, epad.amax(-1) / 448 + 3 * ref.U * s))
    per = scale.cpu().double().repeat_interleave(span, 1)[:, :dim]
    v = q.float().cpu().double() * per
    off = (v - y).abs()
    allowed = torch.maximum(y.abs() * 2.0 ** -4, per * 2.0 ** -10) * (1 + 8 * ref.U) + 2 * e + 4 * ref.U * y.abs()
    assert bool((off <= allowed).all()), float((off - allowed).max())


@pytest.mark.parametrize("rows,dim,io,res", NORM)
@pytest.mark.parametrize("group", [0, 128])
def test_norm_quant(dev, rows, dim, io, res, group):
    x, residual, w, _, _ = _norm_inputs(dev, rows, dim, IO[io], IO.get(res), seed=1)
    q, scale, total = rmsnorm_quant_fwd(x, w, residual, eps=1e-5, group=group)
    torch.cuda.synchronize()
    want = ref.norm(x, w, residual, 1e-5)
    if residual is not None:
        assert torch.equal(total.cpu(), want["sum"])
    assert q.dtype == torch.float8_e4m3fn and scale.shape == (rows, -(-dim // group) if group else 1)
    _check_quant(q, scale, want, group)


@pytest.mark.parametrize("group", [0, 128])
def test_norm_of_zeros_and_non_finite_rows(dev, group):
    x, _, w, _, _ = _norm_inputs(dev, 6, 300, torch.float32, None)
    x[1] = 0.0
    x[2, 5] = NAN
    x[3, 7] = INF
    x[4] *= 1e-30
    y, _ = rmsnorm_fwd(x, w)
    q, scale, _ = rmsnorm_quant_fwd(x, w, group=group)
    torch.cuda.synchronize()
    f = q.float()
    assert float(y[1].abs().max()) == 0.0 and float(f[1].abs().max()) == 0.0
    assert bool((scale[1] == torch.tensor(2.0 ** -100 / 448)).all())
    assert bool(y[2].isnan().all()) and bool(f[2].isnan().all())
    assert bool(y[3, 7].isnan()) and float(y[3].nan_to_num(0.0).abs().max()) == 0.0 and int(y[3].isnan().sum()) == 1
    assert int(f[3].isnan().sum()) == 1
    keep = [0, 4, 5]
    want = ref.norm(x[keep], w, None, 1e-6)
    assert_within("others", y[keep], rounded(want["out"], torch.float32))
    _check_quant(q[keep], scale[keep], want, group)


@pytest.mark.parametrize("dim", [128, 131])
def test_norm_strides_and_in_place(dev, dim):
    """Rows as column slices, the stream and its gradient updated in place,
    neighbouring columns left alone."""
    x, residual, w, dout, ds = _norm_inputs(dev, 19, dim, torch.bfloat16, torch.float32)
    wide = torch.full((19, 3 * dim + 5), 3.0, dtype=torch.bfloat16, device=dev)
    wide[:, 1:dim + 1] = x
    want = ref.norm(x, w, residual, 1e-6, dout, ds)
    room = torch.full((19, dim + 4), 9.0, device=dev)
    room[:, 3:dim + 3] = residual
    stream = room[:, 3:dim + 3]
    y, total = rmsnorm_fwd(wide[:, 1:dim + 1], w, stream, out=wide[:, dim + 1:2 * dim + 1], sum=stream)
    torch.cuda.synchronize()
    assert total.data_ptr() == stream.data_ptr() and torch.equal(stream.cpu(), want["sum"])
    assert_within("out", y, rounded(want["out"], torch.bfloat16))
    assert bool((wide[:, 2 * dim + 1:] == 3).all()) and bool((wide[:, 0] == 3).all())
    assert bool((room[:, :3] == 9).all()) and bool((room[:, dim + 3:] == 9).all())
    grad = ds.clone()
    d = rmsnorm_bwd(stream, w, dout, ds=grad, dresidual=grad)
    torch.cuda.synchronize()
    assert_within("ds in place", grad, rounded(want["dresidual"], torch.float32))
    assert_within("dx", d["dx"], rounded(want["dresidual"], torch.bfloat16))
    q8 = torch.zeros((19, dim + 9), dtype=torch.uint8, device=dev)
    view = q8.view(torch.float8_e4m3fn)[:, 5:dim + 5]
    _, scale, _ = rmsnorm_quant_fwd(x, w, residual, out=view, group=128)
    torch.cuda.synchronize()
    _check_quant(view, scale, want, 128)
    assert int(q8[:, :5].sum()) == 0 and int(q8[:, dim + 5:].sum()) == 0


def test_norm_no_rows(dev):
    x, w = torch.empty((0, 96), device=dev), torch.ones(96, device=dev)
    assert rmsnorm_fwd(x, w)[0].shape == (0, 96)
    q, scale, _ = rmsnorm_quant_fwd(x, w, group=128)
    assert q.shape == (0, 96) and scale.shape == (0, 1)
    d = rmsnorm_bwd(x, w, x)
    torch.cuda.synchronize()
    assert float(d["dweight"].abs().max()) == 0.0


@pytest.mark.parametrize("batch,L,dim,width,io,state", [
    (1, 1, 1, 4, "f32", True), (2, 2, 5, 4, "bf16", True), (1, 3, 64, 4, "f32", True), (2, 5, 33, 3, "bf16", False),
    (1, 7, 20, 2, "f32", True), (2, 9, 70, 1, "bf16", False), (2, 64, 256, 4, "bf16", True),
    (3, 65, 37, 4, "bf16", True), (1, 127, 130, 3, "f32", True), (2, 200, 129, 4, "bf16", False),
    (1, 300, 771, 3, "f32", True), (2, 517, 96, 2, "bf16", True), (1, 1000, 512, 4, "bf16", True),
])
def test_conv_bwd_vs_64_bits(dev, batch, L, dim, width, io, state):
    print(f"conv bwd {batch}x{L}x{dim} W={width} {io}", flush=True)
    g = torch.Generator().manual_seed(L + dim)

    def normal(*shape, to=torch.float32):
        return torch.randn(shape, generator=g).to(to).to(dev)

    x, dout = normal(batch, L, dim, to=IO[io]), normal(batch, L, dim, to=IO[io])
    w, b = normal(dim, width) * 0.5, normal(dim) * 0.5
    st = normal(batch, dim, width - 1, to=IO[io]) if state else None
    dst = normal(batch, dim, width - 1) if state else None
    for bias in (b, None):
        d = conv1d_bwd(x, w, dout, bias, st, dstate_out=dst)
        torch.cuda.synchronize()
        want = ref.conv_bwd(x, w, dout, bias, st, dst)
        assert_within("dxin", d["dxin"], rounded(want["dxin"], IO[io]))
        for name in ("dweight", "dbias", "dstate_in"):
            assert_within(name, d[name], rounded(want[name], torch.float32))


def test_conv_bwd_empty_and_pieces(dev):
    w, b = torch.randn((16, 4), device=dev), torch.randn(16, device=dev)
    dst = torch.randn((2, 16, 3), device=dev)
    e = torch.empty((2, 0, 16), device=dev)
    d = conv1d_bwd(e, w, e, b, None, dstate_out=dst)
    torch.cuda.synchronize()
    assert torch.equal(d["dstate_in"], dst) and float(d["dweight"].abs().max()) == 0.0 == float(d["dbias"].abs().max())
    # two pieces, the second one's state gradient handed to the first
    x, dout = torch.randn((2, 150, 16), device=dev), torch.randn((2, 150, 16), device=dev)
    want = ref.conv_bwd(x, w, dout, b)
    cut = 71
    p, q = x[:, :cut].contiguous(), x[:, cut:].contiguous()
    _, s = conv1d_fwd(p, w, b)
    d2 = conv1d_bwd(q, w, dout[:, cut:].contiguous(), b, s)
    d1 = conv1d_bwd(p, w, dout[:, :cut].contiguous(), b, None, dstate_out=d2["dstate_in"])
    torch.cuda.synchronize()
    assert_within("dxin", torch.cat([d1["dxin"], d2["dxin"]], 1), rounded(want["dxin"], torch.float32))
    v, bound = want["dweight"]
    assert_within("dweight", d1["dweight"] + d2["dweight"], (v, 2 * bound + ref.U * v.abs()))


class _Block:
    """A recurrent block as a user composes it: norm with residual, projection
    to the branch and both gates, convolution, gated recurrence, projection."""

    def __init__(self, dev, dim, inner, io, seed=0):
        g = torch.Generator().manual_seed(seed)

        def p(*shape, scale=1.0):
            return (torch.randn(shape, generator=g) * scale).to(dev)

        self.io, self.inner = io, inner
        self.wn, self.wc, self.bc = 1 + p(dim, scale=0.1), p(inner, 4, scale=0.5), p(inner, scale=0.1)
        self.win, self.wout = p(dim, 3 * inner, scale=dim ** -0.5), p(inner, dim, scale=inner ** -0.5)
        self.A = (-0.01 - torch.rand(inner, generator=g)).to(dev)

    def forward(self, x, res):
        b, L, dim = x.shape
        n = self.inner
        y, s = rmsnorm_fwd(x.view(-1, dim), self.wn, res.view(-1, dim))
        z = (y.float() @ self.win).to(self.io).view(b, L, 3 * n)
        u = z[..., :n].contiguous()
        c, conv_state = conv1d_fwd(u, self.wc, self.bc)
        h, last, marks = gated_scan_fwd(c, z[..., n:2 * n], z[..., 2 * n:], self.A, return_checkpoints=True)
        self.saved = (y, s, z, u, c, h, marks)
        return (h.float() @ self.wout).to(self.io), s.view(b, L, dim), conv_state, last

    def backward(self, dout, ds):
        y, s, z, u, c, h, marks = self.saved
        b, L, dim = dout.shape
        n = self.inner
        dh = (dout.float() @ self.wout.t()).to(self.io)
        dz = torch.empty_like(z)
        d = gated_scan_bwd(c, z[..., n:2 * n], z[..., 2 * n:], self.A, dh, marks, dr=dz[..., n:2 * n], dg=dz[..., 2 * n:],
                           want_dh0=False)
        dc = conv1d_bwd(u, self.wc, d["dx"], self.bc, want_dstate=False)
        dz[..., :n] = dc["dxin"]
        dy = (dz.view(-1, 3 * n).float() @ self.win.t()).to(self.io)
        dn = rmsnorm_bwd(s, self.wn, dy, ds=ds.view(-1, dim))
        return {"x": dn["dx"].view(b, L, dim), "res": dn["dresidual"].view(b, L, dim), "wn": dn["dweight"],
                "A": d["dA"], "wc": dc["dweight"], "bc": dc["dbias"],
                "win": y.float().t() @ dz.view(-1, 3 * n).float(),
                "wout": h.float().view(-1, n).t() @ dout.view(-1, dim).float()}

    def token(self, x, res, conv_state, state):
        n = self.inner
        y, s = rmsnorm_fwd(x, self.wn, res)
        z = (y.float() @ self.win).to(self.io)
        c = conv1d_update(conv_state, z[:, :n].contiguous(), self.wc, self.bc)
        h = gated_update(state, c, z[:, n:2 * n], z[:, 2 * n:], self.A)
        return (h.float() @ self.wout).to(self.io), s

    def plain(self, x, res, grads=None):
        """The same in 64 bits, by automatic differentiation when grads = (dout, ds)."""
        leaves = {k: getattr(self, k).double().requires_grad_() for k in ("wn", "A", "wc", "bc", "win", "wout")}
        leaves["x"], leaves["res"] = x.double().requires_grad_(), res.double().requires_grad_()
        p, n = leaves, self.inner
        s = p["x"] + p["res"]
        y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + 1e-6) * p["wn"]
        z = y @ p["win"]
        u = torch.nn.functional.pad(z[..., :n].transpose(1, 2), (3, 0))
        c = torch.nn.functional.silu(torch.nn.functional.conv1d(u, p["wc"][:, None], p["bc"], groups=n)).transpose(1, 2)
        a = torch.exp(p["A"] * torch.sigmoid(z[..., n:2 * n]))
        b = torch.sqrt(1 - a * a) * torch.sigmoid(z[..., 2 * n:]) * c
        h, hs = torch.zeros_like(b[:, 0]), []
        for t in range(x.shape[1]):
            h = a[:, t] * h + b[:, t]
            hs.append(h)
        out = torch.stack(hs, 1) @ p["wout"]
        if grads is None:
            return out, s
        names = list(leaves)
        got = torch.autograd.grad((out * grads[0].double()).sum() + (s * grads[1].double()).sum(), [leaves[k] for k in names])
        return out.detach(), s.detach(), dict(zip(names, got))


def test_block_trained_and_served(dev):
    """Norm, convolution and recurrence as one block: a training step's
    outputs and gradients, then a prefill continued token by token, against
    the block in 64 bits (the framework's error metric and fp32 tolerance)."""
    blk = _Block(dev, 48, 80, torch.float32)
    g = torch.Generator().manual_seed(5)
    x, res, dout, ds = (torch.randn((2, 200, 48), generator=g).to(dev) for _ in range(4))
    out, s, _, _ = blk.forward(x, res)
    got = blk.backward(dout, ds)
    w_out, w_s, want = _cpu(blk).plain(x.cpu(), res.cpu(), (dout.cpu(), ds.cpu()))
    torch.cuda.synchronize()
    assert norm_err(out.cpu(), w_out) <= TOL["f32"] and norm_err(s.cpu(), w_s) <= TOL["f32"]
    for name, t in want.items():
        assert norm_err(got[name].cpu(), t) <= TOL["f32"], name
    _, _, conv_state, state = blk.forward(x[:, :180].contiguous(), res[:, :180].contiguous())
    for t in range(180, 200):
        o, _ = blk.token(x[:, t].contiguous(), res[:, t].contiguous(), conv_state, state)
        assert norm_err(o.cpu(), w_out[:, t]) <= TOL["f32"], t


def _cpu(blk):
    c = object.__new__(_Block)
    c.__dict__.update({k: v.cpu() if isinstance(v, torch.Tensor) else v for k, v in blk.__dict__.items()})
    return c


def test_block_in_a_graph(dev):
    """A captured training step and token, replayed on new inputs with eager
    calls and synchronizations between, give the eager results each time."""
    blk = _Block(dev, 64, 192, torch.bfloat16)
    x, res, dout, ds = (torch.randn((2, 700, 64), device=dev).bfloat16() for _ in range(4))
    xt, rt = x[:, 0].contiguous(), res[:, 0].contiguous()
    cs, st = torch.zeros((2, 192, 3), dtype=torch.bfloat16, device=dev), torch.zeros((2, 192), device=dev)

    def step():
        v, w = torch.randn_like(xt), torch.ones(64, device=dev)
        out, s, conv_state, last = blk.forward(x, res)
        d = blk.backward(dout, ds)
        tok, _ = blk.token(xt, rt, cs, st)
        q, scale, _ = rmsnorm_quant_fwd(xt, w, rt, group=128)
        return [out, s, conv_state, last, tok, q.float(), scale] + [d[k] for k in sorted(d)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        for t in (x, res, dout, ds):
            t.copy_(torch.randn(t.shape, device=dev))
        cs.zero_()
        st.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        cs.zero_()
        st.zero_()
        want = step()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (k, i)


def test_two_streams_at_once(dev):
    """Calls in flight on two streams do not meet."""
    a, b = _gated_inputs(dev, 2, 5000, 256, torch.bfloat16), _gated_inputs(dev, 2, 5000, 256, torch.bfloat16, seed=1)
    want = [gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], return_checkpoints=True) for v in (a, b)]
    wantd = [gated_scan_bwd(v["x"], v["r"], v["g"], v["A"], v["dout"], w[2]) for v, w in zip((a, b), want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for s, v, w in zip(streams, (a, b), want):
            with torch.cuda.stream(s):
                o = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], return_checkpoints=True)
                got.append((w, o, gated_scan_bwd(v["x"], v["r"], v["g"], v["A"], v["dout"], o[2])))
    torch.cuda.synchronize()
    for k, (w, o, d) in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(w, o))
        assert all(torch.equal(d[n], wantd[k % 2][n]) for n in d)


def test_offsets_past_32_bits(dev):
    """Tensors of more than 2^31 elements: the end of a long sequence is what
    a call on the end alone gives, from the state that enters it."""
    L, dim, tail = 262144 + 65, 8200, 128 + 65
    g = torch.Generator(device=dev).manual_seed(9)
    x, r, i = (torch.randn((1, L, dim), generator=g, device=dev, dtype=torch.bfloat16) for _ in range(3))
    A = -0.01 - torch.rand(dim, generator=g, device=dev)
    assert x.numel() > 2 ** 31 and (L - tail) % 128 == 0
    out, last, marks = gated_scan_fwd(x, r, i, A, return_checkpoints=True)
    e = [t[:, -tail:].contiguous() for t in (x, r, i)]
    o, h, m = gated_scan_fwd(*e, A, h0=marks[:, (L - tail) // CHECKPOINT].contiguous(), return_checkpoints=True)
    torch.cuda.synchronize()
    assert torch.equal(out[:, -tail:], o) and torch.equal(last, h) and torch.equal(marks[:, -m.shape[1]:], m)
    d = gated_scan_bwd(x, r, i, A, out, marks)
    de = gated_scan_bwd(*e, A, o, m)
    torch.cuda.synchronize()
    for k in ("dx", "dr", "dg"):
        assert torch.equal(d[k][:, -tail:], de[k]), k
    del d, de, marks, r, i
    w, b = torch.randn((dim, 4), generator=g, device=dev), torch.randn(dim, generator=g, device=dev)
    dc = conv1d_bwd(x, w, out, b, want_dstate=False)
    ec = conv1d_bwd(x[:, -tail:].contiguous(), w, out[:, -tail:].contiguous(), b,
                    x[:, -tail - 3:-tail].transpose(1, 2).contiguous(), want_dstate=False)
    torch.cuda.synchronize()
    assert torch.equal(dc["dxin"][:, -tail + 3:], ec["dxin"][:, 3:])
    y, _ = rmsnorm_fwd(x.view(L, dim), torch.ones(dim, device=dev))
    ye, _ = rmsnorm_fwd(x.view(L, dim)[-tail:], torch.ones(dim, device=dev))
    torch.cuda.synchronize()
    assert torch.equal(y[-tail:], ye)


def test_strides_past_32_bits(dev):
    """Rows so far apart that offsets within a tile pass 32 bits."""
    wide, dim, L = 1 << 26, 66, 37
    room = torch.empty((1, L, wide), dtype=torch.bfloat16, device=dev)
    v = _gated_inputs(dev, 1, L, dim, torch.bfloat16)
    x, out = room[..., 5:5 + dim], room[..., wide - dim:]
    x.copy_(v["x"])
    _, last, marks = gated_scan_fwd(x, v["r"], v["g"], v["A"], out=out, return_checkpoints=True)
    dx = room[..., wide // 2:wide // 2 + dim]
    d = gated_scan_bwd(x, v["r"], v["g"], v["A"], v["dout"], marks, dx=dx)
    torch.cuda.synchronize()
    want = ref.gated(v["x"], v["r"], v["g"], v["A"], None, None, v["dout"])
    assert_within("out", out, rounded(want["out"], torch.bfloat16))
    assert_within("dx", dx, rounded(want["dx"], torch.bfloat16))
    assert_within("dA", d["dA"], rounded(want["dA"], torch.float32))
    rows = room[0]
    y, _ = rmsnorm_fwd(rows[:, 5:5 + dim], torch.ones(dim, device=dev), out=rows[:, wide - dim:])
    torch.cuda.synchronize()
    assert_within("norm", y, rounded(ref.norm(v["x"][0], torch.ones(dim), None, 1e-6)["out"], torch.bfloat16))
    st = torch.zeros((L, dim), device=dev)
    o = gated_update(st, rows[:, 5:5 + dim], v["r"][0], v["g"][0], v["A"], out=rows[:, wide - dim:])
    torch.cuda.synchronize()
    one = ref.gated(v["x"][0][:, None], v["r"][0][:, None], v["g"][0][:, None], v["A"])
    assert_within("token", o, rounded(tuple(t[:, 0] for t in one["out"]), torch.bfloat16))


def test_gated_beside_other_work(dev):
    """Workgroups that start late, because another stream fills the GPU, change nothing."""
    v = _gated_inputs(dev, 4, 6000, 384, torch.bfloat16, resets=0.001)

    def both():
        out, last, marks = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], reset=v["reset"], return_checkpoints=True)
        d = gated_scan_bwd(v["x"], v["r"], v["g"], v["A"], v["dout"], marks, reset=v["reset"])
        return [out, last, marks] + [d[k] for k in ("dx", "dr", "dg", "dA", "dh0")]

    want = both()
    torch.cuda.synchronize()
    side, a = torch.cuda.Stream(), torch.randn((4096, 4096), device=dev)
    b = torch.empty((1 << 27,), device=dev)
    for _ in range(4):
        with torch.cuda.stream(side):
            for _ in range(4):
                a @ a
                b.fill_(1.0)
        got = both()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_python_refusals(dev):
    """What a call must not be given, by name, before anything is launched."""
    from selective_state_space_56_amd.binding import MambaScanError
    v = _gated_inputs(dev, 2, 10, 16, torch.float32)
    x, r, g, A = v["x"], v["r"], v["g"], v["A"]
    marks = torch.zeros((2, 1, 16), device=dev)
    with pytest.raises(TypeError, match="r has dtype"):
        gated_scan_fwd(x, r.bfloat16(), g, A)
    with pytest.raises(ValueError, match="g has shape"):
        gated_scan_fwd(x, r, g[:, :5], A)
    with pytest.raises(ValueError, match="A has shape"):
        gated_scan_fwd(x, r, g, A[:8])
    with pytest.raises(ValueError, match="h0 is on cpu"):
        gated_scan_fwd(x, r, g, A, h0=torch.zeros((2, 16)))
    with pytest.raises(ValueError, match="reset has shape"):
        gated_scan_fwd(x, r, g, A, reset=torch.zeros((2, 9), dtype=torch.bool, device=dev))
    with pytest.raises(ValueError, match="must be contiguous"):
        gated_scan_fwd(x, r, g, A, reset=torch.zeros((10, 2), dtype=torch.uint8, device=dev).t())
    with pytest.raises(MambaScanError, match="out overlaps x"):
        gated_scan_fwd(x, r, g, A, out=x)
    with pytest.raises(MambaScanError, match="A is NULL"):
        gated_scan_fwd(x, r, g, None)
    with pytest.raises(MambaScanError, match="dr overlaps dg"):
        gated_scan_bwd(x, r, g, A, v["dout"], marks, dr=(t := torch.empty_like(x)), dg=t)
    with pytest.raises(MambaScanError, match="checkpoints is NULL"):
        gated_scan_bwd(x, r, g, A, v["dout"], None)
    with pytest.raises(ValueError, match="checkpoints has shape"):
        gated_scan_bwd(x, r, g, A, v["dout"], torch.zeros((2, 2, 16), device=dev))
    with pytest.raises(MambaScanError, match="out overlaps x"):
        gated_update(v["h0"], x[:, 0], r[:, 0], g[:, 0], A, out=x[:, 0])
    s = torch.randn((4, 16), device=dev)
    w = torch.ones(16, device=dev)
    with pytest.raises(TypeError, match="residual has dtype"):
        rmsnorm_fwd(s, w, s.bfloat16())
    with pytest.raises(ValueError, match="there is none without a residual"):
        rmsnorm_fwd(s, w, sum=s.clone())
    with pytest.raises(MambaScanError, match="sum overlaps x"):
        rmsnorm_fwd(s, w, s.clone(), sum=s)
    with pytest.raises(MambaScanError, match="group 32 is not"):
        rmsnorm_quant_fwd(s, w, group=32)
    with pytest.raises(MambaScanError, match="eps"):
        rmsnorm_fwd(s, w, eps=-1.0)
    with pytest.raises(MambaScanError, match="dim 65537 too large"):
        rmsnorm_fwd(torch.zeros((1, 65537), device=dev), torch.ones(65537, device=dev))
    with pytest.raises(ValueError, match="weight has shape"):
        rmsnorm_bwd(s, w[:4], s.clone())
    with pytest.raises(MambaScanError, match="dresidual overlaps sum"):
        rmsnorm_bwd(s, w, s.clone(), dresidual=s)
    c = torch.zeros((1, 6, 16), device=dev)
    with pytest.raises(MambaScanError, match="width 5 not supported"):
        conv1d_bwd(c, torch.zeros((16, 5), device=dev), c.clone())
    with pytest.raises(ValueError, match="dout has shape"):
        conv1d_bwd(c, torch.zeros((16, 4), device=dev), c[:, :3].contiguous())
    with pytest.raises(ValueError, match="must be contiguous"):
        conv1d_bwd(torch.zeros((1, 6, 32), device=dev)[..., ::2], torch.zeros((16, 4), device=dev), c)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(dev, seed):
    """Seeded shapes and options of all the operators, each value within its bound."""
    import random
    rng = random.Random(1000 + seed)

    def between(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    io = rng.choice([torch.bfloat16, torch.float32])
    dim, batch = between(1, 700), rng.choice([1, 1, 2, 3, 7])
    L = between(1, 200000 // (dim * batch) + 2)
    v = _gated_inputs(dev, batch, L, dim, io, rng.random() < 0.5, rng.choice([0.0, 0.01, 0.3]), seed)
    print(f"seed {seed}: {batch}x{L}x{dim} {io}", flush=True)
    _check_gated(v, io, rng.random() < 0.5)
    rows, wide = between(1, 400), between(1, 3000)
    res = rng.choice([None, torch.float32, io])
    x, residual, w, dout, ds = _norm_inputs(dev, rows, wide, io, res, seed)
    y, total = rmsnorm_fwd(x, w, residual, eps=1e-5)
    q, scale, _ = rmsnorm_quant_fwd(x, w, residual, eps=1e-5, group=rng.choice([0, 128]))
    stream = x if residual is None else total
    d = rmsnorm_bwd(stream, w, dout, ds=ds, eps=1e-5)
    torch.cuda.synchronize()
    want = ref.norm(x, w, residual, 1e-5, dout, ds)
    assert_within("norm", y, rounded(want["out"], io))
    _check_quant(q, scale, want, 0 if scale.shape[1] == 1 and wide > 128 else 128)
    assert_within("dresidual", d["dresidual"], rounded(want["dresidual"], stream.dtype))
    assert_within("dx", d["dx"], rounded(want["dresidual"], io))
    assert_within("dweight", d["dweight"], rounded(want["dweight"], torch.float32))
    width = rng.choice([1, 2, 3, 4])
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, to=torch.float32):
        return torch.randn(shape, generator=g).to(to).to(dev)

    cx, cd, cw, cb = normal(batch, L, dim, to=io), normal(batch, L, dim, to=io), normal(dim, width), normal(dim)
    st = normal(batch, dim, width - 1, to=io) if rng.random() < 0.5 else None
    dst = normal(batch, dim, width - 1) if rng.random() < 0.5 else None
    d = conv1d_bwd(cx, cw, cd, cb, st, dstate_out=dst)
    torch.cuda.synchronize()
    want = ref.conv_bwd(cx, cw, cd, cb, st, dst)
    assert_within("dxin", d["dxin"], rounded(want["dxin"], io))
    for name in ("dweight", "dbias", "dstate_in"):
        assert_within(name, d[name], rounded(want[name], torch.float32))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gated_ignores_the_gate_of_a_reset(dev, io):
    """At a reset the recurrence gate is not looked at: NaN and infinities there
    change no value, and get no gradient."""
    v = _gated_inputs(dev, 2, 90, 33, IO[io], resets=0.2)
    clean = _check_gated(v, IO[io])
    at = v["reset"].nonzero()
    for k, (b, t) in enumerate(at.tolist()):
        v["r"][b, t] = (NAN, INF, -INF)[k % 3]
    out, last, marks = gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], h0=v["h0"], reset=v["reset"], return_checkpoints=True)
    d = gated_scan_bwd(v["x"], v["r"], v["g"], v["A"], v["dout"], marks, reset=v["reset"], dlast=v["dlast"])
    torch.cuda.synchronize()
    assert torch.equal(out, clean[0]) and torch.equal(last, clean[1]) and torch.equal(marks, clean[2])
    for k in ("dx", "dr", "dg", "dA", "dh0"):
        assert torch.equal(d[k], clean[3][k]), k
    assert float(d["dr"][v["reset"]].abs().max()) == 0.0
