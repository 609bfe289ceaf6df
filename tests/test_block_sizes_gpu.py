"""GPU tests of the block operators at the sizes that take their other paths:
many rows per workgroup in the norm, the convolution's long spans, calls that
stream past the last-level cache (their kernels carry the non-temporal hint).
Values against 64 bits within their bounds; where channels do not meet, on
chosen channels of a full-size call."""
import pytest
import torch

import block_ref as ref
from block_ref import assert_within, rounded
from selective_state_space_56_amd import (conv1d_bwd, gated_scan_bwd, gated_scan_fwd, rmsnorm_bwd, rmsnorm_fwd,
                                          rmsnorm_quant_fwd)
from selective_state_space_56_amd.block import CHECKPOINT
from test_block_gpu import IO, _check_quant, _norm_inputs

pytestmark = pytest.mark.gpu
CACHE = 256 << 20  # bytes; calls that move more take the streaming kernels


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", torch.cuda.current_device())


# rows per workgroup go up where (20 waves, 16 in the backward) per compute unit
# are exceeded, from 5120 (4096) rows of one wave to 512 (256) of sixteen
ROWS = [(16500, 40, "f32", "f32"), (11003, 300, "bf16", "f32"), (9001, 512, "bf16", "bf16"),
        (3001, 2560, "bf16", "f32"), (3100, 2500, "bf16", None), (2050, 2560, "f32", "f32"),
        (1100, 8192, "bf16", "bf16"), (1030, 20000, "bf16", "f32"), (700, 9001, "f32", None)]


@pytest.mark.parametrize("rows,dim,io,res", ROWS)
def test_norm_many_rows(dev, rows, dim, io, res):
    print(f"norm {rows}x{dim} {io} {res}", flush=True)
    x, residual, w, dout, ds = _norm_inputs(dev, rows, dim, IO[io], IO.get(res), seed=3)
    y, total = rmsnorm_fwd(x, w, residual, eps=1e-5)
    stream = x if residual is None else total
    d = rmsnorm_bwd(stream, w, dout, ds=ds, eps=1e-5)
    torch.cuda.synchronize()
    want = ref.norm(x, w, residual, 1e-5, dout, ds)
    assert torch.equal(stream.cpu(), want["sum"])
    assert_within("out", y, rounded(want["out"], IO[io]))
    assert_within("dresidual", d["dresidual"], rounded(want["dresidual"], stream.dtype))
    assert_within("dx", d["dx"], rounded(want["dresidual"], IO[io]))
    assert_within("dweight", d["dweight"], rounded(want["dweight"], torch.float32))
    for group in (0, 128):
        q, scale, again = rmsnorm_quant_fwd(x, w, residual, eps=1e-5, group=group)
        torch.cuda.synchronize()
        assert residual is None or torch.equal(again, total)
        _check_quant(q, scale, want, group)


@pytest.mark.parametrize("rows,dim,io,res", [(3001, 2560, "bf16", "f32"), (9001, 512, "bf16", "bf16"),
                                             (700, 9001, "f32", "f32")])
def test_norm_many_rows_in_place(dev, rows, dim, io, res):
    """The stream and its gradient updated in place while later rows are read ahead."""
    x, residual, w, dout, ds = _norm_inputs(dev, rows, dim, IO[io], IO[res], seed=4)
    y, total = rmsnorm_fwd(x, w, residual)
    d = rmsnorm_bwd(total, w, dout, ds=ds)
    s, g = residual.clone(), ds.clone()
    y2, _ = rmsnorm_fwd(x, w, s, sum=s)
    d2 = rmsnorm_bwd(s, w, dout, ds=g, dresidual=g)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(total, s) and torch.equal(d["dresidual"], g)
    assert torch.equal(d["dx"], d2["dx"]) and torch.equal(d["dweight"], d2["dweight"])


def _channels(dim, g):
    """The first and last channels, those on both sides of the tiles' borders, and some others."""
    c = set(range(3)) | set(range(dim - 3, dim)) | {63, 64, 127, 128, 129}
    c |= set(torch.randint(0, dim, (14,), generator=g).tolist())
    return torch.tensor(sorted(v for v in c if v < dim))


@pytest.mark.parametrize("batch,L,dim,io,resets,streams", [
    (4, 1111, 8191, "bf16", 0.002, True), (2, 1030, 8194, "f32", 0.002, True), (3, 1500, 5100, "bf16", 0.0, False)])
def test_gated_full_size(dev, batch, L, dim, io, resets, streams):
    size = batch * L * dim * (2 if io == "bf16" else 4)
    assert (4 * size > CACHE) == streams and (7 * size > CACHE)
    print(f"gated {batch}x{L}x{dim} {io}", flush=True)
    g = torch.Generator(device=dev).manual_seed(L)

    def normal(*shape, to=torch.float32):
        return torch.randn(shape, generator=g, device=dev).to(to)

    x, dout = normal(batch, L, dim, to=IO[io]), normal(batch, L, dim, to=IO[io])
    gates = normal(batch, L, 2 * dim, to=IO[io])
    r, i = gates[..., :dim], gates[..., dim:]
    A = 8.0 * torch.log(0.9 + 0.099 * torch.rand(dim, generator=g, device=dev))
    h0, dlast = normal(batch, dim), normal(batch, dim)
    reset = torch.rand((batch, L), generator=g, device=dev) < resets if resets else None
    out, last, marks = gated_scan_fwd(x, r, i, A, h0=h0, reset=reset, return_checkpoints=True)
    d = gated_scan_bwd(x, r, i, A, dout, marks, reset=reset, dlast=dlast)
    torch.cuda.synchronize()
    at = _channels(dim, torch.Generator().manual_seed(1)).to(dev)
    want = ref.gated(x[..., at], r[..., at], i[..., at], A[at], h0[:, at], reset, dout[..., at], dlast[:, at])
    assert_within("out", out[..., at], rounded(want["out"], IO[io]))
    assert_within("last_state", last[:, at], rounded(want["last_state"], torch.float32))
    assert_within("checkpoints", marks[..., at], rounded(tuple(t[:, ::CHECKPOINT] for t in want["before"]), torch.float32))
    for name in ("dx", "dr", "dg"):
        assert_within(name, d[name][..., at], rounded(want[name], IO[io]))
    for name in ("dA", "dh0"):
        assert_within(name, d[name][..., at], rounded(want[name], torch.float32))
    for t in (out, last, marks, *d.values()):
        assert bool(t.isfinite().all())


@pytest.mark.parametrize("batch,L,dim,width,io,state,streams", [
    (4, 1501, 8191, 4, "bf16", True, True), (2, 1100, 16385, 3, "f32", False, True),
    (2, 643, 16384, 4, "bf16", True, False), (8, 330, 8190, 2, "bf16", False, False),
    (4, 64, 40000, 1, "f32", False, False), (8, 129, 12001, 4, "f32", True, False)])
def test_conv_bwd_long_spans(dev, batch, L, dim, width, io, state, streams):
    """Spans of 64 steps: four waves per compute unit and more, at two channels per lane."""
    size = batch * L * dim * (2 if io == "bf16" else 4)
    waves = batch * -(-dim // 128) * -(-L // 64)
    assert waves >= 4 * torch.cuda.get_device_properties(dev).multi_processor_count
    assert (3 * size > CACHE) == streams
    print(f"conv bwd {batch}x{L}x{dim} W={width} {io}", flush=True)
    g = torch.Generator(device=dev).manual_seed(L)

    def normal(*shape, to=torch.float32):
        return torch.randn(shape, generator=g, device=dev).to(to)

    x, dout = normal(batch, L, dim, to=IO[io]), normal(batch, L, dim, to=IO[io])
    w, b = normal(dim, width) * 0.5, normal(dim) * 0.5
    st = normal(batch, dim, width - 1, to=IO[io]) if state else None
    dst = normal(batch, dim, width - 1) if state else None
    d = conv1d_bwd(x, w, dout, b, st, dstate_out=dst)
    torch.cuda.synchronize()
    at = _channels(dim, torch.Generator().manual_seed(2)).to(dev)
    pick = [None if t is None else t[:, at] for t in (st, dst)]
    want = ref.conv_bwd(x[..., at], w[at], dout[..., at], b[at], *pick)
    assert_within("dxin", d["dxin"][..., at], rounded(want["dxin"], IO[io]))
    assert_within("dweight", d["dweight"][at], rounded(want["dweight"], torch.float32))
    assert_within("dbias", d["dbias"][at], rounded(want["dbias"], torch.float32))
    assert_within("dstate_in", d["dstate_in"][:, at], rounded(want["dstate_in"], torch.float32))
    for t in d.values():
        assert bool(t.isfinite().all())
