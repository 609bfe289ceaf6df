"""ctypes binding of the block operators around the scan (C ABI in
``include/block/``): the gated linear recurrence, the RMS norm with the
residual's addition, and the convolution's backward.

As ``binding.py``: argument checks, output allocation and the current HIP
stream only. Calls run on the tensors' own device, whichever device is
current.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from .binding import _IO, ConvDesc, _check, _need, _row_stride, load_library

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
CHECKPOINT = 64  # MAMBA_GATED_CHECKPOINT


class GatedDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class GatedStrides(ctypes.Structure):
    """mamba_gated_strides: elements between consecutive token rows (0 = contiguous)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("x", "r", "g", "out", "dx", "dr", "dg")]


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("group", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("residual_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("flags", ctypes.c_uint32)]


class NormStrides(ctypes.Structure):
    """mamba_norm_strides: elements between consecutive rows (0 = contiguous)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("x", "residual", "sum", "out", "dsum", "dresidual", "dx")]


_ready = None
_lock = threading.Lock()


def _library():
    """The native library with the block operators' signatures set, once."""
    global _ready
    if _ready is None:
        lib = load_library()
        with _lock:
            if _ready is None:
                P, vp, sz, st = ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
                gated = [P(GatedDesc), P(GatedStrides)]
                norm = [P(NormDesc), P(NormStrides)]
                for name, res, args in [
                        ("mamba_gated_scan_workspace_size", sz, gated[:1]),
                        ("mamba_gated_scan_bwd_workspace_size", sz, gated[:1]),
                        ("mamba_gated_scan_fwd", st, gated + [vp] * 10 + [sz, vp]),
                        ("mamba_gated_scan_bwd", st, gated + [vp] * 14 + [sz, vp]),
                        ("mamba_gated_update", st, gated + [vp] * 7),
                        ("mamba_rmsnorm_fwd", st, norm + [vp] * 6),
                        ("mamba_rmsnorm_quant_fwd", st, norm + [vp] * 7),
                        ("mamba_rmsnorm_bwd_workspace_size", sz, norm[:1]),
                        ("mamba_rmsnorm_bwd", st, norm + [vp] * 8 + [sz, vp]),
                        ("mamba_conv1d_bwd_workspace_size", sz, [P(ConvDesc)]),
                        ("mamba_conv1d_bwd", st, [P(ConvDesc)] + [vp] * 11 + [sz, vp])]:
                    f = getattr(lib, name)
                    f.restype, f.argtypes = res, args
                _ready = lib
    return _ready


def _p(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object around it (1.7 us less per
# call, of about 9 for a small one), where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev):
    return _raw_stream(dev.index) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream


def _run(dev, f, *args):
    """f(*args, the current stream of dev) with dev as the current device."""
    if dev.index == torch.cuda.current_device():
        st = f(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = f(*args, _stream(dev))
    if st:
        _check(_library(), st)


def _workspace(dev, size, d):
    """(workspace or None, its bytes) by the size function, which may go by the
    current device's compute units."""
    if dev.index == torch.cuda.current_device():
        n = size(d)
    else:
        with torch.cuda.device(dev):
            n = size(d)
    return (torch.empty(n, dtype=torch.uint8, device=dev) if n else None), n


def _plain(t, shape, dtype, dev):
    """Whether t is a contiguous tensor of this kind."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.device == dev)


def _rows(t, name, shape, dtype, dev, rows_axis):
    """_row_stride of a tensor that may be a column slice; 0 for a contiguous
    one and for None. The usual layouts are recognised without its walk over
    the axes."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev:
        if t.is_contiguous():
            return 0
        step = t.stride()
        row = step[rows_axis]
        if step[-1] == 1 and row >= shape[-1] and (rows_axis == 0 or step[0] == row * shape[1]):
            return row
    s = _row_stride(t, name, shape, dtype, dev, rows_axis)
    # rows apart by less than a row's length share elements: reading them is
    # only well defined for the layouts the library takes
    if s < shape[-1] and t.numel():
        raise ValueError(f"{name}: rows overlap")
    return s


def _whole(t, name, shape, dtype, dev):
    if t is not None and not _plain(t, shape, dtype, dev):
        _need(t, name, shape, dtype, dev)


def _io_of(who, x, dims, names):
    if not isinstance(x, torch.Tensor) or x.dim() != dims:
        raise ValueError(f"{who}: {names}")
    if x.device.type != "cuda":
        raise ValueError(f"{who} runs on a GPU tensor")
    if x.dtype not in _IO:
        raise TypeError(f"unsupported io dtype {x.dtype}")
    return x.dtype, x.device


# Outputs are made like an input that has been checked: contiguous, or a column
# slice, whose copy in shape is contiguous (0.5 us less than by shape and type).
def _new(shape, dtype, dev):
    return torch.empty(shape, dtype=dtype, device=dev)


def _reset(reset, shape, dev):
    if reset is None:
        return None
    if isinstance(reset, torch.Tensor) and reset.dtype == torch.bool:
        reset = reset.view(torch.uint8)
    _whole(reset, "reset", shape, torch.uint8, dev)
    return reset


def _strides(cls, *values):
    """The strides' struct, or NULL when every tensor is contiguous."""
    return ctypes.byref(cls(*values)) if any(values) else None


def gated_scan_fwd(x, r, g, A, *, h0=None, reset=None, out=None, last_state=None, return_last_state=True,
                   return_checkpoints=False):
    """Gated linear recurrence over full sequences (mamba_gated_scan_fwd):
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(g_t) x_t with
    a_t = exp(A sigmoid(r_t)).

    x, r, g: (batch, L, dim) float32 or bfloat16 on a GPU, each contiguous or
    a column slice of a wider tensor; A: (dim,) float32, <= 0; h0: (batch,
    dim) float32 or None (zeros); reset: (batch, L) bool or uint8, set where
    a sequence starts (the state before it is dropped), or None. Returns
    (out, last_state): the states in x's dtype and the last one in float32
    (None if not requested). With ``return_checkpoints`` a third value, the
    states that gated_scan_bwd starts from."""
    lib = _library()
    io, dev = _io_of("gated_scan_fwd", x, 3, "x must be (batch, L, dim)")
    shape = x.shape
    batch, L, dim = shape
    sx = _rows(x, "x", shape, io, dev, 1)
    sr = _rows(r, "r", shape, io, dev, 1)
    sg = _rows(g, "g", shape, io, dev, 1)
    _whole(A, "A", (dim,), F32, dev)
    _whole(h0, "h0", (batch, dim), F32, dev)
    reset = _reset(reset, (batch, L), dev)
    if out is None:
        out = torch.empty_like(x)
    so = _rows(out, "out", shape, io, dev, 1)
    if last_state is None and return_last_state:
        last_state = _new((batch, dim), F32, dev)
    _whole(last_state, "last_state", (batch, dim), F32, dev)
    marks = _new((batch, -(-L // CHECKPOINT), dim), F32, dev) if return_checkpoints else None
    d = ctypes.byref(GatedDesc(batch, L, dim, _IO[io], 0))
    ws, nbytes = _workspace(dev, lib.mamba_gated_scan_workspace_size, d)
    _run(dev, lib.mamba_gated_scan_fwd, d, _strides(GatedStrides, sx, sr, sg, so), _p(x), _p(r), _p(g), _p(A), _p(h0),
         _p(reset), _p(out), _p(last_state), _p(marks), _p(ws), nbytes)
    return (out, last_state, marks) if return_checkpoints else (out, last_state)


def gated_scan_bwd(x, r, g, A, dout, checkpoints, *, reset=None, dlast=None, dx=None, dr=None, dg=None,
                   want_dh0=True):
    """Gradients of gated_scan_fwd (mamba_gated_scan_bwd) for dLoss/dout =
    dout and dLoss/d(last_state) = dlast ((batch, dim) float32 or None).
    ``checkpoints`` is the forward's third value; x, r, g, A, reset as given
    to it. Returns a dict with dx, dr, dg (batch, L, dim) in x's dtype, dA
    (dim,) and dh0 (batch, dim, None unless want_dh0) float32. dx, dr and dg
    may be given, also as column slices of wider tensors (dr and dg as halves
    of one gradient buffer)."""
    lib = _library()
    io, dev = _io_of("gated_scan_bwd", x, 3, "x must be (batch, L, dim)")
    shape = x.shape
    batch, L, dim = shape
    sx = _rows(x, "x", shape, io, dev, 1)
    sr = _rows(r, "r", shape, io, dev, 1)
    sg = _rows(g, "g", shape, io, dev, 1)
    so = _rows(dout, "dout", shape, io, dev, 1)
    _whole(A, "A", (dim,), F32, dev)
    _whole(checkpoints, "checkpoints", (batch, -(-L // CHECKPOINT), dim), F32, dev)
    _whole(dlast, "dlast", (batch, dim), F32, dev)
    reset = _reset(reset, (batch, L), dev)
    dx = torch.empty_like(x) if dx is None else dx
    dr = torch.empty_like(x) if dr is None else dr
    dg = torch.empty_like(x) if dg is None else dg
    sdx = _rows(dx, "dx", shape, io, dev, 1)
    sdr = _rows(dr, "dr", shape, io, dev, 1)
    sdg = _rows(dg, "dg", shape, io, dev, 1)
    dA = torch.empty_like(A)
    dh0 = _new((batch, dim), F32, dev) if want_dh0 else None
    d = ctypes.byref(GatedDesc(batch, L, dim, _IO[io], 0))
    ws, nbytes = _workspace(dev, lib.mamba_gated_scan_bwd_workspace_size, d)
    _run(dev, lib.mamba_gated_scan_bwd, d, _strides(GatedStrides, sx, sr, sg, so, sdx, sdr, sdg), _p(x), _p(r), _p(g),
         _p(A), _p(reset), _p(checkpoints), _p(dout), _p(dlast), _p(dx), _p(dr), _p(dg), _p(dA), _p(dh0), _p(ws),
         nbytes)
    return {"dx": dx, "dr": dr, "dg": dg, "dA": dA, "dh0": dh0}


def gated_update(state, x, r, g, A, *, out=None):
    """One decode token of the gated linear recurrence (mamba_gated_update):
    advances ``state`` (batch, dim) float32 in place and returns out (batch,
    dim). x, r, g: (batch, dim), contiguous or column slices."""
    lib = _library()
    io, dev = _io_of("gated_update", x, 2, "x must be (batch, dim)")
    shape = x.shape
    batch, dim = shape
    sx = _rows(x, "x", shape, io, dev, 0)
    sr = _rows(r, "r", shape, io, dev, 0)
    sg = _rows(g, "g", shape, io, dev, 0)
    _whole(state, "state", shape, F32, dev)
    _whole(A, "A", (dim,), F32, dev)
    if out is None:
        out = torch.empty_like(x)
    so = _rows(out, "out", shape, io, dev, 0)
    _run(dev, lib.mamba_gated_update, ctypes.byref(GatedDesc(batch, 1, dim, _IO[io], 0)),
         _strides(GatedStrides, sx, sr, sg, so), _p(state), _p(x), _p(r), _p(g), _p(A), _p(out))
    return out


def _norm_args(who, x, weight, residual, sum_out, group, eps):
    io, dev = _io_of(who, x, 2, "x must be (rows, dim)")
    shape = x.shape
    res = io if residual is None else getattr(residual, "dtype", None)
    if res is not io and res is not F32:
        raise TypeError(f"residual has dtype {res}, expected {io} or {F32}")
    sx = _rows(x, "x", shape, io, dev, 0)
    sres = _rows(residual, "residual", shape, res, dev, 0)
    _whole(weight, "weight", (shape[1],), F32, dev)
    if residual is None and sum_out is not None:
        raise ValueError("sum is the stream with the residual added: there is none without a residual")
    if residual is not None and sum_out is None:
        sum_out = torch.empty_like(residual)
    ssum = _rows(sum_out, "sum", shape, res, dev, 0)
    return io, dev, shape, NormDesc(shape[0], shape[1], group, _IO[io], _IO[res], eps, 0), sum_out, (sx, sres, ssum)


def rmsnorm_fwd(x, weight, residual=None, *, eps=1e-6, out=None, sum=None):
    """RMS norm of x + residual (mamba_rmsnorm_fwd). x: (rows, dim) float32 or
    bfloat16 on a GPU; weight: (dim,) float32; residual: (rows, dim) in x's
    dtype or float32, or None. Returns (out, sum): the normed rows in x's
    dtype, and x + residual in the residual's dtype (None without one), which
    is what is normed. ``sum`` may be the residual itself (updated in place).
    Rows may be column slices of wider tensors."""
    lib = _library()
    io, dev, shape, d, sum, s = _norm_args("rmsnorm_fwd", x, weight, residual, sum, 0, eps)
    if out is None:
        out = torch.empty_like(x)
    so = _rows(out, "out", shape, io, dev, 0)
    _run(dev, lib.mamba_rmsnorm_fwd, ctypes.byref(d), _strides(NormStrides, *s, so), _p(x), _p(residual), _p(weight),
         _p(out), _p(sum))
    return out, sum


def rmsnorm_quant_fwd(x, weight, residual=None, *, eps=1e-6, group=0, out=None, scale=None, sum=None):
    """rmsnorm_fwd with an 8-bit output (mamba_rmsnorm_quant_fwd). Returns (q,
    scale, sum): q (rows, dim) float8_e4m3fn and scale float32, (rows, 1) with
    group 0 or (rows, ceil(dim / 128)) with group 128; q * scale is the normed
    row to e4m3's precision."""
    lib = _library()
    _, dev, shape, d, sum, s = _norm_args("rmsnorm_quant_fwd", x, weight, residual, sum, group, eps)
    if out is None:
        out = _new(shape, F8, dev)
    so = _rows(out, "out", shape, F8, dev, 0)
    scales = (shape[0], -(-shape[1] // group) if group > 0 else 1)
    if scale is None:
        scale = _new(scales, F32, dev)
    _whole(scale, "scale", scales, F32, dev)
    _run(dev, lib.mamba_rmsnorm_quant_fwd, ctypes.byref(d), _strides(NormStrides, *s, so), _p(x), _p(residual),
         _p(weight), _p(out), _p(scale), _p(sum))
    return out, scale, sum


def rmsnorm_bwd(sum, weight, dout, *, ds=None, eps=1e-6, dresidual=None):
    """Gradients of rmsnorm_fwd (mamba_rmsnorm_bwd). sum: the forward's second
    value (x itself without a residual); dout: (rows, dim) dLoss/dout; ds:
    dLoss/d(sum) in sum's dtype, from the stream's later readers, or None.
    Returns a dict: dresidual (rows, dim) in sum's dtype, dx the same
    gradient in dout's dtype (the same tensor when the dtypes are), dweight
    (dim,) float32. ``dresidual`` may be ds itself (updated in place)."""
    lib = _library()
    io, dev = _io_of("rmsnorm_bwd", dout, 2, "dout must be (rows, dim)")
    shape = dout.shape
    res = getattr(sum, "dtype", None)
    if res is not io and res is not F32:
        raise TypeError(f"sum has dtype {res}, expected {io} or {F32}")
    so = _rows(dout, "dout", shape, io, dev, 0)
    ssum = _rows(sum, "sum", shape, res, dev, 0)
    sds = _rows(ds, "ds", shape, res, dev, 0)
    _whole(weight, "weight", (shape[1],), F32, dev)
    if dresidual is None:
        dresidual = torch.empty_like(sum)
    sdr = _rows(dresidual, "dresidual", shape, res, dev, 0)
    dx = None if res is io else torch.empty_like(dout)
    dweight = torch.empty_like(weight)
    d = ctypes.byref(NormDesc(shape[0], shape[1], 0, _IO[io], _IO[res], eps, 0))
    ws, nbytes = _workspace(dev, lib.mamba_rmsnorm_bwd_workspace_size, d)
    _run(dev, lib.mamba_rmsnorm_bwd, d, _strides(NormStrides, 0, 0, ssum, so, sds, sdr, 0), _p(sum), _p(weight),
         _p(dout), _p(ds), _p(dresidual), _p(dx), _p(dweight), _p(ws), nbytes)
    return {"dx": dresidual if dx is None else dx, "dresidual": dresidual, "dweight": dweight}


def conv1d_bwd(xin, weight, dout, bias=None, state_in=None, *, dstate_out=None, want_dstate=True):
    """Gradients of conv1d_fwd(xin, weight, bias, state_in) (mamba_conv1d_bwd)
    for dLoss/dout = dout (batch, L, dim, xin's dtype) and
    dLoss/d(state_out) = dstate_out ((batch, dim, width - 1) float32 or None).
    Returns a dict with dxin (batch, L, dim) in xin's dtype, dweight (dim,
    width), dbias (dim,) and dstate_in (batch, dim, width - 1, None unless
    want_dstate), float32."""
    lib = _library()
    io, dev = _io_of("conv1d_bwd", xin, 3, "xin must be (batch, L, dim)")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be (dim, width)")
    shape = xin.shape
    batch, L, dim = shape
    width = weight.shape[1]
    state = (batch, dim, max(width - 1, 0))
    _whole(xin, "xin", shape, io, dev)
    _whole(dout, "dout", shape, io, dev)
    _whole(weight, "weight", (dim, width), F32, dev)
    _whole(bias, "bias", (dim,), F32, dev)
    _whole(state_in, "state_in", state, io, dev)
    _whole(dstate_out, "dstate_out", state, F32, dev)
    g = {"dxin": torch.empty_like(xin), "dweight": torch.empty_like(weight), "dbias": _new((dim,), F32, dev),
         "dstate_in": _new(state, F32, dev) if want_dstate else None}
    d = ctypes.byref(ConvDesc(batch, L, dim, width, _IO[io], 0))
    ws, nbytes = _workspace(dev, lib.mamba_conv1d_bwd_workspace_size, d)
    _run(dev, lib.mamba_conv1d_bwd, d, _p(xin), _p(weight), _p(bias), _p(state_in), _p(dout), _p(dstate_out),
         _p(g["dxin"]), _p(g["dweight"]), _p(g["dbias"]), _p(g["dstate_in"]), _p(ws), nbytes)
    return g
