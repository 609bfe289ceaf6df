"""ctypes binding of the matrix-state mixer's operators (C ABI in
``include/mixer/``): linear attention with a decay for each head, and the norm
and position rotation of its queries and keys.

As ``block.py``: argument checks, output allocation and the current HIP stream
only. Calls run on the tensors' own device, whichever device is current.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from .binding import _IO, _row_stride, load_library
from .block import F32, _io_of, _new, _p, _run, _strides, _whole, _workspace

HEAD_DECAY, PACKED, ZERO_REST = 1, 2, 4   # MAMBA_LINATTN_*
INTERLEAVED = 1                           # MAMBA_QKNORM_INTERLEAVED
AXES = 4                                  # MAMBA_QKNORM_AXES


class LinattnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seqlen", "nheads", "ngroups", "dkey", "dvalue")] + [
        ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("scale", ctypes.c_float)]


class LinattnStrides(ctypes.Structure):
    """mamba_linattn_strides: elements between consecutive token rows (0 = contiguous)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("q", "k", "v", "out", "dq", "dk", "dv")]


_Sections = ctypes.c_int64 * AXES


class QkNormDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "qheads", "kheads", "headdim", "rotary")] + [
        ("sections", _Sections), ("naxes", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
        ("eps", ctypes.c_float), ("flags", ctypes.c_uint32)]


class QkNormStrides(ctypes.Structure):
    """mamba_qknorm_strides: elements between consecutive token rows (0 = contiguous)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("q", "k", "qo", "ko", "dq", "dk")]


_ready = None
_lock = threading.Lock()


def _library():
    """The native library with the mixer operators' signatures set, once."""
    global _ready
    if _ready is None:
        lib = load_library()
        with _lock:
            if _ready is None:
                P, vp, sz, st = ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
                attn = [P(LinattnDesc), P(LinattnStrides)]
                norm = [P(QkNormDesc), P(QkNormStrides)]
                for name, res, args in [
                        ("mamba_linattn_workspace_size", sz, attn[:1]),
                        ("mamba_linattn_bwd_workspace_size", sz, attn[:1]),
                        ("mamba_linattn_fwd", st, attn + [vp] * 9 + [sz, vp]),
                        ("mamba_linattn_bwd", st, attn + [vp] * 14 + [sz, vp]),
                        ("mamba_linattn_update", st, attn + [vp] * 7),
                        ("mamba_qknorm_fwd", st, norm + [vp] * 9),
                        ("mamba_qknorm_bwd_workspace_size", sz, norm[:1]),
                        ("mamba_qknorm_bwd", st, norm + [vp] * 13 + [sz, vp])]:
                    f = getattr(lib, name)
                    f.restype, f.argtypes = res, args
                _ready = lib
    return _ready


def _heads(t, name, shape, dtype, dev):
    """Row stride of a (..., heads, size) tensor whose token rows may be column
    slices of wider ones; 0 for a contiguous one and for None. The usual
    layouts are recognised without a walk over the axes."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev:
        if t.is_contiguous():
            return 0
        heads, size = shape[-2:]
        step = t.stride()
        row = step[-3]
        if (step[-1] == 1 and step[-2] == size and row >= heads * size and heads > 1
                and (len(shape) == 3 or step[0] == row * shape[1])):
            return row
    s = _row_stride(t, name, shape, dtype, dev, len(shape) - 3)
    # rows apart by less than a row's length share elements
    if s < shape[-2] * shape[-1] and t.numel():
        raise ValueError(f"{name}: rows overlap")
    return s


class _Call:
    """The checked arguments that linear attention's calls share."""

    def __init__(self, who, q, k, v, g, scale, offsets=None, token=False):
        dims = 4 if offsets is None and not token else 3
        what = ("(batch, heads, size)" if token else "(batch, L, heads, size)" if dims == 4 else "(tokens, heads, size)")
        self.io, self.dev = io, dev = _io_of(who, v, dims, f"v must be {what}")
        if not isinstance(q, torch.Tensor) or q.dim() != dims:
            raise ValueError(f"{who}: q must be {what}")
        self.shape, self.qk = shape, qk = v.shape, q.shape
        *lead, H, V = shape
        *other, G, K = qk
        if other != lead:
            raise ValueError(f"q has shape {tuple(qk)}, expected {(*lead, G, K)}")
        if G < 1 or H % G:
            raise ValueError(f"{who}: {G} heads of q and k must divide the {H} of v")
        self.sq, self.sk = _heads(q, "q", qk, io, dev), _heads(k, "k", qk, io, dev)
        self.sv = _heads(v, "v", shape, io, dev)
        flags = 0
        if g is None:
            raise TypeError("g must be a torch.Tensor")
        if isinstance(g, torch.Tensor) and g.dim() == 1:
            _whole(g, "g", (H,), F32, dev)
            flags = HEAD_DECAY
        else:
            _whole(g, "g", (*lead, H), F32, dev)
        if offsets is None:
            batch, seqlen = lead[0], 1 if token else lead[1]
        else:
            if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 1:
                raise ValueError(f"{who}: offsets must be (sequences + 1,)")
            _whole(offsets, "offsets", offsets.shape, torch.int64, dev)
            batch, seqlen = offsets.shape[0] - 1, lead[0]
            flags |= PACKED
        self.state = (batch, H, K, V)
        self.desc = LinattnDesc(batch, seqlen, H, G, K, V, _IO[io], flags, K ** -0.5 if scale is None and K else scale or 0.0)

    def zero_rest(self):
        if self.desc.flags & PACKED:
            self.desc.flags |= ZERO_REST

    def strides(self, so=0, sdq=0, sdk=0, sdv=0):
        return _strides(LinattnStrides, self.sq, self.sk, self.sv, so, sdq, sdk, sdv)


def linear_attn_fwd(q, k, v, g, *, scale=None, h0=None, offsets=None, out=None, last_state=None,
                    return_last_state=True):
    """Linear attention with a decay for each head over whole sequences
    (mamba_linattn_fwd): S_t = exp(g_t) S_{t-1} + k_t v_t^T and
    out_t = scale S_t^T q_t.

    q, k: (batch, L, G, K) and v: (batch, L, H, V), float32 or bfloat16 on a
    GPU, token rows contiguous or column slices of wider ones, H a multiple of
    G; K and V multiples of 8 up to 256. g: the log of the decay, float32,
    (batch, L, H) or (H,). scale: K ** -0.5 without one. h0: (batch, H, K, V)
    float32 or None (zeros). Returns (out, last_state): out as v, and the
    states after the last tokens in float32 (None if not requested).

    With ``offsets`` ((sequences + 1,) int64 on the same device, not
    decreasing) the tensors are (tokens, heads, size), sequence i being rows
    offsets[i] to offsets[i + 1] - 1, and states are per sequence. Rows before
    the first and behind the last sequence are left as they were in an ``out``
    that is given, and are zeros in one that is not."""
    lib = _library()
    c = _Call("linear_attn_fwd", q, k, v, g, scale, offsets)
    _whole(h0, "h0", c.state, F32, c.dev)
    so = _heads(out, "out", c.shape, c.io, c.dev)
    if out is None:
        out = torch.empty_like(v)
        c.zero_rest()
    _whole(last_state, "last_state", c.state, F32, c.dev)
    if last_state is None and return_last_state:
        last_state = _new(c.state, F32, c.dev)
    d = ctypes.byref(c.desc)
    ws, nbytes = _workspace(c.dev, lib.mamba_linattn_workspace_size, d)
    _run(c.dev, lib.mamba_linattn_fwd, d, c.strides(so), _p(q), _p(k), _p(v), _p(g), _p(h0), _p(offsets), _p(out),
         _p(last_state), _p(ws), nbytes)
    return out, last_state


def linear_attn_bwd(q, k, v, g, dout, *, scale=None, h0=None, offsets=None, dlast=None, dq=None, dk=None, dv=None,
                    want_dg=True, want_dh0=True):
    """Gradients of linear_attn_fwd (mamba_linattn_bwd) for dLoss/dout = dout
    and dLoss/d(last_state) = dlast ((batch, H, K, V) float32 or None), from
    the forward's inputs. Returns a dict with dq, dk, dv (as q, k, v, in their
    dtype), dg (as g, None unless want_dg) and dh0 (batch, H, K, V, None unless
    want_dh0) float32. dq, dk and dv may be given, also as column slices of one
    gradient buffer. Packed rows of no sequence are left as they were in those
    that are given, and are zeros in the others."""
    lib = _library()
    c = _Call("linear_attn_bwd", q, k, v, g, scale, offsets)
    so = _heads(dout, "dout", c.shape, c.io, c.dev)
    if dout is None:
        raise TypeError("dout must be a torch.Tensor")
    _whole(h0, "h0", c.state, F32, c.dev)
    _whole(dlast, "dlast", c.state, F32, c.dev)
    make = torch.empty_like
    if dq is None and dk is None and dv is None:
        c.zero_rest()
    elif offsets is not None:
        make = torch.zeros_like
    sdq, sdk = _heads(dq, "dq", c.qk, c.io, c.dev), _heads(dk, "dk", c.qk, c.io, c.dev)
    sdv = _heads(dv, "dv", c.shape, c.io, c.dev)
    dq = make(q) if dq is None else dq
    dk = make(k) if dk is None else dk
    dv = make(v) if dv is None else dv
    dg = make(g) if want_dg else None
    dh0 = _new(c.state, F32, c.dev) if want_dh0 else None
    d = ctypes.byref(c.desc)
    ws, nbytes = _workspace(c.dev, lib.mamba_linattn_bwd_workspace_size, d)
    _run(c.dev, lib.mamba_linattn_bwd, d, c.strides(so, sdq, sdk, sdv), _p(q), _p(k), _p(v), _p(g), _p(h0),
         _p(offsets), _p(dout), _p(dlast), _p(dq), _p(dk), _p(dv), _p(dg), _p(dh0), _p(ws), nbytes)
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dh0": dh0}


def linear_attn_update(state, q, k, v, g, *, scale=None, out=None):
    """One decode token of linear attention (mamba_linattn_update): advances
    ``state`` (batch, H, K, V) float32 in place and returns out (batch, H, V).
    q, k: (batch, G, K), v: (batch, H, V), contiguous or column slices; g:
    (batch, H) or (H,) float32."""
    lib = _library()
    c = _Call("linear_attn_update", q, k, v, g, scale, token=True)
    if state is None:
        raise TypeError("state must be a torch.Tensor")
    _whole(state, "state", c.state, F32, c.dev)
    so = _heads(out, "out", c.shape, c.io, c.dev)
    if out is None:
        out = torch.empty_like(v)
    _run(c.dev, lib.mamba_linattn_update, ctypes.byref(c.desc), c.strides(so), _p(state), _p(q), _p(k), _p(v), _p(g),
         _p(out))
    return out


class _QkCall:
    """The checked arguments that the norm's and rotation's calls share."""

    def __init__(self, who, q, k, positions, freqs, q_weight, k_weight, eps, sections, interleaved):
        self.io, self.dev = _io_of(who, q, 3, "q must be (tokens, heads, size)")
        io, dev = self.io, self.dev
        n, hq, dim = q.shape
        if k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 3):
            raise ValueError(f"{who}: k must be (tokens, heads, size)")
        hk = 0 if k is None else k.shape[1]
        self.qs, self.ks = q.shape, (n, hk, dim)
        self.sq, self.sk = _heads(q, "q", self.qs, io, dev), _heads(k, "k", self.ks, io, dev)
        if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
            raise ValueError(f"{who}: freqs must be (pairs,)")
        pairs = freqs.shape[0]
        _whole(freqs, "freqs", (pairs,), F32, dev)
        if sections is None:
            sections = (pairs,)
        else:
            sections = tuple(int(v) for v in sections)
            if not 1 <= len(sections) <= AXES:
                raise ValueError(f"{who}: 1 to {AXES} sections")
        if positions is None:
            raise TypeError("positions must be a torch.Tensor")
        one = len(sections) == 1 and isinstance(positions, torch.Tensor) and positions.dim() == 1
        _whole(positions, "positions", (n,) if one else (len(sections), n), torch.int64, dev)
        _whole(q_weight, "q_weight", (dim,), F32, dev)
        _whole(k_weight, "k_weight", (dim,), F32, dev)
        self.dim = dim
        self.desc = QkNormDesc(n, hq, hk, dim, 2 * pairs, _Sections(*sections), len(sections), _IO[io], eps,
                               INTERLEAVED if interleaved else 0)

    def strides(self, sqo, sko, sdq=0, sdk=0):
        return _strides(QkNormStrides, self.sq, self.sk, sqo, sko, sdq, sdk)


def qk_norm_rope_fwd(q, k, positions, freqs, q_weight=None, k_weight=None, *, eps=1e-6, sections=None,
                     interleaved=False, q_out=None, k_out=None):
    """RMS norm of each query and key head and rotation by the token's position
    in one pass (mamba_qknorm_fwd). q: (tokens, Hq, D), k: (tokens, Hk, D) or
    None, float32 or bfloat16 on a GPU, token rows contiguous or column slices;
    D a multiple of 8 up to 256. positions: (tokens,) int64, or (axes, tokens)
    with ``sections``, the numbers of pairs that each axis turns; freqs:
    (pairs,) float32, radians for each position, pairs a multiple of 4 and at
    most D / 2. The pairs are channels i and i + pairs, or 2 i and 2 i + 1 if
    ``interleaved``; later channels are not turned. q_weight, k_weight: (D,)
    float32 or None (ones). Returns (q_out, k_out); each may be given, also the
    input itself (in place)."""
    lib = _library()
    c = _QkCall("qk_norm_rope_fwd", q, k, positions, freqs, q_weight, k_weight, eps, sections, interleaved)
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    s = c.strides(_heads(q_out, "q_out", c.qs, c.io, c.dev), _heads(k_out, "k_out", c.ks, c.io, c.dev))
    if q_out is None:
        q_out = torch.empty_like(q)
    if k_out is None and k is not None:
        k_out = torch.empty_like(k)
    _run(c.dev, lib.mamba_qknorm_fwd, ctypes.byref(c.desc), s, _p(q), _p(k), _p(positions), _p(freqs), _p(q_weight),
         _p(k_weight), _p(q_out), _p(k_out))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, positions, freqs, q_weight, k_weight, dq_out, dk_out, *, eps=1e-6, sections=None,
                     interleaved=False, dq=None, dk=None):
    """Gradients of qk_norm_rope_fwd (mamba_qknorm_bwd) for dLoss/dq_out and
    dLoss/dk_out, from the forward's inputs. Returns a dict: dq, dk (as q, k)
    and dq_weight, dk_weight (D,) float32 (None for a weight of None). dq and
    dk may be given, also dq_out and dk_out themselves (in place) or column
    slices of one gradient buffer."""
    lib = _library()
    c = _QkCall("qk_norm_rope_bwd", q, k, positions, freqs, q_weight, k_weight, eps, sections, interleaved)
    if (k is None) != (dk_out is None) or dq_out is None:
        raise TypeError("dq_out, and dk_out with k, must be torch.Tensors")
    if k is None and dk is not None:
        raise ValueError("dk without k")
    sqo, sko = _heads(dq_out, "dq_out", c.qs, c.io, c.dev), _heads(dk_out, "dk_out", c.ks, c.io, c.dev)
    s = c.strides(sqo, sko, _heads(dq, "dq", c.qs, c.io, c.dev), _heads(dk, "dk", c.ks, c.io, c.dev))
    if dq is None:
        dq = torch.empty_like(q)
    if dk is None and k is not None:
        dk = torch.empty_like(k)
    dwq = None if q_weight is None else torch.empty_like(q_weight)
    dwk = None if k_weight is None else torch.empty_like(k_weight)
    d = ctypes.byref(c.desc)
    ws, nbytes = _workspace(c.dev, lib.mamba_qknorm_bwd_workspace_size, d)
    _run(c.dev, lib.mamba_qknorm_bwd, d, s, _p(q), _p(k), _p(positions), _p(freqs), _p(q_weight), _p(k_weight),
         _p(dq_out), _p(dk_out), _p(dq), _p(dk), _p(dwq), _p(dwk), _p(ws), nbytes)
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}
