"""Plain implementations of the block operators in 64 bits, with the bound
that float32 arithmetic keeps to for each value: (value, bound) pairs.

u = 2^-24 is half a float32 step. The bounds follow the formulas operation by
operation: one u per add, multiply or fma, 2 u (one step) for a hardware
exponential, reciprocal or root; an exponent's argument error of |v| u becomes
a relative error of the same size of the result. Sums of n terms in any order
are off by at most n u times the sum of the magnitudes (a kernel's own chains are
shorter). An output rounded to b bits of precision adds half a step of it.
"""
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rounded(pair, dtype):
    """The bound of a value stored in `dtype`: half a step of what is rounded,
    and of the smallest normal number below it."""
    v, e = pair
    return v, e + HALF[dtype] * (v.abs() + e) + torch.finfo(dtype).tiny * HALF[dtype] * 2


def assert_within(name, got, pair):
    v, e = pair
    got = got.detach().to("cpu", torch.float64)
    assert got.shape == v.shape, (name, got.shape, v.shape)
    if got.numel() == 0:
        return
    bad = ~((got - v).abs() <= e)
    both = (got.isnan() & v.isnan()) | (got == v)
    bad &= ~both
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside; first at {at}: got {float(got[at])!r}, "
                             f"expected {float(v[at])!r} +- {float(e[at])!r}")


def d64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def sigmoid(v):
    """1 / (1 + e^-v) and its relative error."""
    return torch.sigmoid(v), (v.abs().clamp(max=700.0) + 6) * U


def _gates(r, g, A, reset):
    sr, esr = sigmoid(r)
    sg, esg = sigmoid(g)
    v = A * sr
    a = torch.exp(v)
    ea = v.abs() * (esr + 2 * U) + 3 * U                     # relative error of a
    w2 = -torch.expm1(2 * v)
    small = -2 * v < 0.25
    ew = torch.where(small, (esr + U) / 2 + 4 * U, (a * a * ea + U) / w2.clamp(min=1e-300) + 2 * U) + 2 * U
    w = w2.sqrt()
    if reset is not None:
        on = reset.to("cpu").bool()[..., None].expand_as(a)
        a, w = a.masked_fill(on, 0.0), w.masked_fill(on, 1.0)
        ea, ew = ea.masked_fill(on, 0.0), ew.masked_fill(on, 0.0)
    return sr, esr, sg, esg, a, ea, w, ew


def gated(x, r, g, A, h0=None, reset=None, dout=None, dlast=None):
    """The gated linear recurrence and, with dout, its gradients: a dict of
    (value, bound) for out, last_state, before (the states entering each
    step), dx, dr, dg, dA, dh0, before any rounding to an output's type."""
    x, r, g, A = d64(x), d64(r), d64(g), d64(A)
    batch, L, dim = x.shape
    zero = torch.zeros((batch, dim), dtype=torch.float64)
    sr, esr, sg, esg, a, ea, w, ew = _gates(r, g, A, reset)
    b = w * sg * x
    eb = b.abs() * (ew + esg + 3 * U)
    h = zero if h0 is None else d64(h0)
    mag, eh = h.abs(), zero.clone()
    out, bound, before, ebefore = [], [], [], []
    on = None if reset is None else reset.to("cpu").bool()

    def keep(t, v):  # a reset drops the state whatever it is
        return v if on is None else torch.where(on[:, t, None], zero, v)

    for t in range(L):
        before.append(h)
        ebefore.append(eh)
        p, pm, pe = keep(t, h), keep(t, mag), keep(t, eh)
        h = a[:, t] * p + b[:, t]
        # the state's own error decays with it; a product of decays over a span
        # adds its factors' errors, one multiplication each
        eh = a[:, t] * pe + a[:, t] * pm * (ea[:, t] + 3 * U) + eb[:, t] + U * h.abs()
        mag = a[:, t] * pm + b[:, t].abs()
        out.append(h)
        bound.append(eh)
    res = {"last_state": (h, eh)}

    def stack(v):
        return torch.stack(v, 1) if v else torch.zeros((batch, 0, dim), dtype=torch.float64)

    res["out"] = (stack(out), stack(bound))
    res["before"] = (stack(before), stack(ebefore))
    if dout is None:
        return res
    dout = d64(dout)
    carry, ec, mc = (zero if dlast is None else d64(dlast)), zero.clone(), (zero if dlast is None else d64(dlast).abs())
    lam, elam = [None] * L, [None] * L
    for t in range(L - 1, -1, -1):
        lam[t] = dout[:, t] + carry
        m = dout[:, t].abs() + mc
        elam[t] = ec + 2 * U * m
        carry = a[:, t] * lam[t]
        ec = a[:, t] * elam[t] + a[:, t] * m * (ea[:, t] + 3 * U)
        mc = a[:, t] * m
    res["dh0"] = (carry, ec)
    lam, elam = stack(lam), stack(elam)
    hb, ehb = res["before"]
    res["dx"] = (lam * w * sg, elam * w * sg + (lam * w * sg).abs() * (ew + esg + 3 * U))
    one_g, eone_g = 1 - sg, sg * esg + U                     # 1 - sigmoid: absolute error
    dg = lam * w * x * sg
    res["dg"] = (dg * one_g, (elam * (w * x * sg).abs() + dg.abs() * (ew + esg + 4 * U)) * one_g + dg.abs() * eone_g)
    slope = torch.where(w > 0, a * a / w.clamp(min=1e-300), torch.zeros_like(w))
    left, right = a * hb, slope * sg * x
    d = left - right
    ed = left.abs() * (ea + 2 * U) + a * ehb + right.abs() * (2 * ea + ew + esg + 7 * U)
    if on is not None:
        off = on[..., None].expand_as(d)
        d, ed = d.masked_fill(off, 0.0), ed.masked_fill(off, 0.0)
    dv, edv = lam * d, elam * d.abs() + lam.abs() * ed + 2 * U * (lam * d).abs()
    one_r, eone_r = 1 - sr, sr * esr + U
    dr = dv * A * sr
    res["dr"] = (dr * one_r, (edv * (A * sr).abs() + dr.abs() * (esr + 4 * U)) * one_r + dr.abs() * eone_r)
    part = dv * sr
    n = batch * L
    res["dA"] = (part.sum((0, 1)), (edv * sr + part.abs() * (esr + U)).sum((0, 1)) + n * U * part.abs().sum((0, 1)))
    return res


def norm(x, weight, residual, eps, dout=None, ds=None):
    """The RMS norm: dict of (value, bound) for sum (exact: the stored
    stream), out and, with dout, dresidual and dweight."""
    stream = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    s, w = d64(stream), d64(weight)
    rows, dim = s.shape
    res = {"sum": stream.to("cpu")}
    ms = (s * s).mean(-1, keepdim=True) + eps
    rstd = ms.rsqrt()
    er = (dim * U + 2 * U) / 2 + 3 * U                       # relative error of rstd
    y = s * rstd * w
    res["out"] = (y, y.abs() * (er + 2 * U))
    if dout is None:
        return res
    dy = d64(dout)
    uu, n = w * dy, s * rstd
    c = (uu * n).mean(-1, keepdim=True)
    ec = (uu * n).abs().mean(-1, keepdim=True) * (dim * U + er + 4 * U)
    ds64 = torch.zeros_like(s) if ds is None else d64(ds)
    d = rstd * (uu - n * c)
    ed = rstd * (uu.abs() * (er + 5 * U) + n.abs() * ec + (n * c).abs() * (2 * er + 5 * U))
    total = ds64 + d
    res["dresidual"] = (total, ed + U * total.abs())
    part = dy * n
    res["dweight"] = (part.sum(0), part.abs().sum(0) * (er + 2 * U + rows * U))
    return res


def conv_bwd(xin, weight, dout, bias=None, state_in=None, dstate_out=None):
    """Gradients of the causal convolution + SiLU: dict of (value, bound)."""
    x, w, dy = d64(xin), d64(weight), d64(dout)
    batch, L, dim = x.shape
    W = w.shape[1]
    first = torch.zeros((batch, W - 1, dim), dtype=torch.float64) if state_in is None else d64(state_in).transpose(1, 2)
    seen = torch.cat([first, x], 1)
    v = torch.zeros_like(x) if bias is None else d64(bias).expand(batch, L, dim).clone()
    mag = v.abs()
    for j in range(W):
        v = v + w[:, j] * seen[:, j:j + L]
        mag = mag + (w[:, j] * seen[:, j:j + L]).abs()
    ev = W * U * mag
    sig = torch.sigmoid(v)
    dv = dy * sig * (1 + v * (1 - sig))
    # silu' moves by at most half of v's error; its own arithmetic as written
    edv = dy.abs() * (0.5 * ev + (1 + v.abs()) * (v.abs() + 12) * U)
    dall, eall = torch.zeros_like(seen), torch.zeros_like(seen)
    for j in range(W):
        dall[:, j:j + L] += w[:, j] * dv
        eall[:, j:j + L] += w[:, j].abs() * (edv + W * U * dv.abs())
    if dstate_out is not None and W > 1:
        add = d64(dstate_out).transpose(1, 2)
        dall[:, L:] += add
        eall[:, L:] += U * (add.abs() + dall[:, L:].abs())
    n = batch * L
    taps = [(dv * seen[:, j:j + L]).sum((0, 1)) for j in range(W)]
    etaps = [((edv + n * U * dv.abs()) * seen[:, j:j + L].abs()).sum((0, 1)) for j in range(W)]
    return {"dxin": (dall[:, W - 1:], eall[:, W - 1:]),
            "dstate_in": (dall[:, :W - 1].transpose(1, 2), eall[:, :W - 1].transpose(1, 2)),
            "dweight": (torch.stack(taps, 1), torch.stack(etaps, 1)),
            "dbias": (dv.sum((0, 1)), (edv + n * U * dv.abs()).sum((0, 1)))}
