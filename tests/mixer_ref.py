"""Plain implementations of the matrix-state mixer's operators in 64 bits, with
the bound that the kernels' arithmetic keeps to for each value: (value, bound)
pairs, to be rounded and compared by block_ref.

u = 2^-24 is half a float32 step. Linear attention: every output is a sum of
terms decay x (q . k) x v, and the reference runs the same recurrence on
magnitudes, so that each bound is a number of roundings times the sum of its
terms' magnitudes:

* additions: t + K + V + 128 of them lie behind any output of step t (steps,
  head sizes, a chunk's own sums), each off by at most 2 u of the magnitude (the
  matrix cores may cut instead of rounding);
* products and factors: 16 u;
* operands of bfloat16 products are float32 values in two parts, each part off
  by half a step of 8 bits: 2^-17 for the scores and for the state, together
  2^-16 (float32 io has none of it);
* a decay e^d, d the sum of some g: d is rounded to float32 and multiplied by a
  rounded log2(e), 2 u |d|, the exponential is off by 2 u, and a decay over many
  chunks is a product of one factor for each, 3 u each. |d| e^d is carried along as a
  recurrence of its own.
"""
import torch

from block_ref import U, d64

SPLIT = {torch.bfloat16: 2.0 ** -16, torch.float32: 0.0}


def scan(q, k, v, g, scale, S, before=None):
    """One sequence forward: per step (value, magnitude, |d| magnitude) of S,
    and of the outputs. q, k: (L, H, K); v: (L, H, V); g: (L, H); S: (H, K, V)."""
    zero = torch.zeros_like(S)
    M, D = S.abs(), zero
    outs, states = [], []
    for t in range(v.shape[0]):
        cut = g[t] <= -104
        e = torch.where(cut, 0.0, g[t].exp())[:, None, None]
        gt = torch.where(cut, 0.0, g[t]).abs()[:, None, None]

        def keep(x):
            return torch.where(cut[:, None, None], zero, x)
        if before is not None:
            before.append((e, keep(S), keep(M), keep(D)))
        own = k[t][:, :, None] * v[t][:, None, :]
        S = e * keep(S) + own
        D = e * (keep(D) + gt * keep(M))
        M = e * keep(M) + own.abs()
        states.append((S, M, D))
        outs.append(tuple((abs(scale) if i else scale) * torch.einsum("hk,hkv->hv", q[t].abs() if i else q[t], x)
                          for i, x in enumerate((S, M, D))))
    return outs, states


def bound(M, D, n, io):
    """n: additions behind the value."""
    chunks = 3 * (n // 32 + 2)
    return M * ((2 * n + 16 + chunks) * U + SPLIT[io]) + 4 * U * D


def _expand(x, H):
    return x.repeat_interleave(H // x.shape[-2], -2)


def _sequences(v, offsets):
    """Index of each sequence's tokens into flattened rows."""
    if offsets is None:
        b, n = v.shape[:2]
        return [torch.arange(i * n, (i + 1) * n) for i in range(b)]
    o = offsets.tolist()
    return [torch.arange(a, max(a, b)) for a, b in zip(o[:-1], o[1:])]


def linattn(q, k, v, g, scale, h0=None, offsets=None, dout=None, dlast=None):
    """Linear attention and, with dout, its gradients: a dict of (value,
    bound) for out, last_state, dq, dk, dv, dg, dh0, before any rounding to an
    output's type. Rows of no sequence are 0 with bound 0."""
    io = v.dtype
    H, G = v.shape[-2], q.shape[-2]
    K, V = q.shape[-1], v.shape[-1]
    rows = v.shape[:-2].numel()
    flat = [d64(x).reshape((rows,) + x.shape[-2:]) for x in (q, k, v)]
    qe, ke, ve = _expand(flat[0], H), _expand(flat[1], H), flat[2]
    fixed = g.dim() == 1
    ge = d64(g).expand(rows, H) if fixed else d64(g).reshape(rows, H)
    do = None if dout is None else d64(dout).reshape(rows, H, V)

    def empty(*shape):
        return [torch.zeros(shape, dtype=torch.float64) for _ in range(2)]
    out, last = empty(rows, H, V), []
    grads = {"dq": empty(rows, H, K), "dk": empty(rows, H, K), "dv": empty(rows, H, V), "dg": empty(rows, H)}
    dh0 = []
    for i, at in enumerate(_sequences(v, offsets)):
        n = len(at)
        S = torch.zeros((H, K, V), dtype=torch.float64) if h0 is None else d64(h0)[i]
        gs = ge[at]
        before = []
        outs, states = scan(qe[at], ke[at], ve[at], gs, scale, S, before)
        N = K + V + 128
        for t, (o, m, d) in enumerate(outs):
            out[0][at[t]], out[1][at[t]] = o, bound(m, d, t + N, io)
        s, m, d = states[-1] if states else (S, S.abs(), torch.zeros_like(S))
        last.append((s, bound(m, d, n + N, io) if states else torch.zeros_like(S)))
        if do is None:
            continue
        dS = torch.zeros((H, K, V), dtype=torch.float64) if dlast is None else d64(dlast)[i]
        M, D = dS.abs(), torch.zeros_like(dS)
        worst = torch.zeros(H, dtype=torch.float64)
        for t in range(n - 1, -1, -1):
            r = at[t]
            own = scale * qe[r][:, :, None] * do[r][:, None, :]
            dS, M = dS + own, M + own.abs()
            _, Sm, Sd = states[t]
            ad = do[r].abs()
            grads["dq"][0][r] = scale * torch.einsum("hkv,hv->hk", states[t][0], do[r])
            grads["dq"][1][r] = bound(abs(scale) * torch.einsum("hkv,hv->hk", Sm, ad), abs(scale) * torch.einsum("hkv,hv->hk", Sd, ad),
                                      t + N, io)
            av, ak = ve[r].abs(), ke[r].abs()
            grads["dk"][0][r] = torch.einsum("hkv,hv->hk", dS, ve[r])
            grads["dk"][1][r] = bound(torch.einsum("hkv,hv->hk", M, av), torch.einsum("hkv,hv->hk", D, av), n - t + N, io)
            grads["dv"][0][r] = torch.einsum("hkv,hk->hv", dS, ke[r])
            grads["dv"][1][r] = bound(torch.einsum("hkv,hk->hv", M, ak), torch.einsum("hkv,hk->hv", D, ak), n - t + N, io)
            e, Sb, Mb, Db = before[t]
            grads["dg"][0][r] = (e * dS * Sb).sum((1, 2))
            # what a chunk's sums and its neighbours' carried-on products hold: at most the
            # largest <|S|, |dS|> of the sequence, formed from both states' terms
            worst = torch.maximum(worst, (M * Sm).sum((1, 2)))
            gt = torch.where(gs[t] <= -104, 0.0, gs[t]).abs()[:, None, None]
            cut = (gs[t] <= -104)[:, None, None]
            dS = torch.where(cut, 0.0, e * dS)
            D = torch.where(cut, 0.0, e * (D + gt * M))
            M = torch.where(cut, 0.0, e * M)
        # at most 16 stretches' sums between two states from which it starts anew, each off
        # by the additions behind both runs and by 104 u at most for its decays
        grads["dg"][1][at] = (16 * worst * ((4 * (n + K + V + 128) + 300) * U + 2 * SPLIT[io]))[None]
        dh0.append((dS, bound(M, D, n + N, io)))

    def pair(x, shape):
        return x[0].reshape(shape), x[1].reshape(shape)

    def shared(x, like):
        both = [p.unflatten(1, (G, H // G)).sum(2).reshape(like.shape) for p in x]
        total = both[0]
        return total, both[1] + (H // G) * U * total.abs() * 2

    def states_of(pairs):
        if not pairs:
            return empty(0, H, K, V)
        return torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])
    res = {"out": pair(out, v.shape), "last_state": states_of(last)}
    if do is None:
        return res
    res["dq"], res["dk"], res["dv"] = shared(grads["dq"], q), shared(grads["dk"], k), pair(grads["dv"], v.shape)
    res["dh0"] = states_of(dh0)
    dg, e = grads["dg"]
    if fixed:
        res["dg"] = dg.sum(0), e.sum(0) + 2 * U * rows * dg.abs().sum(0)
    else:
        res["dg"] = pair((dg, e), g.shape)
    return res


def update(state, q, k, v, g, scale):
    """One token: (value, bound) of out and of the new state."""
    H, K = v.shape[1], q.shape[2]
    q, k, v, s, g = _expand(d64(q), H), _expand(d64(k), H), d64(v), d64(state), d64(g)
    g = g.expand(v.shape[:2])[..., None, None]
    cut = g <= -104
    e = torch.where(cut, 0.0, g.exp())
    kept = torch.where(cut, 0.0, e * torch.where(cut, 0.0, s))
    own = k[..., :, None] * v[..., None, :]
    new = kept + own
    err = kept.abs() * (torch.where(cut, 0.0, g.abs()) * 2 * U + 4 * U) + 2 * U * (kept.abs() + own.abs())
    o = scale * (q[..., None] * new).sum(-2)
    mag = abs(scale) * (q.abs()[..., None] * (new.abs() + err)).sum(-2)
    return {"state": (new, err), "out": (o, abs(scale) * (q.abs()[..., None] * err).sum(-2) + mag * (K + 4) * U)}


def angles(positions, freqs, sections):
    pos = positions.to("cpu", torch.float64).reshape(-1, positions.shape[-1])
    sections = [freqs.numel()] if sections is None else list(sections)
    axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], dtype=torch.long)
    return pos[axis].T * d64(freqs)


def _pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, e, angle, interleaved):
    """x (tokens, heads, D) with error e, its pairs turned by angle (tokens, pairs)."""
    a, b = _pairs(2 * angle.shape[1], interleaved)
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y, ey = x.clone(), e.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    # sine and cosine are off by 2^-23 at most (argument, series and result rounded)
    size = x[..., a].abs() + x[..., b].abs()
    moved = e[..., a] * c.abs() + e[..., b] * s.abs() + 4 * U * size
    ey[..., a] = moved
    ey[..., b] = e[..., b] * c.abs() + e[..., a] * s.abs() + 4 * U * size
    return y, ey


def _norm(x, eps):
    D = x.shape[-1]
    r = ((x * x).mean(-1, keepdim=True) + eps).rsqrt()
    return x * r, r, (D + 2) * U / 2 + 4 * U      # relative error of r


def qknorm(x, weight, positions, freqs, eps, sections=None, interleaved=False, dy=None):
    """Queries or keys: (value, bound) of y, and with dy of dx and dweight."""
    x = d64(x)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if weight is None else d64(weight)
    angle = angles(positions, freqs, sections)
    n, r, er = _norm(x, eps)
    y = n * w
    res = {"y": turn(y, y.abs() * (er + 3 * U), angle, interleaved)}
    if dy is None:
        return res
    D = x.shape[-1]
    dy = d64(dy)
    u, eu = turn(dy, torch.zeros_like(dy), -angle, interleaved)
    wu, ewu = u * w, eu * w.abs() + U * (u * w).abs()
    c = (wu * n).mean(-1, keepdim=True)
    ec = (ewu * n.abs() + (wu * n).abs() * (er + (D + 3) * U)).mean(-1, keepdim=True)
    dx = r * (wu - n * c)
    res["dx"] = (dx, r * (ewu + n.abs() * ec + (wu.abs() + (n * c).abs()) * (2 * er + 6 * U)))
    part = u * n
    rows = x.shape[0] * x.shape[1]
    res["dweight"] = (part.sum((0, 1)), (eu * n.abs() + part.abs() * (er + 2 * U + (rows + 64) * U)).sum((0, 1)))
    return res
