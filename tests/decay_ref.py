"""The gradients of linear attention's decays in 64 bits, from the definition, with a
bound for each token and head from that token's own terms.

  dg_t = e^{g_t} <dS_t, S_{t-1}>

u = 2^-24 is half a float32 step. A kernel that works in chunks of C steps
forms it from what crosses step t: the state S_in that enters t's chunk with the
gradient dS_out of the one that leaves it, S_in with the chunk's queries from t
on, its keys before t with dS_out, and pairs of both. With G_S and G_dS the
magnitudes of S_{t-1} and dS_t by these parts (|S_in| decayed plus the chunk's own
|k v^T|, and alike), E_S and E_dS their errors, and D_S, D_dS the same sums with each
term times the decay's exponent:

  bound = e^{g_t} (<G_dS, E_S> + <E_dS, G_S> + (2 (K + V) + 64) u <G_dS, G_S>
          + 4 u (<G_dS, D_S> + <D_dS, G_S>)) + 2^-126 (..)

* E of S_in and dS_out: what float32 states are off by (every addition by 2 u at most
  since the matrix cores may cut, the factors of the chunks that they went through by 3 u each,
  each decay e^d by 4 u |d|), as for last_state and dh0;
* the dot products over K and V channels behind each term: 2 u for each addition;
  64 u for the factors, the sums over a chunk's steps in 64 bits, and roundings between;
* exponents: 4 u |d| of a term, as above;
* float32's range: a factor, a part of a value or a product below the smallest normal number, 2^-126, may
  count as 0, which costs that much times what it is multiplied by. With F the sums over all steps of a run
  of 3 |x| + |x| |y| + 3 |y| + 2 (three parts of either operand times the other, the decay times both, the
  product and the decayed state themselves), without decays: 2^-126 (<F_dS, G_S> + <G_dS, F_S> + <F_dS, F_S>).
Nothing is subtracted: an error that went by the other tokens' terms, however large
these are, would not stay within it.
"""
import torch

from block_ref import U, d64
from mixer_ref import _expand, _sequences

TINY = 2.0 ** -126


def states(x, y, g, S, chunk, reverse=False):
    """A run of S <- e^g S + x y^T over the steps of one sequence, and what bounds it: a list over
    steps of (S, E, G, D, F, the part of S that entered the chunk) before each step (after it, in reverse)."""
    n = x.shape[0]
    err = torch.zeros_like(S)
    mag, exps = S.abs(), torch.zeros_like(S)      # of the whole run: what the state's own errors go by
    F = S.abs() + 1
    G, D, came = S.abs(), torch.zeros_like(S), S  # since the chunk's start
    seen = []
    for i in range(n):
        t = n - 1 - i if reverse else i
        if (t + 1 == n or (t + 1) % chunk == 0) if reverse else t % chunk == 0:
            err = mag * ((2 * (i + 64) + 3 * (i // chunk + 2)) * U) + 4 * U * exps if i else torch.zeros_like(S)
            G, D, came = S.abs(), torch.zeros_like(S), S
        own = x[t][:, :, None] * y[t][:, None, :]
        more = 3 * x[t].abs()[:, :, None] + own.abs() + 3 * y[t].abs()[:, None, :] + 2
        if reverse:
            F = F + more
        cut = (g[t] <= -104)[:, None, None]
        e = torch.where(cut, 0.0, g[t][:, None, None].exp())
        size = torch.where(cut, 0.0, g[t][:, None, None]).abs()

        def decayed(v):
            return torch.where(cut, 0.0, e * v)

        def add():
            return S + own, mag + own.abs(), G + own.abs()
        if reverse:
            S, mag, G = add()
            seen.append((S, err, G, D, F, came))
            exps, D = decayed(exps + size * mag), decayed(D + size * G)
            S, mag, G, err, came = (decayed(x) for x in (S, mag, G, err, came))
        else:
            seen.append((S, err, G, D, F, came))
            exps, D = decayed(exps + size * mag), decayed(D + size * G)
            S, mag, G, err, came = (decayed(x) for x in (S, mag, G, err, came))
            S, mag, G = add()
            F = F + more
    return seen[::-1] if reverse else seen


def dg(q, k, v, g, scale, dout, h0=None, dlast=None, offsets=None, chunk=None, parts=None):
    """(value, bound) of dg, shaped as g, before its rounding. Rows of no sequence are 0.
    parts: a dict that receives what the value is the sum of ("through", "keys", "queries",
    "pairs"), shaped as it."""
    chunk = chunk or (64 if v.dtype == torch.bfloat16 else 32)
    H, K, V = v.shape[-2], q.shape[-1], v.shape[-1]
    rows = v.shape[:-2].numel()
    qe, ke, ve, do = (_expand(d64(x).reshape((rows,) + x.shape[-2:]), H) for x in (q, k, v, dout))
    ge = d64(g).expand(rows, H) if g.dim() == 1 else d64(g).reshape(rows, H)
    value, bound = torch.zeros(rows, H, dtype=torch.float64), torch.zeros(rows, H, dtype=torch.float64)
    split = {n: torch.zeros(rows, H, dtype=torch.float64) for n in ("through", "keys", "queries", "pairs")}
    zero = torch.zeros((H, K, V), dtype=torch.float64)
    for i, at in enumerate(_sequences(v, offsets)):
        if not len(at):
            continue
        gs = ge[at]
        fwd = states(ke[at], ve[at], gs, zero if h0 is None else d64(h0)[i], chunk)
        bwd = states(scale * qe[at], do[at], gs, zero if dlast is None else d64(dlast)[i], chunk, reverse=True)
        for t in range(len(at)):
            (S, ES, GS, DS, FS, Sin), (dS, EdS, GdS, DdS, FdS, dSout) = fwd[t], bwd[t]
            e = torch.where(gs[t] <= -104, 0.0, gs[t].exp())

            def dot(x, y):
                return torch.where(e == 0, 0.0, e * (x * y).sum((1, 2)))
            value[at[t]] = dot(dS, S)
            bound[at[t]] = (dot(GdS, ES) + dot(EdS, GS) + (2 * (K + V) + 64) * U * dot(GdS, GS)
                            + 4 * U * (dot(GdS, DS) + dot(DdS, GS))
                            + torch.where(e == 0, 0.0, TINY * (FdS * GS + GdS * FS + FdS * FS).sum((1, 2))))
            for n, x, y in (("through", dSout, Sin), ("keys", dSout, S - Sin), ("queries", dS - dSout, Sin),
                            ("pairs", dS - dSout, S - Sin)):
                split[n][at[t]] = dot(x, y)
    if parts is not None:
        parts.update({n: x.sum(0) if g.dim() == 1 else x.reshape(g.shape) for n, x in split.items()})
    if g.dim() == 1:  # a sum for each chunk is rounded, and they are added in float32
        n = rows // chunk + (v.shape[0] if offsets is None else len(offsets))
        return value.sum(0), bound.sum(0) + (2 * n + 4) * U * value.abs().sum(0)
    return value.reshape(g.shape), bound.reshape(g.shape)
