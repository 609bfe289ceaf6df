"""Cases and plain forms of the token mixer with a matrix state per head.

Two operators that follow each other in a layer. The first makes the mixer's
queries and keys from a projection's rows: a root-mean-square norm of each head
and a rotation of pairs of channels by the token's position (one position, or
several axes that each turn a section of the pairs). The second is linear
attention with a decay for each head: per sequence and head

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,     o_t = scale S_t^T q_t,

with queries and keys shared by groups of heads, for whole sequences (of one
length, or packed one after another), for their gradients, and for a single
token whose states are updated in place. Each case is one call, or a forward
and its backward for the training ones.

``run`` computes a case in elementary torch operations (``own`` false) or by
this package's kernels (``own`` true); ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
SPAN = 128               # tokens that the plain form joins by one matrix


def listed():
    return [
        # One sequence's next token, where a call's latency is nearly all there is.
        {"name": "step_1", "op": "step", "batch": 1, "heads": 40, "groups": 40, "K": 128, "V": 128, "io": "bf16",
         "fixed": False},
        # A full decode batch: every state is read and written once.
        {"name": "step_256", "op": "step", "batch": 256, "heads": 40, "groups": 40, "K": 128, "V": 128, "io": "bf16",
         "fixed": False},
        # Prefill of a batch of prompts, a decay for each token and head.
        {"name": "prompt", "op": "prompt", "batch": 8, "len": 2048, "lens": "", "heads": 40, "groups": 40, "K": 128,
         "V": 128, "io": "bf16", "fixed": False, "state": False},
        # Packed prompts of different lengths continued from states, keys shared by ten heads, fixed decays.
        {"name": "prompt_packed", "op": "prompt", "batch": 0, "len": 0, "lens": "4096,17,0,1301,1,2500,640,777",
         "heads": 80, "groups": 8, "K": 128, "V": 64, "io": "bf16", "fixed": True, "state": True},
        # One very long document: few heads, many tokens.
        {"name": "prompt_long", "op": "prompt", "batch": 1, "len": 131072, "lens": "", "heads": 20, "groups": 20,
         "K": 128, "V": 128, "io": "bf16", "fixed": False, "state": True},
        # A training step, every gradient.
        {"name": "train", "op": "train", "batch": 8, "len": 2048, "lens": "", "heads": 20, "groups": 20, "K": 128,
         "V": 128, "io": "bf16", "fixed": False, "state": False},
        # A training step on packed documents in fp32, at head sizes that fill no tile, gradients of shared keys.
        {"name": "train_odd", "op": "train", "batch": 0, "len": 0, "lens": "301,1,0,64,515", "heads": 6, "groups": 2,
         "K": 40, "V": 72, "io": "f32", "fixed": False, "state": True},
        # A training step with a learned decay for each head and keys shared by two heads.
        {"name": "train_fixed", "op": "train", "batch": 4, "len": 1000, "lens": "", "heads": 32, "groups": 16,
         "K": 64, "V": 128, "io": "bf16", "fixed": True, "state": False},
        # The norm and rotation for a decode batch at far positions.
        {"name": "turn_64", "op": "turn", "tokens": 64, "hq": 40, "hk": 40, "dim": 128, "rot": 128, "axes": 1,
         "inter": False, "io": "bf16"},
        # The same for a prefill.
        {"name": "turn_16384", "op": "turn", "tokens": 16384, "hq": 40, "hk": 8, "dim": 128, "rot": 128, "axes": 1,
         "inter": False, "io": "bf16"},
        # The norm and rotation with their gradients in a training step.
        {"name": "turn_train", "op": "turn_train", "tokens": 16384, "hq": 20, "hk": 20, "dim": 128, "rot": 64,
         "axes": 1, "inter": False, "io": "bf16"},
        # The same in fp32 for video tokens (time, height, width), neighbouring channels as pairs, odd sizes.
        {"name": "turn_train_video", "op": "turn_train", "tokens": 1521, "hq": 6, "hk": 2, "dim": 80, "rot": 80,
         "axes": 3, "inter": True, "io": "f32"},
    ]


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["step", "prompt", "prompt", "train", "train", "turn", "turn_train"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("turn", "turn_train"):
        dim = rng.choice([64, 128, 128, 256, 80, 96, 40])
        hk = rng.choice([1, 2, 4, 5, 8, 16, 20])
        hq = hk * rng.choice([1, 1, 2, 3, 4])
        axes = rng.choice([1, 1, 1, 2, 3])
        return {"op": op, "tokens": between(1, min(16384, (1 << 26) // (dim * (hq + hk)))), "hq": hq, "hk": hk,
                "dim": dim, "rot": dim if rng.random() < 0.6 else dim // 16 * 8, "axes": axes,
                "inter": rng.random() < 0.4, "io": io}
    K, V = rng.choice([32, 64, 64, 128, 128, 256, 96, 40]), rng.choice([32, 64, 64, 128, 128, 256, 80, 24])
    groups = rng.choice([1, 2, 3, 4, 5, 8, 16])
    heads = groups * rng.choice([1, 1, 1, 2, 3, 5])
    case = {"op": op, "heads": heads, "groups": groups, "K": K, "V": V, "io": io, "fixed": rng.random() < 0.3}
    if op == "step":
        return {**case, "batch": between(1, min(512, (1 << 27) // (heads * K * V)))}
    most = (1 << (26 if op == "prompt" else 24)) // (heads * max(K, V))  # tokens
    case.update({"batch": 0, "len": 0, "lens": "", "state": rng.random() < 0.5})
    if rng.random() < 0.5:
        case["len"] = between(1, min(most, 65536 if op == "prompt" else 4096))
        case["batch"] = between(1, max(1, min(16, most // case["len"])))
    else:
        n = between(1, 12)
        case["lens"] = ",".join(str(0 if rng.random() < 0.05 else between(1, max(1, min(8192, most // n))))
                                for _ in range(n))
        if not any(int(v) for v in case["lens"].split(",")):
            case["lens"] += ",7"
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    io, op = IO[case["io"]], case["op"]

    def normal(*shape, io=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(io)

    s = {"op": op}
    if op in ("turn", "turn_train"):
        n, hq, hk, dim, rot, axes = (case[k] for k in ("tokens", "hq", "hk", "dim", "rot", "axes"))
        rows = normal(n, (hq + 2 * hk) * dim, io=io, scale=1.5)  # a projection's rows: queries, keys, values
        s["q"] = rows[:, :hq * dim].unflatten(1, (hq, dim))
        s["k"] = rows[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
        at = torch.arange(n, device="cuda")
        start = int(torch.randint(0, 1 << 20, (1,), generator=gen, device="cuda"))
        if axes == 1:
            s["pos"], s["sections"] = at + start, None
        else:  # frames of 24 x 32 patches
            s["pos"] = torch.stack([at // 768 + start % 4096, at // 32 % 24, at % 32][-axes:]).contiguous()
            half = rot // 2
            s["sections"] = (half - 2 * (half // 3), half // 3, half // 3) if axes == 3 else (half - half // 2, half // 2)
        s["freqs"] = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        s["wq"], s["wk"] = 1.0 + normal(dim, scale=0.1), 1.0 + normal(dim, scale=0.1)
        s["inter"] = case["inter"]
        if op == "turn_train":
            s["dq"], s["dk"] = normal(n, hq, dim, io=io), normal(n, hk, dim, io=io)
        return s
    H, G, K, V = case["heads"], case["groups"], case["K"], case["V"]
    s["scale"] = K ** -0.5
    lens = [int(v) for v in case["lens"].split(",")] if case.get("lens") else None
    if op == "step":
        lead, n = (case["batch"],), case["batch"]
    elif lens is None:
        lead, n = (case["batch"], case["len"]), case["batch"]
    else:
        lead, n = (sum(lens),), len(lens)
        s["lens"] = lens
        s["offsets"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], device="cuda", dtype=torch.int64)
    s["q"], s["k"], s["v"] = normal(*lead, G, K, io=io), normal(*lead, G, K, io=io), normal(*lead, H, V, io=io)
    # memories from a few tokens to some thousands
    s["g"] = -torch.exp(torch.rand(H, generator=gen, device="cuda") * 7.0 - 8.0)
    if not case["fixed"]:
        s["g"] = s["g"] * torch.nn.functional.softplus(normal(*lead, H))
    if op == "step":
        s["state"] = normal(n, H, K, V)
        return s
    s["h0"] = normal(n, H, K, V) if case["state"] else None
    if op == "train":
        s["dout"] = normal(*lead, H, V, io=io)
        s["dlast"] = normal(n, H, K, V) if case["state"] else None
    return s


def run(s):
    return OWN[s["op"]](s) if own else PLAIN[s["op"]](s)


# ---- by this package's kernels ----

def own_step(s):
    from selective_state_space_56_amd import linear_attn_update
    return linear_attn_update(s["state"], s["q"], s["k"], s["v"], s["g"], scale=s["scale"]), s["state"]


def own_prompt(s):
    from selective_state_space_56_amd import linear_attn_fwd
    return linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], h0=s["h0"], offsets=s.get("offsets"))


def own_train(s):
    from selective_state_space_56_amd import linear_attn_bwd, linear_attn_fwd
    q, k, v, g = s["q"], s["k"], s["v"], s["g"]
    more = {"scale": s["scale"], "h0": s["h0"], "offsets": s.get("offsets")}
    out, last = linear_attn_fwd(q, k, v, g, **more)
    d = linear_attn_bwd(q, k, v, g, s["dout"], dlast=s["dlast"], want_dh0=s["h0"] is not None, **more)
    return out, last, d["dq"], d["dk"], d["dv"], d["dg"], d["dh0"]


def own_turn(s):
    from selective_state_space_56_amd import qk_norm_rope_fwd
    return qk_norm_rope_fwd(s["q"], s["k"], s["pos"], s["freqs"], s["wq"], s["wk"], eps=EPS, sections=s["sections"],
                            interleaved=s["inter"])


def own_turn_train(s):
    from selective_state_space_56_amd import qk_norm_rope_bwd, qk_norm_rope_fwd
    args, more = (s["q"], s["k"], s["pos"], s["freqs"], s["wq"], s["wk"]), {
        "eps": EPS, "sections": s["sections"], "interleaved": s["inter"]}
    q, k = qk_norm_rope_fwd(*args, **more)
    d = qk_norm_rope_bwd(*args, s["dq"], s["dk"], **more)
    return q, k, d["dq"], d["dk"], d["dq_weight"], d["dk_weight"]


OWN = {"step": own_step, "prompt": own_prompt, "train": own_train, "turn": own_turn, "turn_train": own_turn_train}


# ---- in elementary operations, 32 bits throughout, rounded once at the end ----

def padded(s, x):
    """Packed rows as (sequences, longest rounded up to whole spans, ...), zeros behind each one."""
    lens = s.get("lens") or [x.shape[1]] * x.shape[0]
    most = max(SPAN, -(-max(lens) // SPAN) * SPAN)
    if "lens" in s:
        at = s["offsets"][:-1, None] + torch.arange(most, device=x.device)
        live = at < s["offsets"][1:, None]
        x = x[at.clamp(max=x.shape[0] - 1)] * live.view(*live.shape, *[1] * (x.dim() - 1))
    else:
        x = torch.nn.functional.pad(x, [0, 0] * (x.dim() - 2) + [0, most - x.shape[1]])
    return x


def unpadded(s, x, like):
    if "lens" not in s:
        return x[:, :like.shape[1]]
    row = torch.arange(like.shape[0], device=x.device)
    seq = torch.searchsorted(s["offsets"], row, right=True) - 1
    return x[seq, row - s["offsets"][seq]]


def spans(x):
    """(n, L, H, ...) as (n, H, L / SPAN, SPAN, ...)."""
    return x.unflatten(1, (-1, SPAN)).movedim(3, 1)


def unspans(x):
    return x.movedim(1, 3).flatten(1, 2)


def wide(s, x):
    """fp32, padded, heads of a group beside each other, in spans."""
    return spans(padded(s, x).float().repeat_interleave(s["v"].shape[-2] // x.shape[-2], -2))


def gates(s):
    """The log decays of every padded token (n, L, H), in 64 bits."""
    g = s["g"].double()
    g = g.expand(s["v"].shape[:-1]) if g.dim() == 1 else g
    return padded(s, g)


def mix(q, k, v, g, first):
    """S_t = exp(g_t) S_{t-1} + k_t v_t^T and S_t^T q_t over spans: the outputs, the states that enter each
    span and the last one; and what else the gradients of the decays take."""
    ell = spans(g).cumsum(-1)
    total = ell[..., -1]
    near = (ell[..., :, None] - ell[..., None, :]).tril().exp().float().tril()
    from_start, to_end = ell.exp().float(), (total[..., None] - ell).exp().float()
    part = (k * to_end[..., None]).transpose(-1, -2) @ v
    upto = torch.cat([torch.zeros_like(total[..., :1]), total.cumsum(-1)], -1)   # decay before each span's start
    far = (upto[..., :, None] - upto[..., None, 1:]).tril(-1).exp().float().tril(-1)
    states = (far @ part.flatten(-2)).unflatten(-1, part.shape[-2:])
    if first is not None:
        states = states + upto.exp().float()[..., None, None] * first[:, :, None]
    scores = (q @ k.transpose(-1, -2)) * near
    out = scores @ v + from_start[..., None] * (q @ states[:, :, :-1])
    return out, states[:, :, :-1], states[:, :, -1], (near, from_start, to_end, total)


def plain_step(s):
    q, k, v = (s[n].float().repeat_interleave(s["v"].shape[1] // s[n].shape[1], 1) for n in "qkv")
    g = s["g"].expand(v.shape[:2])
    s["state"].copy_(g.exp()[..., None, None] * s["state"] + k[..., :, None] * v[..., None, :])
    out = s["scale"] * (q[..., None, :] @ s["state"])[..., 0, :]
    return out.to(s["v"].dtype), s["state"]


def plain_prompt(s):
    out, _, last, _ = mix(wide(s, s["q"]) * s["scale"], wide(s, s["k"]), wide(s, s["v"]), gates(s), s["h0"])
    return unpadded(s, unspans(out), s["v"]).to(s["v"].dtype), last


def plain_train(s):
    io, G = s["v"].dtype, s["q"].shape[-2]
    q, k, v, dout, g = wide(s, s["q"]) * s["scale"], wide(s, s["k"]), wide(s, s["v"]), wide(s, s["dout"]), gates(s)
    out, before, last, (near, from_start, to_end, total) = mix(q, k, v, g, s["h0"])

    def back(x):
        return x.flip(2, 3)

    def turned(x):
        return None if x is None else x.transpose(-1, -2)

    # the same map with other operands, and with time reversed: a step's decay then lies behind it
    later = torch.cat([torch.zeros_like(g[:, :1]), g.flip(1)[:, :-1]], 1)
    dq = mix(dout, v, k, g, turned(s["h0"]))[0] * s["scale"]
    dk = back(mix(back(v), back(dout), back(q), later, turned(s["dlast"]))[0])
    dv, behind, first, _ = mix(back(k), back(q), back(dout), later, s["dlast"])
    dv = back(dv)
    behind = (behind * spans(later)[..., 0].exp().float()[..., None, None]).flip(2)  # gradients of the states leaving each span
    # a decay's gradient: exp(g_t) <dS_t, S_{t-1}>, from what enters, leaves and stays within its span
    through = total.exp().float() * (before * behind).sum((-1, -2))
    leaves = to_end * ((v @ turned(behind)) * k).sum(-1)
    enters = from_start * ((dout @ turned(before)) * q).sum(-1)
    within = ((q @ turned(k)) * (dout @ turned(v)) * near).tril(-1)
    stays = enters + within.sum(-1) - within.sum(-2)
    stays, leaves = stays.double(), leaves.double()
    dg = through[..., None] + (leaves.cumsum(-1) - leaves) + stays.flip(-1).cumsum(-1).flip(-1)
    dg = unpadded(s, unspans(dg), s["v"])
    dg = dg.sum(tuple(range(dg.dim() - 1))) if s["g"].dim() == 1 else dg
    dh0 = None if s["h0"] is None else g[:, 0].exp().float()[..., None, None] * first

    def shared(x, like):
        x = unpadded(s, unspans(x), like)
        return x.unflatten(-2, (G, -1)).sum(-2).to(io)

    return (unpadded(s, unspans(out), s["v"]).to(io), last, shared(dq, s["q"]), shared(dk, s["k"]),
            unpadded(s, unspans(dv), s["v"]).to(io), dg.float(), dh0)


def angles(s):
    """Cosine and sine per token and pair of channels."""
    pos = s["pos"].double()
    if s["sections"] is not None:
        axis = torch.arange(len(s["sections"])).repeat_interleave(torch.tensor(s["sections"])).to(pos.device)
        pos = pos[axis].T
    else:
        pos = pos[:, None]
    a = pos * s["freqs"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]


def rotated(x, cos, sin, inter):
    rot = 2 * cos.shape[-1]
    turn, rest = x[..., :rot], x[..., rot:]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if inter else (turn[..., :rot // 2], turn[..., rot // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    turn = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turn, rest], -1)


def normed(x):
    x = x.float()
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * rstd, rstd


def plain_turn(s):
    cos, sin = angles(s)
    return tuple(rotated(normed(s[n])[0] * s["w" + n], cos, sin, s["inter"]).to(s[n].dtype) for n in "qk")


def plain_turn_train(s):
    cos, sin = angles(s)
    grads = []
    for n in "qk":
        hat, rstd = normed(s[n])
        dy = rotated(s["d" + n].float(), cos, -sin, s["inter"])
        u = dy * s["w" + n]
        grads.append(((u - hat * (u * hat).mean(-1, keepdim=True)) * rstd).to(s[n].dtype))
        grads.append((dy * hat).sum((0, 1)))
    dq, dwq, dk, dwk = grads
    return (*plain_turn(s), dq, dk, dwq, dwk)


PLAIN = {"step": plain_step, "prompt": plain_prompt, "train": plain_train, "turn": plain_turn,
         "turn_train": plain_turn_train}


# ---- what a pass cannot do without ----

def work(case):
    op, eb = case["op"], 2 if case["io"] == "bf16" else 4
    if op in ("turn", "turn_train"):
        n, heads, dim = case["tokens"], case["hq"] + case["hk"], case["dim"]
        small = 8 * n * case["axes"] + 2 * case["rot"] + 8 * dim
        passes, flops = (5, 26) if op == "turn_train" else (2, 9)
        return {"bytes": n * heads * dim * eb * passes + small + 8 * dim * (passes > 2),
                "flops": n * heads * dim * flops + n * case["rot"] * 30}
    H, G, K, V = case["heads"], case["groups"], case["K"], case["V"]
    lens = [int(v) for v in case["lens"].split(",")] if case.get("lens") else None
    n = len(lens) if lens else case["batch"]
    tokens = n if op == "step" else sum(lens) if lens else case["batch"] * case["len"]
    state, gate = n * H * K * V * 4, 4 * H * (1 if case["fixed"] else tokens)
    one = tokens * (2 * G * K + H * V) * eb  # queries, keys and values, or their gradients
    flops = tokens * H * K * V
    if op == "step":
        return {"bytes": one + tokens * H * V * eb + gate + 2 * state, "flops": 6 * flops}
    total = one + tokens * H * V * eb + gate + state * (1 + case["state"])
    if op == "prompt":
        return {"bytes": total, "flops": 5 * flops}
    total += one + tokens * H * V * eb + gate + state * 2 * case["state"]
    return {"bytes": total, "flops": 18 * flops}


# ---- from the definitions, in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s)


def rows_of(s):
    """For packed sequences: where each sequence's tokens are, (sequences, longest), -1 for none."""
    most = max(s["lens"])
    at = torch.full((len(s["lens"]), most), -1, dtype=torch.long)
    row = 0
    for i, n in enumerate(s["lens"]):
        at[i, :n] = torch.arange(row, row + n)
        row += n
    return at.cuda()


def by_sequence(s, x, at):
    """64 bits, (tokens, sequences, heads, ...); 0 where a sequence has ended."""
    H = s["v"].shape[-2]
    if x.dim() == 1:  # decays that are the same for every token
        lead = (s["v"].shape[:2] if at is None else at.shape)
        x = x.double().expand(*lead, H) * (1 if at is None else (at >= 0)[..., None])
        return x.transpose(0, 1).contiguous()
    x = x.double()
    if at is not None:
        x = torch.cat([x, torch.zeros_like(x[:1])])[at]
    if x.dim() == 4 and x.shape[2] != H:
        x = x[:, :, torch.arange(H, device=x.device) // (H // x.shape[2])]
    return x.transpose(0, 1).contiguous()


def to_rows(s, x, at, like):
    x = x.transpose(0, 1)
    if at is None:
        return x
    out = torch.zeros((like.shape[0],) + x.shape[2:], dtype=x.dtype, device=x.device)
    out[at[at >= 0]] = x[at >= 0]
    return out


def exact_step(s):
    H = s["v"].shape[1]
    g = s["g"].double()
    pick = torch.arange(H, device=g.device) // (H // s["q"].shape[1])
    S = s["state"].double() * torch.exp(g.expand(s["v"].shape[:2]))[:, :, None, None]
    S = S + torch.einsum("bhk,bhv->bhkv", s["k"].double()[:, pick], s["v"].double())
    return (S * s["q"].double()[:, pick][..., None]).sum(2) * s["scale"], S


def walk(k, v, g, S, t):
    return torch.addcmul(S * g[t].exp()[..., None, None], k[t][..., :, None], v[t][..., None, :])


def exact_parts(s):
    at = rows_of(s) if "lens" in s else None
    q, k, v, g = (by_sequence(s, s[n], at) for n in "qkvg")
    n, H = v.shape[1:3]
    S = s["h0"].double() if s["h0"] is not None else v.new_zeros(n, H, k.shape[-1], v.shape[-1])
    return at, q, k, v, g, S


def exact_prompt(s):
    at, q, k, v, g, S = exact_parts(s)
    out = torch.empty_like(v)
    for t in range(v.shape[0]):
        S = walk(k, v, g, S, t)
        out[t] = (q[t][..., None, :] @ S)[..., 0, :]
    return to_rows(s, out * s["scale"], at, s["v"]), S


def exact_train(s):
    at, q, k, v, g, S = exact_parts(s)
    do = by_sequence(s, s["dout"], at)
    L, every = v.shape[0], 64
    out, dq, dk, dv, dg = (torch.empty_like(x) for x in (v, k, k, v, g))
    marks = []
    for t in range(L):
        if t % every == 0:
            marks.append(S)
        S = walk(k, v, g, S, t)
        out[t] = (q[t][..., None, :] @ S)[..., 0, :] * s["scale"]
        dq[t] = (S @ do[t][..., None])[..., 0] * s["scale"]
    dS = torch.zeros_like(S) if s["dlast"] is None else s["dlast"].double()
    for c in range(len(marks) - 1, -1, -1):
        seen = [marks[c]]  # the states before each step
        for t in range(c * every, min(L, (c + 1) * every) - 1):
            seen.append(walk(k, v, g, seen[-1], t))
        for t in range(min(L, (c + 1) * every) - 1, c * every - 1, -1):
            dS = dS + q[t][..., :, None] * do[t][..., None, :] * s["scale"]
            dk[t] = (dS @ v[t][..., None])[..., 0]
            dv[t] = (k[t][..., None, :] @ dS)[..., 0, :]
            dS = dS * g[t].exp()[..., None, None]
            dg[t] = (dS * seen[t - c * every]).sum((-1, -2))
    G = s["q"].shape[-2]
    dq, dk = (to_rows(s, x.unflatten(2, (G, -1)).sum(3), at, s["q"]) for x in (dq, dk))
    dg = to_rows(s, dg, at, s["v"])
    if s["g"].dim() == 1:
        dg = dg.flatten(0, -2).sum(0)
    return (to_rows(s, out, at, s["v"]), S, dq, dk, to_rows(s, dv, at, s["v"]), dg,
            None if s["h0"] is None else dS)


def turn_table(s, sign=1.0):
    """A rotation's matrix entries per token: pairs of channels, cosine, sine."""
    f, half = s["freqs"].double(), s["freqs"].numel()
    pos = s["pos"].double().reshape(-1, s["q"].shape[0])
    where = [0] * half if s["sections"] is None else [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    angle = torch.stack([pos[where[i]] * f[i] for i in range(half)], 1)
    first = [2 * i if s["inter"] else i for i in range(half)]
    second = [2 * i + 1 if s["inter"] else i + half for i in range(half)]
    return first, second, torch.cos(angle)[:, None], sign * torch.sin(angle)[:, None]


def turn64(x, table):
    first, second, c, sn = table
    y = x.clone()
    y[..., first] = x[..., first] * c - x[..., second] * sn
    y[..., second] = x[..., second] * c + x[..., first] * sn
    return y


def exact_turn(s):
    table, got = turn_table(s), []
    for n in "qk":
        x = s[n].double()
        got.append(turn64(x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * s["w" + n].double(), table))
    return tuple(got)


def exact_turn_train(s):
    table, dx, dw = turn_table(s, -1.0), [], []
    for n in "qk":
        x, w = s[n].double(), s["w" + n].double()
        dy = turn64(s["d" + n].double(), table)
        r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        dx.append(dy * w * r - x * r ** 3 * (dy * w * x).sum(-1, keepdim=True) / x.shape[-1])
        dw.append((dy * x * r).flatten(0, 1).sum(0))
    return (*exact_turn(s), *dx, *dw)


EXACT = {"step": exact_step, "prompt": exact_prompt, "train": exact_train, "turn": exact_turn,
         "turn_train": exact_turn_train}
