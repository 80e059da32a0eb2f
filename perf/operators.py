"""Gated causal linear attention and the per-head query/key norm with rotation: cases, plain forms, exact values.

The operators, per batch row and head, with q_t, k_t, v_t of d channels and a
log decay g_t <= 0:

  gated_forward    S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale * S_t^T q_t
  gated_backward   the gradients of q, k, v, g and the initial state
  gated_step       the same recurrence for one token, the state updated in place
  qk_norm          y = x / sqrt(mean(x^2) + eps) * weight per head, then pairs of
                   channels rotated by the token's position (a cos/sin table)
  qk_norm_backward the gradients of q, k and of both weights
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
BASE = 10000.0
CHUNK = 64


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the causal language-model shape of the benchmark, trained or prefilled from an empty state
        dict(name="forward_lm_4096", op="gated_forward", B=4, N=4096, H=12, d=64, dtype="bf16", state=False),
        # the 65536-token grid of the benchmark read as one sequence: few (batch, head) pairs, a long axis
        dict(name="forward_long_65536", op="gated_forward", B=4, N=65536, H=6, d=64, dtype="bf16", state=False),
        # a ragged float32 continuation of a prompt from a kept state, head size off the tile sizes
        dict(name="forward_ragged_f32_d48", op="gated_forward", B=2, N=1021, H=5, d=48, dtype="f32", state=True),
        # training at the language-model shape
        dict(name="backward_lm_4096", op="gated_backward", B=4, N=4096, H=12, d=64, dtype="bf16", state=False),
        # training with many narrow heads
        dict(name="backward_heads70_d32", op="gated_backward", B=2, N=16384, H=70, d=32, dtype="bf16", state=False),
        # truncated back-propagation through a carried state, float32, the widest head, odd length
        dict(name="backward_ragged_f32_d128", op="gated_backward", B=1, N=777, H=3, d=128, dtype="f32", state=True),
        # serving: one token for each of 64 sequences
        dict(name="step_64", op="gated_step", B=64, N=1, H=12, d=64, dtype="bf16", state=True),
        # serving one sequence: latency alone
        dict(name="step_1", op="gated_step", B=1, N=1, H=12, d=64, dtype="bf16", state=True),
        # queries and keys of the language-model shape after their projection, positions 0..N-1
        dict(name="qk_norm_lm_4096", op="qk_norm", B=4, N=4096, H=12, Hk=12, d=64, dtype="bf16", pairs=32,
             layout="half", ragged=False),
        # serving: one token of each sequence at a position of its own, fewer key heads
        dict(name="qk_norm_decode_64", op="qk_norm", B=64, N=1, H=12, Hk=4, d=64, dtype="bf16", pairs=32,
             layout="half", ragged=True),
        # training on the 65536-token grid
        dict(name="qk_norm_backward_65536", op="qk_norm_backward", B=4, N=65536, H=6, Hk=6, d=64, dtype="bf16",
             pairs=32, layout="half", ragged=False),
        # float32, an odd length, part of an odd-sized head rotated, neighbouring channels paired
        dict(name="qk_norm_backward_f32_d40", op="qk_norm_backward", B=3, N=517, H=5, Hk=2, d=40, dtype="f32",
             pairs=9, layout="interleaved", ragged=True),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, uniform in its logarithm, odd as often as even."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["gated_forward", "gated_backward", "gated_step", "qk_norm", "qk_norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "gated_step":
        d = rng.choice([32, 48, 64, 64, 96, 128])
        return dict(op=op, B=_spread(rng, 1, 256), N=1, H=rng.randint(1, 16), d=d, dtype=dtype, state=True)
    if op.startswith("gated"):
        d = rng.choice([32, 40, 64, 64, 80, 128])
        N = _spread(rng, 1, 32768)
        H = rng.randint(1, 16)
        B = max(1, min(rng.randint(1, 8), (1 << 20) // (N * H)))
        return dict(op=op, B=B, N=N, H=H, d=d, dtype=dtype, state=rng.random() < 0.5)
    d = rng.choice([32, 40, 64, 64, 80, 128])
    N = _spread(rng, 1, 65536)
    H = rng.randint(1, 16)
    B = max(1, min(rng.randint(1, 32), (1 << 20) // (N * H)))
    pairs = rng.choice([d // 2, d // 2, d // 4, 0])
    return dict(op=op, B=B, N=N, H=H, Hk=rng.choice([H, 1, max(1, H // 2)]), d=d, dtype=dtype, pairs=pairs,
                layout=rng.choice(["half", "interleaved"]), ragged=rng.random() < 0.5)


def work(case):
    B, N, H, d = case["B"], case["N"], case["H"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    tokens, states = B * N * H, 4 * B * H * d * d
    if case["op"] == "gated_forward":   # q, k, v, g in, o out, the state in (if kept) and out
        return {"bytes": tokens * (4 * d + 1) * e + states * (2 if case["state"] else 1), "flops": 4 * tokens * d * d}
    if case["op"] == "gated_backward":  # q, k, v, g, do in, dq, dk, dv, dg out; the state and its gradients
        return {"bytes": tokens * (7 * d + 2) * e + states * (3 if case["state"] else 0), "flops": 10 * tokens * d * d}
    if case["op"] == "gated_step":
        return {"bytes": tokens * (4 * d + 1) * e + 2 * states, "flops": 4 * tokens * d * d}
    rows = B * N * (H + case["Hk"])
    table = 8 * N * case["pairs"] + (4 * B * N if case["ragged"] else 0)
    if case["op"] == "qk_norm":
        return {"bytes": 2 * rows * d * e + table, "flops": 8 * rows * d}
    return {"bytes": 3 * rows * d * e + table, "flops": 16 * rows * d}


# ------------------------------------------------------------------ inputs


def _rotation_table(P, pairs, device):
    """cos and sin of position times BASE^(-i / pairs), worked out in 64 bits, [P, pairs, 2] float32."""
    freq = BASE ** (-torch.arange(pairs, dtype=torch.float64, device=device) / max(pairs, 1))
    angle = torch.arange(P, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    B, N, H, d = case["B"], case["N"], case["H"], case["d"]
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)
    if case["op"].startswith("gated"):
        # heads remember between a few and a few hundred tokens
        bias = torch.linspace(1.0, 6.0, H, device=dev)
        s = {"case": dict(case), "scale": d ** -0.5,
             "q": normal(B, N, H, d).to(dt), "k": normal(B, N, H, d).to(dt), "v": normal(B, N, H, d).to(dt),
             "g": torch.nn.functional.logsigmoid(normal(B, N, H) + bias).to(dt)}
        s["state"] = normal(B, H, d, d) if case["state"] else None
        if case["op"] == "gated_backward":
            s["dout"] = normal(B, N, H, d).to(dt)
            s["dstate_out"] = normal(B, H, d, d) if case["state"] else None
        return s
    Hk, pairs = case["Hk"], case["pairs"]
    P = 4 * N + 1024 if case["ragged"] else N
    s = {"case": dict(case), "q": normal(B, N, H, d).to(dt), "k": normal(B, N, Hk, d).to(dt),
         "q_weight": 1 + 0.1 * normal(d), "k_weight": 1 + 0.1 * normal(d),
         "table": _rotation_table(P, pairs, dev) if pairs else None, "positions": None}
    if case["ragged"] and pairs:   # each row of the batch starts at a position of its own
        start = torch.randint(0, P - N + 1, (B, 1), generator=gen, device=dev)
        s["positions"] = (start + torch.arange(N, device=dev)).to(torch.int32).contiguous()
    if case["op"] == "qk_norm_backward":
        s["dq_out"], s["dk_out"] = normal(B, N, H, d).to(dt), normal(B, N, Hk, d).to(dt)
    return s


# ------------------------------------------------------------------ plain forms


def _recur(q, k, v, g, scale, state):
    """The recurrence over chunks of CHUNK tokens: within a chunk as a masked
    product, between chunks through the states at their ends.  q, k, v
    [B, N, H, d] in 32 bits; g [B, N, H] in 64, where the sums of a long
    sequence's decays are taken.  Returns o [B, N, H, d] and the last state."""
    B, N, H, d = q.shape
    n = -(-N // CHUNK)
    pad = lambda x: torch.cat((x, x.new_zeros(B, n * CHUNK - N, *x.shape[2:])), 1)
    q, k, v = (pad(x).view(B, n, CHUNK, H, d).permute(0, 3, 1, 2, 4) for x in (q, k, v))
    b = pad(g).view(B, n, CHUNK, H).permute(0, 3, 1, 2).cumsum(-1)      # [B, H, n, CHUNK]
    keep = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(keep, b[..., :, None] - b[..., None, :], -math.inf).exp().float()
    inner = ((q @ k.transpose(-1, -2)) * decay) @ v
    total = b[..., -1]
    local = (k * (total[..., None] - b).exp().float()[..., None]).transpose(-1, -2) @ v   # [B, H, n, d, d]
    ends = total.cumsum(-1)
    before = torch.cat((torch.zeros_like(ends[..., :1]), ends), -1)                       # [B, H, n + 1]
    past = torch.ones(n + 1, n, dtype=torch.bool, device=q.device).tril(-1)
    weight = torch.where(past, before[..., :, None] - ends[..., None, :], -math.inf).exp().float()
    states = (weight @ local.reshape(B, H, n, d * d)).view(B, H, n + 1, d, d)
    if state is not None:
        states = states + before.exp().float()[..., None, None] * state[:, :, None]
    outer = b.exp().float()[..., None] * (q @ states[:, :, :n])
    o = scale * (inner + outer)
    return o.permute(0, 2, 3, 1, 4).reshape(B, n * CHUNK, H, d)[:, :N], states[:, :, n]


def _plain_gated_forward(s):
    q, k, v = (s[n].float() for n in "qkv")
    o, state = _recur(q, k, v, s["g"].double(), s["scale"], s["state"])
    return {"out": o.to(s["q"].dtype), "state": state}


def _plain_gated_backward(s):
    q, k, v, do = (s[n].float() for n in ("q", "k", "v", "dout"))
    g, scale, state, last = s["g"].double(), s["scale"], s["state"], s["dstate_out"]
    turn = lambda x: x.transpose(-1, -2) if x is not None else None
    # dq_t = scale S_t do_t: the recurrence with do, v, k in the places of q, k, v
    dq, end = _recur(do, v, k, g, scale, turn(state))
    # the gradient of the state runs backwards: the recurrence over the reversed
    # sequence, each decay one token later
    back = lambda x: x.flip(1)
    later = torch.cat((torch.zeros_like(g[:, :1]), back(g)[:, :-1]), 1)
    dv, first = _recur(back(k), back(q * scale), back(do), later, 1.0, last)
    dk, _ = _recur(back(v), back(do * scale), back(q), later, 1.0, turn(last))
    dk, dv = back(dk), back(dv)
    # dg_t - dg_{t+1} = q_t.dq_t - k_t.dk_t, from <S_N, dS_N> at the end
    step = ((q.double() * dq).sum(-1) - (k.double() * dk).sum(-1)).flip(1).cumsum(1).flip(1)
    if last is not None:
        step = step + (end.transpose(-1, -2).double() * last).sum((-1, -2))[:, None]
    dt = s["q"].dtype
    out = {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "dg": step.to(dt)}
    if state is not None:
        out["dstate"] = g[:, 0].exp().float()[..., None, None] * first
    return out


def _plain_gated_step(s):
    q, k, v = (s[n].float()[:, 0] for n in "qkv")                       # [B, H, d]
    new = s["g"].float()[:, 0].exp()[..., None, None] * s["state"] + k[..., :, None] * v[..., None, :]
    s["state"].copy_(new)
    o = s["scale"] * (q[..., :, None] * new).sum(-2)
    return {"out": o[:, None].to(s["q"].dtype), "state": s["state"]}


def _cos_sin(s):
    """cos and sin of every token, [B or 1, N, 1, pairs]."""
    rows = s["table"][s["positions"].long()] if s["positions"] is not None else s["table"][None, :s["q"].shape[1]]
    return rows[..., 0][:, :, None], rows[..., 1][:, :, None]


def _split(x, pairs, layout):
    if layout == "half":
        return x[..., :pairs], x[..., pairs:2 * pairs], x[..., 2 * pairs:]
    return x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2], x[..., 2 * pairs:]


def _rotate(x, s, sign):
    pairs, layout = s["case"]["pairs"], s["case"]["layout"]
    if not pairs:
        return x
    a, b, rest = _split(x, pairs, layout)
    cos, sin = _cos_sin(s)
    sin = sign * sin
    lo, hi = a * cos - b * sin, a * sin + b * cos
    both = torch.cat((lo, hi), -1) if layout == "half" else torch.stack((lo, hi), -1).flatten(-2)
    return torch.cat((both, rest), -1)


def _plain_qk_norm(s):
    out = {}
    for name in "qk":
        x = s[name].float()
        y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * s[name + "_weight"]
        out[name] = _rotate(y, s, 1.0).to(s[name].dtype)
    return out


def _plain_qk_norm_backward(s):
    out = {}
    for name in "qk":
        x, dz = s[name].float(), s["d%s_out" % name].float()
        r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        dy = _rotate(dz, s, -1.0)
        unit, m = x * r, dy * s[name + "_weight"]
        out["d" + name] = (r * (m - unit * (unit * m).mean(-1, keepdim=True))).to(s[name].dtype)
        out["d%s_weight" % name] = (dy * unit).sum((0, 1, 2), dtype=torch.float64).float()
    return out


# ------------------------------------------------------------------ the framework's calls


def _own(s):
    import token_level_head_block_gb300 as mhla

    op = s["case"]["op"]
    if op == "gated_forward":
        out, state = mhla.gated_forward(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], state=s["state"])
        return {"out": out, "state": state}
    if op == "gated_backward":
        dq, dk, dv, dg, dstate = mhla.gated_backward(s["q"], s["k"], s["v"], s["g"], s["dout"], scale=s["scale"],
                                                     state=s["state"], dstate_out=s["dstate_out"])
        out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg}
        if s["state"] is not None:
            out["dstate"] = dstate
        return out
    if op == "gated_step":
        out = mhla.gated_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"])
        return {"out": out, "state": s["state"]}
    how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, table=s["table"], positions=s["positions"],
               layout=s["case"]["layout"])
    if op == "qk_norm":
        q, k = mhla.qk_norm(s["q"], s["k"], **how)
        return {"q": q, "k": k}
    dq, dk, dq_weight, dk_weight = mhla.qk_norm_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], **how)
    return {"dq": dq, "dk": dk, "dq_weight": dq_weight, "dk_weight": dk_weight}


def run(state):
    if own:
        return _own(state)
    return {"gated_forward": _plain_gated_forward, "gated_backward": _plain_gated_backward,
            "gated_step": _plain_gated_step, "qk_norm": _plain_qk_norm,
            "qk_norm_backward": _plain_qk_norm_backward}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact values


def _exact_gated(s):
    """The recurrence token by token in 64 bits."""
    q, k, v = (s[n].double().transpose(0, 1) for n in "qkv")            # [N, B, H, d]
    a = s["g"].double().transpose(0, 1).exp()[..., None, None]          # [N, B, H, 1, 1]
    N, B, H, d = q.shape
    start = s["state"].double() if s["state"] is not None else torch.zeros(B, H, d, d, dtype=q.dtype, device=q.device)
    if "dout" not in s:
        S, out = start, torch.empty_like(q)
        for t in range(N):
            S = torch.addcmul(a[t] * S, k[t, ..., :, None], v[t, ..., None, :])
            torch.matmul(q[t, ..., None, :], S, out=out[t, ..., None, :])
        return {"out": (s["scale"] * out).transpose(0, 1), "state": S}
    if N * B * H * d * d * 8 > 40e9:    # every state is kept
        return None
    do = s["scale"] * s["dout"].double().transpose(0, 1)
    S = torch.empty(N + 1, B, H, d, d, dtype=q.dtype, device=q.device)
    S[0] = start
    for t in range(N):
        torch.addcmul(a[t] * S[t], k[t, ..., :, None], v[t, ..., None, :], out=S[t + 1])
    dq = (S[1:] @ do[..., None])[..., 0]
    dk, dv, dg = torch.empty_like(k), torch.empty_like(v), torch.empty_like(a)
    dS = s["dstate_out"].double() if s["dstate_out"] is not None else torch.zeros_like(start)
    for t in range(N - 1, -1, -1):
        dS = torch.addcmul(dS, q[t, ..., :, None], do[t, ..., None, :])
        torch.matmul(dS, v[t, ..., None], out=dk[t, ..., None])
        torch.matmul(k[t, ..., None, :], dS, out=dv[t, ..., None, :])
        dS = a[t] * dS
        torch.sum(dS * S[t], (-2, -1), keepdim=True, out=dg[t])
    out = {n: x.transpose(0, 1) for n, x in (("dq", dq), ("dk", dk), ("dv", dv), ("dg", dg[..., 0, 0]))}
    if s["state"] is not None:
        out["dstate"] = dS
    return out


def _exact_norm(s):
    """Norm and rotation in 64 bits, each pair as a complex number; the gradients by the formula of the quotient."""
    case, out = s["case"], {}
    pairs, half = case["pairs"], case["layout"] == "half"
    for name in "qk":
        x, w = s[name].double(), s[name + "_weight"].double()
        d = x.shape[-1]
        first = torch.arange(pairs, device=x.device) if half else torch.arange(0, 2 * pairs, 2, device=x.device)
        second = first + (pairs if half else 1)
        if pairs:
            at = s["positions"].long() if s["positions"] is not None else torch.arange(x.shape[1], device=x.device)[None]
            turn = torch.view_as_complex(s["table"].double())[at][:, :, None]
        length = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
        if case["op"] == "qk_norm":
            z = x / length * w
            if pairs:
                c = torch.complex(z[..., first], z[..., second]) * turn
                z[..., first], z[..., second] = c.real, c.imag
            out[name] = z
            continue
        dy = s["d%s_out" % name].double().clone()
        if pairs:
            c = torch.complex(dy[..., first], dy[..., second]) * turn.conj()
            dy[..., first], dy[..., second] = c.real, c.imag
        out["d%s_weight" % name] = (dy * x / length).sum((0, 1, 2))
        dy = dy * w
        out["d" + name] = dy / length - x * (dy * x).sum(-1, keepdim=True) / (d * length.pow(3))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_gated(s) if case["op"].startswith("gated") else _exact_norm(s)
