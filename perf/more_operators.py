"""The gated delta rule and the projections around it: cases, plain forms, exact values.

The operators, per batch row and head, with q_t, k_t (of head h // (H / Hk)) and
v_t of d channels, a log decay g_t <= 0 and a writing strength beta_t:

  delta_forward    S'_t = exp(g_t) S_{t-1},  w_t = beta_t (v_t - S'_t^T k_t),
                   S_t = S'_t + k_t w_t^T,   o_t = scale * S_t^T q_t
  delta_backward   the gradients of q, k, v, g, beta and the initial state
  delta_step       the same recurrence for one token, the state updated in place
  linear_act       out = act(x w^T + bias) + residual, and x w^T + bias if kept
  linear_act_backward
                   with dz = dout * act'(pre): dz w, dz^T x and the sum of dz
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the causal language-model shape of the benchmark, trained or prefilled from an empty state
        dict(name="delta_lm_4096", op="delta_forward", B=4, N=4096, H=12, Hk=12, d=64, dtype="bf16", state=False),
        # the 65536-token grid of the benchmark read as one sequence: few (batch, head) pairs, a long axis
        dict(name="delta_long_65536", op="delta_forward", B=4, N=65536, H=6, Hk=6, d=64, dtype="bf16", state=False),
        # a ragged float32 continuation of a prompt from a kept state, shared keys, head size off the tile sizes
        dict(name="delta_ragged_f32_d48", op="delta_forward", B=2, N=1021, H=6, Hk=3, d=48, dtype="f32", state=True),
        # training at the language-model shape
        dict(name="delta_backward_lm_4096", op="delta_backward", B=4, N=4096, H=12, Hk=12, d=64, dtype="bf16",
             state=False),
        # truncated back-propagation through a carried state, float32, the widest head, shared keys, odd length
        dict(name="delta_backward_f32_d128", op="delta_backward", B=1, N=777, H=4, Hk=2, d=128, dtype="f32",
             state=True),
        # serving: one token for each of 64 sequences
        dict(name="delta_step_64", op="delta_step", B=64, N=1, H=12, Hk=12, d=64, dtype="bf16", state=True),
        # serving one sequence, two value heads a key head: latency alone
        dict(name="delta_step_1", op="delta_step", B=1, N=1, H=12, Hk=6, d=64, dtype="bf16", state=True),
        # the language-model shape's projection of q, k and v, activated, the values under the activation kept
        dict(name="linear_qkv_16384", op="linear_act", rows=16384, k=768, n=2304, dtype="bf16", act="silu",
             bias=True, residual=False, keep=True),
        # the 65536-token grid's projection out of the heads, added to the residual stream
        dict(name="linear_out_262144", op="linear_act", rows=262144, k=384, n=384, dtype="bf16", act="none",
             bias=True, residual=True, keep=False),
        # serving one token: the widening projection of a feed-forward layer
        dict(name="linear_step_1", op="linear_act", rows=1, k=768, n=2304, dtype="bf16", act="gelu_tanh",
             bias=True, residual=False, keep=False),
        # training of the language-model shape's projection
        dict(name="linear_backward_16384", op="linear_act_backward", rows=16384, k=768, n=2304, dtype="bf16",
             act="silu", bias=True),
        # float32, nothing a multiple of a tile
        dict(name="linear_backward_f32", op="linear_act_backward", rows=1021, k=333, n=201, dtype="f32", act="gelu",
             bias=True),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, uniform in its logarithm, odd as often as even."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["delta_forward", "delta_backward", "delta_step", "linear_act", "linear_act_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("delta"):
        Hk = rng.randint(1, 8)
        H = Hk * rng.choice([1, 1, 2, 3])
        d = rng.choice([32, 40, 64, 64, 80, 96, 128])
        if op == "delta_step":
            return dict(op=op, B=_spread(rng, 1, 256), N=1, H=H, Hk=Hk, d=d, dtype=dtype, state=True)
        N = _spread(rng, 1, 32768)
        B = max(1, min(rng.randint(1, 8), (1 << 18) // (N * H)))
        return dict(op=op, B=B, N=N, H=H, Hk=Hk, d=d, dtype=dtype, state=rng.random() < 0.5)
    # half of the widths are those of models, multiples of 64, the others any
    width = lambda: 64 * _spread(rng, 1, 32) if rng.random() < 0.5 else _spread(rng, 8, 2048)
    k, n = width(), width()
    rows = _spread(rng, 1, max(1, min(65536, (1 << (34 if dtype == "bf16" else 32)) // (k * n))))
    case = dict(op=op, rows=rows, k=k, n=n, dtype=dtype, act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                bias=rng.random() < 0.7)
    if op == "linear_act":
        case.update(residual=rng.random() < 0.5, keep=rng.random() < 0.3)
    return case


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("linear"):
        rows, k, n = case["rows"], case["k"], case["n"]
        bias = n if case["bias"] else 0
        if case["op"] == "linear_act":
            outs = rows * n * (1 + case["residual"] + case["keep"])
            return {"bytes": (rows * k + n * k + bias + outs) * e, "flops": 2 * rows * k * n}
        kept = 0 if case["act"] == "none" else rows * n
        return {"bytes": (2 * rows * k + 2 * n * k + bias + rows * n + kept) * e, "flops": 4 * rows * k * n}
    B, N, H, Hk, d = case["B"], case["N"], case["H"], case["Hk"], case["d"]
    tokens, keys, states = B * N * H, B * N * Hk, 4 * B * H * d * d
    if case["op"] == "delta_forward":   # q, k, v, g, beta in, o out, the state in (if kept) and out
        return {"bytes": (2 * keys * d + tokens * (2 * d + 2)) * e + states * (2 if case["state"] else 1),
                "flops": 6 * tokens * d * d}
    if case["op"] == "delta_backward":  # q, k, v, g, beta, do in and their gradients out; the state, its gradients
        return {"bytes": (4 * keys * d + tokens * (3 * d + 4)) * e + states * (3 if case["state"] else 0),
                "flops": 16 * tokens * d * d}
    return {"bytes": (2 * keys * d + tokens * (2 * d + 2)) * e + 2 * states, "flops": 6 * tokens * d * d}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)
    s = {"case": dict(case)}
    if case["op"].startswith("linear"):
        rows, k, n = case["rows"], case["k"], case["n"]
        s["x"], s["w"] = normal(rows, k).to(dt), (normal(n, k) / math.sqrt(k)).to(dt)
        s["bias"] = (0.1 * normal(n)).to(dt) if case["bias"] else None
        if case["op"] == "linear_act":
            s["residual"] = normal(rows, n).to(dt) if case["residual"] else None
            return s
        s["dout"], s["pre"] = normal(rows, n).to(dt), None
        if case["act"] != "none":   # as the forward pass left it
            pre = s["x"].float() @ s["w"].float().t()
            s["pre"] = (pre + s["bias"].float() if case["bias"] else pre).to(dt)
        return s
    B, N, H, Hk, d = case["B"], case["N"], case["H"], case["Hk"], case["d"]
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()
    # heads remember between a few and a few hundred tokens
    bias = torch.linspace(1.0, 6.0, H, device=dev)
    s.update(scale=d ** -0.5, q=unit(normal(B, N, Hk, d)).mul_(d ** 0.5).to(dt), k=unit(normal(B, N, Hk, d)).to(dt),
             v=normal(B, N, H, d).to(dt), g=torch.nn.functional.logsigmoid(normal(B, N, H) + bias).to(dt),
             beta=normal(B, N, H).sigmoid().to(dt))
    s["state"] = normal(B, H, d, d) if case["state"] else None
    if case["op"] == "delta_backward":
        s["dout"] = normal(B, N, H, d).to(dt)
        s["dstate_out"] = normal(B, H, d, d) if case["state"] else None
    return s


# ------------------------------------------------------------------ plain forms


def _turn(x):
    return x.transpose(-1, -2)


def _inverse(L):
    """(1 + L)^-1 of strictly lower triangular [..., CHUNK, CHUNK]: the diagonal blocks' inverses, doubled in size."""
    T = torch.eye(CHUNK, device=L.device).expand(L.shape).contiguous()
    size = 1
    while size < CHUNK:
        n = CHUNK // (2 * size)
        cells = lambda x: x.view(*x.shape[:-2], n, 2 * size, n, 2 * size).diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        t, l = cells(T), cells(L)
        t[..., size:, :size] = -(t[..., size:, size:] @ l[..., size:, :size] @ t[..., :size, :size])
        size *= 2
    return T


def _scan(A, X, first):
    """States Y_0 = first, Y_{i+1} = A_i Y_i + X_i of [..., n, d, d], by doubling the span that A and X cover."""
    n = A.shape[-3]
    A, X = A.clone(), X.clone()
    X[..., 0, :, :] += A[..., 0, :, :] @ first
    step = 1
    while step < n:
        more = A[..., step:, :, :]
        X = torch.cat((X[..., :step, :, :], X[..., step:, :, :] + more @ X[..., :-step, :, :]), -3)
        A = torch.cat((A[..., :step, :, :], more @ A[..., :-step, :, :]), -3)
        step *= 2
    return torch.cat((first[..., None, :, :], X), -3)


def _chunks(s):
    """Inputs by chunks of CHUNK tokens, [B, H, n, CHUNK, ...] in 32 bits, and what a chunk does to the state."""
    N, H, Hk = s["case"]["N"], s["case"]["H"], s["case"]["Hk"]
    n = -(-N // CHUNK)

    def cut(x):
        x = torch.cat((x, x.new_zeros(x.shape[0], n * CHUNK - N, *x.shape[2:])), 1)
        x = x.view(x.shape[0], n, CHUNK, *x.shape[2:]).movedim(3, 1)
        return x.repeat_interleave(H // x.shape[1], 1)

    c = {name: cut(s[name]).float() for name in ("q", "k", "v", "beta")}
    c["cut"] = cut
    b = cut(s["g"]).double().cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=b.device).tril()
    gap = torch.where(lower, b[..., :, None] - b[..., None, :], -math.inf).exp().float()
    c["gap"] = gap
    c["inside"] = b.exp().float()[..., None]                       # decay from the chunk's start to t
    c["after"] = (b[..., -1:] - b).exp().float()[..., None]        # from t to the chunk's end
    c["all"] = b[..., -1].exp().float()[..., None, None]
    k, beta = c["k"], c["beta"][..., None]
    c["keys"] = (k @ _turn(k) * gap).tril(-1)
    c["scores"] = s["scale"] * (c["q"] @ _turn(k) * gap)
    c["T"] = _inverse(beta * c["keys"])
    c["U"] = c["T"] @ (beta * c["v"])
    c["K"] = c["T"] @ (beta * c["inside"] * k)
    d = k.shape[-1]
    c["A"] = c["all"] * torch.eye(d, device=k.device) - _turn(c["after"] * k) @ c["K"]
    first = s["state"] if s["state"] is not None else k.new_zeros(*k.shape[:2], d, d)
    c["S"] = _scan(c["A"], _turn(c["after"] * k) @ c["U"], first)
    c["W"] = c["U"] - c["K"] @ c["S"][:, :, :-1]
    return c


def _join(x, N):
    """[B, H, n, CHUNK, ...] back to [B, N, H, ...]."""
    x = x.movedim(1, 3)
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :N]


def _plain_delta_forward(s):
    c = _chunks(s)
    o = s["scale"] * c["inside"] * (c["q"] @ c["S"][:, :, :-1]) + c["scores"] @ c["W"]
    return {"out": _join(o, s["case"]["N"]).to(s["v"].dtype), "state": c["S"][:, :, -1]}


def _plain_delta_backward(s):
    c, scale = _chunks(s), s["scale"]
    N, H, Hk = s["case"]["N"], s["case"]["H"], s["case"]["Hk"]
    q, k, v, beta, S0, W = c["q"], c["k"], c["v"], c["beta"][..., None], c["S"][:, :, :-1], c["W"]
    do = c["cut"](s["dout"]).float()
    # the gradient of the state, from the last chunk to the first
    through = _turn(c["scores"]) @ do
    X = scale * _turn(c["inside"] * q) @ do - _turn(c["K"]) @ through
    last = s["dstate_out"] if s["dstate_out"] is not None else torch.zeros_like(c["S"][:, :, 0])
    G = _scan(_turn(c["A"]).flip(2), X.flip(2), last).flip(2)
    dS = G[:, :, 1:]
    dW = through + c["after"] * (k @ dS)
    dR = _turn(c["T"]) @ dW
    dscores, dkeys = scale * (do @ _turn(W)) * c["gap"], -beta * (dR @ _turn(W)) * c["gap"].tril(-1)
    carry, back = c["inside"] * (do @ _turn(S0)), dR @ _turn(S0)
    dq = scale * carry + dscores @ k
    left = W @ _turn(dS) * c["after"]
    dk = _turn(dscores) @ q + dkeys @ k + _turn(dkeys) @ k - beta * c["inside"] * back + left
    dbeta = (dR * (v - c["inside"] * (k @ S0))).sum(-1) - ((dR @ _turn(W)) * c["keys"]).sum(-1)
    # a gate decays what passes it: pairs of a later and an earlier token, and the state that enters or leaves
    pairs = dscores * (q @ _turn(k)) + dkeys * (k @ _turn(k))
    pairs = pairs.tril(-1).double()
    over = pairs.flip(-2).cumsum(-2).flip(-2)                      # over[j, s] = sum of pairs[t, s] for t >= j
    crossing = over.tril(-1).sum(-1)
    enters = ((scale * carry * q).sum(-1) - (beta * c["inside"] * back * k).sum(-1)).double()
    leaves = (left * k).sum(-1).double()
    dg = crossing + enters.flip(-1).cumsum(-1).flip(-1) + (leaves.cumsum(-1) - leaves)
    dg = dg + (c["all"] * S0 * dS).double().sum((-1, -2))[..., None]
    dt = s["v"].dtype
    shared = lambda x: _join(x, N).view(x.shape[0], N, Hk, H // Hk, -1).sum(3).to(dt)
    out = {"dq": shared(dq), "dk": shared(dk), "dv": _join(beta * dR, N).to(dt), "dg": _join(dg, N).to(dt),
           "dbeta": _join(dbeta, N).to(dt)}
    if s["state"] is not None:
        out["dstate"] = G[:, :, 0]
    return out


def _plain_delta_step(s):
    times = s["case"]["H"] // s["case"]["Hk"]
    q, k = (s[n].float()[:, 0].repeat_interleave(times, 1) for n in "qk")
    v, g, beta = (s[n].float()[:, 0] for n in ("v", "g", "beta"))
    S = g.exp()[..., None, None] * s["state"]
    w = beta[..., None] * (v - (k[..., :, None] * S).sum(-2))
    S = S + k[..., :, None] * w[..., None, :]
    s["state"].copy_(S)
    o = s["scale"] * (q[..., :, None] * S).sum(-2)
    return {"out": o[:, None].to(s["v"].dtype), "state": s["state"]}


def _plain_linear_act(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    act = s["case"]["act"]
    y = z
    if act == "relu":
        y = z.clamp(min=0)
    elif act == "gelu":
        y = 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    elif act == "gelu_tanh":
        y = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    elif act == "silu":
        y = z * torch.sigmoid(z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"out": y.to(s["x"].dtype)}
    if s["case"]["keep"]:
        out["pre"] = z.to(s["x"].dtype)
    return out


def _plain_linear_act_backward(s):
    dz, act = s["dout"].float(), s["case"]["act"]
    if act != "none":
        z = s["pre"].float()
        if act == "relu":
            slope = (z > 0).float()
        elif act == "gelu":
            slope = 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        elif act == "gelu_tanh":
            a = math.sqrt(2 / math.pi)
            t = torch.tanh(a * (z + 0.044715 * z * z * z))
            slope = 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
        else:
            p = torch.sigmoid(z)
            slope = p * (1 + z * (1 - p))
        dz = dz * slope
    dt = s["x"].dtype
    out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt)}
    if s["bias"] is not None:
        out["dbias"] = dz.sum(0, dtype=torch.float64).to(dt)
    return out


# ------------------------------------------------------------------ the framework's calls


def _own(s):
    import token_level_head_block_gb300 as mhla

    case = s["case"]
    op = case["op"]
    if op == "linear_act":
        pre = torch.empty(case["rows"], case["n"], dtype=s["x"].dtype, device=s["x"].device) if case["keep"] else None
        out = mhla.linear_act(s["x"], s["w"], s["bias"], activation=case["act"], residual=s["residual"], pre=pre)
        return {"out": out, "pre": pre} if case["keep"] else {"out": out}
    if op == "linear_act_backward":
        dx, dw, dbias = mhla.linear_act_backward(s["x"], s["w"], s["dout"], activation=case["act"], pre=s["pre"],
                                                 bias=case["bias"])
        return {"dx": dx, "dw": dw, "dbias": dbias} if case["bias"] else {"dx": dx, "dw": dw}
    args = tuple(s[n] for n in ("q", "k", "v", "g", "beta"))
    if op == "delta_forward":
        out, state = mhla.delta_forward(*args, scale=s["scale"], state=s["state"])
        return {"out": out, "state": state}
    if op == "delta_step":
        out = mhla.delta_step(*args, s["state"], scale=s["scale"])
        return {"out": out, "state": s["state"]}
    dq, dk, dv, dg, dbeta, dstate = mhla.delta_backward(*args, s["dout"], scale=s["scale"], state=s["state"],
                                                        dstate_out=s["dstate_out"])
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}
    if s["state"] is not None:
        out["dstate"] = dstate
    return out


def run(state):
    if own:
        return _own(state)
    return {"delta_forward": _plain_delta_forward, "delta_backward": _plain_delta_backward,
            "delta_step": _plain_delta_step, "linear_act": _plain_linear_act,
            "linear_act_backward": _plain_linear_act_backward}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact values


def _exact_delta(s):
    """The recurrence token by token in 64 bits, and its adjoint."""
    case = s["case"]
    times = case["H"] // case["Hk"]
    along = lambda name: s[name].double().transpose(0, 1)          # [N, B, heads, ...]
    q, k = (along(n).repeat_interleave(times, 2) for n in "qk")
    v, a, beta = along("v"), along("g").exp()[..., None, None], along("beta")[..., None]
    N, B, H, d = v.shape
    start = s["state"].double() if s["state"] is not None else torch.zeros(B, H, d, d, dtype=v.dtype, device=v.device)

    def token(S, t):
        M = a[t] * S
        miss = v[t] - torch.matmul(k[t, ..., None, :], M)[..., 0, :]
        w = beta[t] * miss
        return M, miss, w, torch.addcmul(M, k[t, ..., :, None], w[..., None, :])

    if "dout" not in s:
        S, out = start, torch.empty_like(v)
        for t in range(N):
            S = token(S, t)[3]
            torch.matmul(q[t, ..., None, :], S, out=out[t, ..., None, :])
        return {"out": (s["scale"] * out).transpose(0, 1), "state": S}
    if N * B * H * d * d * 8 > 40e9:    # every state is kept
        return None
    do = s["scale"] * along("dout")
    S = torch.empty(N + 1, B, H, d, d, dtype=v.dtype, device=v.device)
    S[0] = start
    for t in range(N):
        S[t + 1] = token(S[t], t)[3]
    dq = (S[1:] @ do[..., None])[..., 0]
    dk, dv, dg, dbeta = (torch.empty_like(x) for x in (v, v, beta[..., 0], beta[..., 0]))
    dS = s["dstate_out"].double() if s["dstate_out"] is not None else torch.zeros_like(start)
    for t in range(N - 1, -1, -1):
        M, miss, w, _ = token(S[t], t)
        dS = torch.addcmul(dS, q[t, ..., :, None], do[t, ..., None, :])
        dw = torch.matmul(k[t, ..., None, :], dS)[..., 0, :]
        dmiss = beta[t] * dw
        dv[t] = dmiss
        dbeta[t] = (dw * miss).sum(-1)
        dk[t] = (torch.matmul(dS, w[..., None]) - torch.matmul(M, dmiss[..., None]))[..., 0]
        dM = dS - k[t, ..., :, None] * dmiss[..., None, :]
        dg[t] = (dM * M).sum((-2, -1))
        dS = a[t] * dM
    shared = lambda x: x.view(N, B, case["Hk"], times, d).sum(3).transpose(0, 1)
    out = {"dq": shared(dq), "dk": shared(dk), "dv": dv.transpose(0, 1), "dg": dg.transpose(0, 1),
           "dbeta": dbeta.transpose(0, 1)}
    if s["state"] is not None:
        out["dstate"] = dS
    return out


def _exact_linear(s):
    """Products in 64 bits; the activations by their integrals' and quotients' formulas, their slopes by autograd."""
    case = s["case"]
    half = lambda z: torch.special.erfc(-z / math.sqrt(2)) / 2
    act = {"none": lambda z: 1 * z, "relu": lambda z: torch.where(z > 0, z, 0 * z), "gelu": lambda z: z * half(z),
           "gelu_tanh": lambda z: z / (1 + torch.exp(-math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))),
           "silu": lambda z: z / (1 + torch.exp(-z))}[case["act"]]
    x, w = s["x"].double(), s["w"].double()
    if case["op"] == "linear_act":
        z = torch.nn.functional.linear(x, w, s["bias"].double() if case["bias"] else None)
        out = {"out": act(z) + (s["residual"].double() if case["residual"] else 0)}
        if case["keep"]:
            out["pre"] = z
        return out
    dz = s["dout"].double()
    if s["pre"] is not None:
        z = s["pre"].double().requires_grad_()
        dz, = torch.autograd.grad(act(z), z, dz)
    out = {"dx": dz @ w, "dw": dz.t() @ x}
    if case["bias"]:
        out["dbias"] = dz.sum(0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linear(s) if case["op"].startswith("linear") else _exact_delta(s)
