"""Linear layers with activation and residual, norm and the delta rule together, as a layer of a model runs them.

One layer: qkv = silu(x W_qkv^T + b), q and k normed in place in qkv's rows (k to unit length), decays and write strengths from
a second projection, the delta rule over views of those rows, x + o W_out^T, then y + gelu(y W_up^T + b) W_down^T.  The stages
pass their type on; the reference takes each stage in float64 on what that stage was given, so each answers for itself and the
whole for the handing over.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HK, H, D = 2, 4, 32
C = 96
UP = 200
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().cpu().double().numpy()


class Layer:
    def __init__(self, seed, dtype):
        r = np.random.default_rng(seed)
        new = lambda *s, by=1.0: torch.from_numpy((by * r.standard_normal(s)).astype(np.float32)).to(dtype).to(DEV)
        self.p = {"qkv": new((2 * HK + H) * D, C, by=C ** -0.5), "qkv_bias": new((2 * HK + H) * D, by=0.1),
                  "gates": new(2 * H, C, by=C ** -0.5), "gates_bias": new(2 * H, by=0.1),
                  "out": new(C, H * D, by=(H * D) ** -0.5), "up": new(UP, C, by=C ** -0.5), "up_bias": new(UP, by=0.1),
                  "down": new(C, UP, by=UP ** -0.5)}
        self.unit = torch.full((D,), D ** -0.5, device=DEV)

    def sequence(self, x):
        """q, k (normed), v as views of the projection's rows, decays, strengths; and what the backward pass needs."""
        p, (B, N) = self.p, x.shape[:2]
        pre = torch.empty(B, N, (2 * HK + H) * D, dtype=x.dtype, device=DEV)
        rows = mhla.linear_act(x, p["qkv"], p["qkv_bias"], "silu", pre=pre)
        raw = rows.clone()
        heads = rows.view(B, N, 2 * HK + H, D)
        q, k, v = heads[:, :, :HK], heads[:, :, HK:2 * HK], heads[:, :, 2 * HK:]
        mhla.qk_norm(q, k, self.unit, self.unit, q_out=q, k_out=k)
        z = mhla.linear_act(x, p["gates"], p["gates_bias"])
        g, beta = torch.nn.functional.logsigmoid(z[..., :H] + 2), z[..., H:].sigmoid()
        return (q, k, v, g, beta), {"pre": pre, "raw": raw, "z": z}

    def after(self, x, o):
        p = self.p
        y = mhla.linear_act(o.flatten(2), p["out"], residual=x)
        pre = torch.empty(*x.shape[:-1], UP, dtype=x.dtype, device=DEV)
        hidden = mhla.linear_act(y, p["up"], p["up_bias"], "gelu", pre=pre)
        return mhla.linear_act(hidden, p["down"], residual=y), {"y": y, "hidden": hidden, "up": pre}

    def forward(self, x, state=None):
        args, _ = self.sequence(x)
        o, last = mhla.delta_forward(*args, state=state)
        return self.after(x, o)[0], last

    def step(self, x, state):
        args, _ = self.sequence(x)
        return self.after(x, mhla.delta_step(*args, state))[0]

    def backward(self, x, dout):
        """(dx, {name: gradient}) of sum(dout * forward(x)[0])."""
        p, (B, N) = self.p, x.shape[:2]
        args, kept = self.sequence(x)
        o, _ = mhla.delta_forward(*args)
        _, more = self.after(x, o)
        grads = {}
        dhidden, grads["down"], _ = mhla.linear_act_backward(more["hidden"], p["down"], dout, bias=False)
        dy, grads["up"], grads["up_bias"] = mhla.linear_act_backward(more["y"], p["up"], dhidden, "gelu", more["up"])
        dy += dout
        do, grads["out"], _ = mhla.linear_act_backward(o.flatten(2), p["out"], dy, bias=False)
        drows = torch.empty_like(kept["raw"])
        heads = drows.view(B, N, 2 * HK + H, D)
        dq, dk, dv = heads[:, :, :HK], heads[:, :, HK:2 * HK], heads[:, :, 2 * HK:]
        _, _, _, dg, dbeta, _ = mhla.delta_backward(*args, do.view(B, N, H, D), dq=dq, dk=dk, dv=dv)
        raw = kept["raw"].view(B, N, 2 * HK + H, D)
        mhla.qk_norm_backward(raw[:, :, :HK], raw[:, :, HK:2 * HK], dq, dk, self.unit, self.unit, dq=dq, dk=dk)
        dx, grads["qkv"], grads["qkv_bias"] = mhla.linear_act_backward(x, p["qkv"], drows, "silu", kept["pre"])
        z = kept["z"]
        dz = torch.cat((dg * (-(z[..., :H] + 2)).sigmoid(), dbeta * args[4] * (1 - args[4])), -1)
        dx_gates, grads["gates"], grads["gates_bias"] = mhla.linear_act_backward(x, p["gates"], dz)
        return dx + dx_gates + dy, grads


def tokens(seed, B, N, dtype):
    return torch.randn(B, N, C, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def check_linear(got, x, w, bias, kind, residual, dtype):
    """k products in float32 (each of a sum of at most 2 k steps), what bf16 keeps of the sum, and the activation's slope, at
    most 1.2: float32 itself works it out to 2^-20 of its size."""
    x, w, res = f64(x), f64(w), 0.0 if residual is None else f64(residual)
    ref, z = oracle.linear_act(x, w, None if bias is None else f64(bias), kind, None if residual is None else res)
    size = np.abs(x) @ np.abs(w).T + (0.0 if bias is None else np.abs(f64(bias)))
    bound = HALF[dtype] * np.abs(ref) + 1.2 * (2 * x.shape[-1] + 8) * 2.0 ** -24 * size + 2.0 ** -20 * (np.abs(z) + np.abs(ref) + np.abs(res))
    assert (np.abs(f64(got) - ref) <= bound).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,N", [(1, 1), (2, 50), (3, 333)])
def test_each_stage_of_a_layer(B, N, dtype):
    layer, x = Layer(1, dtype), tokens(2, B, N, dtype)
    p = layer.p
    args, kept = layer.sequence(x)
    o, state = mhla.delta_forward(*args)
    out, more = layer.after(x, o)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    check_linear(kept["raw"], x, p["qkv"], p["qkv_bias"], "silu", None, dtype)
    raw = kept["raw"].view(B, N, 2 * HK + H, D)
    q, k, v, g, beta = args
    for got, t in ((q, raw[:, :, :HK]), (k, raw[:, :, HK:2 * HK])):
        ref = oracle.qk_norm(f64(t), f64(layer.unit), 1e-6)
        assert (np.abs(f64(got) - ref) <= HALF[dtype] * np.abs(ref) + (D + 16) * 2.0 ** -24 * np.abs(ref)).all()
    assert torch.equal(v, raw[:, :, 2 * HK:])                            # the values' rows are as they were
    ref, end, all_S, w = oracle.delta(*(f64(t) for t in args), steps=True)
    # as tests of the rule alone have it: 16 u of the largest state and a chunk's w a chunk, T of norm 2 at most; unit q and k
    u, chunk = (2.0 ** -16, 64) if dtype == torch.bfloat16 else (2.0 ** -23, 32)
    X = float(np.linalg.norm(all_S, axis=(-2, -1)).max()) + float(np.linalg.norm(w, axis=-1).max()) * min(N, chunk) ** 0.5
    E = 16 * u * (N // chunk + 1) * X
    scores = 2.0 ** -8 * np.abs(w).sum(1, keepdims=True) if dtype == torch.bfloat16 else 0.0
    assert (np.abs(f64(o) - ref) <= HALF[dtype] * np.abs(ref) + 1.01 * (E + scores)).all()
    assert (np.abs(f64(state) - end) <= E).all()
    check_linear(more["y"], o.flatten(2), p["out"], None, "none", x, dtype)
    check_linear(more["hidden"], more["y"], p["up"], p["up_bias"], "gelu", None, dtype)
    check_linear(out, more["hidden"], p["down"], None, "none", more["y"], dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_steps_and_parts_continue_a_sequence(dtype):
    """A prompt in two parts and then token by token against the whole at once.  The stages round their float32 results to the
    type; where those differ in their last bits a rounding may fall the other way, a step of the type, 2 half ones, and a stage's
    own results are then of inputs a step off: six stages, at most 6 steps in all of rows of one size (a residual stream that
    every stage's result is added to)."""
    B, N, first, cut = 3, 150, 70, 131
    layer, x = Layer(3, dtype), tokens(4, B, N, dtype)
    whole, end = layer.forward(x)
    a, state = layer.forward(x[:, :first].contiguous())
    b, state = layer.forward(x[:, first:cut].contiguous(), state)
    got = [a, b] + [layer.step(x[:, t:t + 1].contiguous(), state) for t in range(cut, N)]
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    half = max(HALF[dtype], 2.0 ** -20)                                  # float32: sums of 200 terms of random sign
    assert (torch.cat(got, 1).double() - whole.double()).norm() <= 12 * half * whole.double().norm()
    assert (state - end).norm() <= 12 * half * end.norm()


def reference(layer, x):
    """The layer in float64 with automatic differentiation: (out, leaves)."""
    leaf = lambda t: t.detach().cpu().double().requires_grad_()
    p, x = {n: leaf(t) for n, t in layer.p.items()}, leaf(x)
    B, N = x.shape[:2]
    F = torch.nn.functional
    rows = F.silu(x @ p["qkv"].T + p["qkv_bias"]).view(B, N, 2 * HK + H, D)
    norm = lambda t: t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * D ** -0.5
    q, k = (norm(t).repeat_interleave(H // HK, 2) for t in (rows[:, :, :HK], rows[:, :, HK:2 * HK]))
    v, z = rows[:, :, 2 * HK:], x @ p["gates"].T + p["gates_bias"]
    g, beta = F.logsigmoid(z[..., :H] + 2), z[..., H:].sigmoid()
    S, o = torch.zeros(B, H, D, D, dtype=torch.float64), []
    for t in range(N):
        S = g[:, t].exp()[..., None, None] * S
        w = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(-2))
        S = S + k[:, t, :, :, None] * w[:, :, None, :]
        o.append((S * q[:, t, :, :, None]).sum(-2))
    y = x + torch.stack(o, 1).flatten(2) @ p["out"].T
    return y + F.gelu(y @ p["up"].T + p["up_bias"]) @ p["down"].T, x, p


def test_gradients_of_a_layer():
    """Every gradient of the float32 layer against automatic differentiation in float64.  Each of the twelve stages (six of each
    direction) is good to 2^-16 of its result's norm: float32 sums of at most 200 terms, three bf16 terms or two of fp16 a
    factor.  The maps in between have random weights of norm below 2, so what a stage leaves grows by less than 4 on its way."""
    B, N = 2, 70
    layer, x = Layer(5, torch.float32), tokens(6, B, N, torch.float32)
    dout = tokens(7, B, N, torch.float32)
    dx, grads = layer.backward(x, dout)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    out, x64, p = reference(layer, x)
    out.backward(dout.cpu().double())
    for name, got, ref in [("x", dx, x64.grad)] + [(n, grads[n], p[n].grad) for n in p]:
        assert float((got.cpu().double() - ref).norm()) <= 12 * 4 * 2.0 ** -16 * float(ref.norm()), name


def test_a_layer_captured_with_its_gradients():
    """Both directions in one graph, replayed on new tokens beside eager calls of the same layer: the same bits."""
    B, N = 2, 130
    layer = Layer(8, torch.bfloat16)
    x, dout = tokens(9, B, N, torch.bfloat16), tokens(10, B, N, torch.bfloat16)
    run = lambda: (layer.forward(x), layer.backward(x, dout))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (out, last), (dx, grads) = run()
    for seed in (11, 12):
        x.copy_(tokens(seed, B, N, torch.bfloat16))
        graph.replay()
        (out2, last2), (dx2, grads2) = run()
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(last, last2) and torch.equal(dx, dx2)
        assert all(torch.equal(grads[n], grads2[n]) for n in grads)
    assert mhla.device_status() == 0


def test_two_layers_at_once():
    """Two streams at once, each with what its calls allocate: the same bits as one after the other."""
    B, N = 4, 700
    layers = [Layer(s, torch.bfloat16) for s in (13, 14)]
    xs, douts = ([tokens(s, B, N, torch.bfloat16) for s in pair] for pair in ((15, 16), (17, 18)))
    want = [(l.forward(x), l.backward(x, d)) for l, x, d in zip(layers, xs, douts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, l, x, d in zip(streams, layers, xs, douts):
            with torch.cuda.stream(s):
                got.append((l.forward(x), l.backward(x, d)))
        torch.cuda.synchronize()
        for ((out, last), (dx, grads)), ((o2, l2), (dx2, g2)) in zip(want, got):
            assert torch.equal(out, o2) and torch.equal(last, l2) and torch.equal(dx, dx2)
            assert all(torch.equal(grads[n], g2[n]) for n in grads)


# ------------------------------------------------------------------ streams

def stream_calls():
    gen = torch.Generator(device=DEV).manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    B, N, d = 2, 3001, 64
    q, k, v, dout = (normal(B, N, 12, d).bfloat16() for _ in range(4))
    k = k / d ** 0.5
    g, beta = torch.nn.functional.logsigmoid(normal(B, N, 12) + 3).bfloat16(), normal(B, N, 12).sigmoid().bfloat16()
    state, x, w, dz = normal(B, 12, d, d), normal(6002, 768).bfloat16(), normal(768, 768).bfloat16() / 28, normal(6002, 768).bfloat16()
    one = [t[:, :1] for t in (q, k, v, g, beta)]
    return {"delta_forward": lambda **kw: mhla.delta_forward(q, k, v, g, beta, state=state, **kw),
            "delta_backward": lambda **kw: mhla.delta_backward(q, k, v, g, beta, dout, state=state, **kw),
            "delta_step": lambda **kw: (mhla.delta_step(*one, state.clone(), **kw),),
            "linear_act": lambda **kw: (mhla.linear_act(x, w, activation="gelu", **kw),),
            "linear_act_backward": lambda **kw: mhla.linear_act_backward(x, w, dz, "gelu", dz, **kw)}


NAMES = ["delta_forward", "delta_backward", "delta_step", "linear_act", "linear_act_backward"]


@pytest.mark.parametrize("name", [n for n in NAMES if n != "delta_step"])
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_memory_is_not_handed_to_another_stream(name, handle):
    """An output dropped while its stream may still write it: the current stream gets other memory."""
    run = stream_calls()[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = run(stream=s.cuda_stream if handle else s)
    places = [(t.data_ptr(), t.numel() * t.element_size(), t.shape, t.dtype) for t in got if t is not None]
    del got
    for at, size, shape, dtype in places:
        if size < 1 << 20:      # small blocks come from shared segments: their addresses say nothing
            continue
        other = [torch.empty(shape, dtype=dtype, device=DEV) for _ in range(3)]
        assert all(t.data_ptr() != at for t in other)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_the_same_bits_as_on_the_current_stream(name):
    run = stream_calls()[name]
    want = run()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0, torch.cuda.default_stream()):
        torch.cuda.synchronize()
        got = run(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got) if a is not None)


# ------------------------------------------------------------------ waits that give up

def raw_status():
    """(status, flags) of mhla_device_status without raising."""
    flags = ctypes.c_uint32(0)
    st = mhla.lib().mhla_device_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream) or None, ctypes.byref(flags))
    return int(st), int(flags.value)


# a warp that fetches for the scan or for the gradients' chain; the one that issues the linear layer's products, whose waits
# outlast a first look (there the hook acts on those alone)
@pytest.mark.parametrize("name,warp", [("delta_forward", 4), ("delta_forward", 7), ("delta_backward", 5), ("linear_act", 1)])
def test_a_wait_that_gives_up_is_reported_and_the_context_recovers(name, warp):
    run = stream_calls()[name]
    want = run()
    torch.cuda.synchronize()
    assert raw_status() == (0, 0)
    mhla.debug_stall_waits(warp, 1_000_000)
    try:
        run()
        torch.cuda.synchronize()
        status, flags = raw_status()
    finally:
        mhla.debug_stall_waits(-1)
    assert status == 5 and flags & 1, (status, flags)
    assert raw_status() == (0, 0)
    got = run()
    torch.cuda.synchronize()
    assert raw_status() == (0, 0)
    assert all(torch.equal(a, b) for a, b in zip(want, got) if a is not None)
