"""The gated delta rule, its gradients and its single-token form against the float64 oracle.

Tolerances.  A chunk is a triangular solve and four products whose factors enter the tensor cores as sums of
bf16 terms, which keep each factor to u = 2^-16 (bf16 calls, two terms of half a step 2^-8 each) or 2^-23 (float32
calls, where the float32 sums round as much).  Eight such roundings (state, K^, T twice, U, W, the chunk's sum, the decay) meet in
what a chunk adds to the state, each a share u of something no larger than X = max |S_t| + |w of a chunk| (norms, from
the oracle) times the norm of T, at most 2 here; and as |1 - beta k k^T| <= 1 for unit keys a later chunk does not enlarge
what it is handed.  So after n chunks
  |dS| <= 16 u n X =: E.
A result is within half a step of its type, 2^-8 |ref| for bf16, plus what its formula makes of E:
  out      scale |q_t| E, and for bf16 calls the scores' one rounding, 2^-8 scale |q_t| sum over the chunk |w_s,c|
           (|k_s| <= 1, decay <= 1)
  gradients  products of two quantities known to a share 16 u n of their norms: S or w (X) with dout or dS (Y)
"""

import numpy as np
import pytest
import torch

import oracle
import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -16, "f32": 2.0 ** -23}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
CHUNK = {"bf16": 64, "f32": 32}
INPUTS = ("q", "k", "v", "g", "beta")


def draw(seed, B, N, Hk, times, d, dtype, state=True, remember=3.0):
    r = np.random.default_rng(seed)
    H = Hk * times
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))
    x = {"q": f(B, N, Hk, d), "k": f(B, N, Hk, d), "v": f(B, N, H, d), "dout": f(B, N, H, d)}
    # the longest key stays below 1 after its rounding
    x["k"] = x["k"] / x["k"].norm(dim=-1, keepdim=True) * 0.99
    x["g"] = torch.nn.functional.logsigmoid(f(B, N, H) + remember)
    x["beta"] = f(B, N, H).sigmoid()
    x = {n: t.to(DT[dtype]) for n, t in x.items()}
    x["state"] = f(B, H, d, d) if state else None
    x["dstate_out"] = f(B, H, d, d) if state else None
    return x


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def gpu(t):
    return None if t is None else t.to(DEV)


def norm(x):
    return float(np.linalg.norm(x))


def heads(x, H):
    return np.repeat(x, H // x.shape[2], axis=2)


def over_chunks(x, C):
    """[B, N, ...] summed over each chunk, at each of its tokens."""
    out = np.empty_like(x)
    for t in range(0, x.shape[1], C):
        out[:, t:t + C] = x[:, t:t + C].sum(1, keepdims=True)
    return out


def reference(x, dtype, scale):
    """Oracle's forward with E and the bound of every output."""
    q, k, v, g, beta, S = (f64(x[n]) for n in INPUTS + ("state",))
    o, last, all_S, w = oracle.delta(q, k, v, g, beta, scale, S, steps=True)
    C, B, N, H = CHUNK[dtype], v.shape[0], v.shape[1], v.shape[2]
    n = -(-N // C)
    # norms of each (b, h): of the largest state and of the w of a chunk
    states = np.sqrt((all_S ** 2).sum((-1, -2))).max(0)
    if S is not None:
        states = np.maximum(states, np.sqrt((S ** 2).sum((-1, -2))))
    X = states + np.sqrt(over_chunks((w ** 2).sum(-1), C)).max(1)          # [B, H]
    E = 16 * U[dtype] * n * X
    size_q = abs(scale) * np.sqrt((heads(q, H) ** 2).sum(-1))               # [B, N, H]
    bound = HALF[dtype] * np.abs(o) + (size_q * E[:, None])[..., None]
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * size_q[..., None] * over_chunks(np.abs(w), C)
    return o, last, bound, E, X


def check_forward(x, dtype, scale, out, last):
    o, end, bound, E, _ = reference(x, dtype, scale)
    got = f64(out)
    assert got.shape == o.shape and np.isfinite(got).all()
    assert (np.abs(got - o) <= bound + 1e-30).all(), f"out: {np.abs(got - o).max():.3e} off"
    off = np.sqrt(((f64(last) - end) ** 2).sum((-1, -2)))
    assert (off <= E + 1e-30).all(), f"state: {off.max():.3e} off, bound {E.min():.3e}"


def run_forward(x, scale, **kw):
    out, last = mhla.delta_forward(*(gpu(x[n]) for n in INPUTS), scale=scale, state=gpu(x["state"]), **kw)
    torch.cuda.synchronize()
    return out, last


def run_backward(x, scale, **kw):
    got = mhla.delta_backward(*(gpu(x[n]) for n in INPUTS), gpu(x["dout"]), scale=scale, state=gpu(x["state"]),
                              dstate_out=gpu(x["dstate_out"]), **kw)
    torch.cuda.synchronize()
    return got


def check_backward(x, dtype, scale, got):
    q, k, v, g, beta, do, S, dS = (f64(x[n]) for n in INPUTS + ("dout", "state", "dstate_out"))
    *ref, Y = oracle.delta_backward(q, k, v, g, beta, do, scale, S, dS, steps=True)
    _, _, _, _, X = reference(x, dtype, scale)
    X = norm(X)
    N = v.shape[1]
    n, root = -(-N // CHUNK[dtype]), N ** 0.5
    share = 16 * U[dtype] * n
    do_n, q_n, w_n = norm(do), norm(q), X * n
    # norms of the products that each gradient sums; bf16 calls round the scores' part of dS and dq once more (2^-8 of
    # what a chunk adds)
    Y = Y + abs(scale) * q_n * do_n / max(1, n) ** 0.5
    terms = {"dq": abs(scale) * X * do_n, "dk": Y * w_n + X * Y * root, "dv": Y * root, "dg": X * Y * root,
             "dbeta": Y * root * (norm(v) / root + X), "dstate": Y}
    for (name, size), a, r in zip(terms.items(), got, ref):
        a = f64(a)
        assert a.shape == r.shape and np.isfinite(a).all(), name
        own = 2.0 ** -24 if name == "dstate" else HALF[dtype]
        # one rounding of the result, one of shared heads' or scores' parts
        allowed = 3 * own * norm(r) + share * size
        assert norm(a - r) <= allowed, f"{name}: {norm(a - r):.3e} off, {allowed:.3e} allowed, of {norm(r):.3e}"


# batch, tokens, key heads, value heads a key head, channels: one token, around the chunks of 32 and 64, several of them;
# head sizes on and off the tile sizes
SHAPES = [(1, 1, 1, 1, 64), (2, 2, 3, 1, 64), (1, 31, 1, 2, 32), (1, 32, 2, 1, 64), (1, 33, 1, 1, 128), (1, 63, 2, 1, 32),
          (2, 64, 1, 2, 64), (1, 65, 1, 1, 128), (2, 129, 1, 3, 64), (1, 200, 2, 1, 48), (1, 130, 2, 1, 7), (1, 97, 1, 1, 1),
          (2, 300, 1, 2, 100), (1, 700, 2, 1, 64), (1, 400, 1, 1, 33), (1, 260, 1, 2, 80)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,Hk,times,d", SHAPES)
@pytest.mark.parametrize("state", [True, False], ids=["state", "empty"])
def test_forward(B, N, Hk, times, d, dtype, state):
    x = draw(N + d, B, N, Hk, times, d, dtype, state)
    check_forward(x, dtype, d ** -0.5, *run_forward(x, d ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,Hk,times,d", SHAPES)
@pytest.mark.parametrize("state", [True, False], ids=["state", "empty"])
def test_backward(B, N, Hk, times, d, dtype, state):
    x = draw(N + d + 1, B, N, Hk, times, d, dtype, state)
    check_backward(x, dtype, d ** -0.5, run_backward(x, d ** -0.5))


# more tiles of 16 columns than SMs (twice as many in the last): a CTA takes two tiles, the last one of 48 channels a half
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,Hk,times,d", [(3, 150, 7, 2, 64), (4, 70, 13, 1, 48), (5, 70, 4, 4, 60), (2, 90, 40, 1, 32)])
def test_many_heads(B, N, Hk, times, d, dtype):
    x = draw(N + d, B, N, Hk, times, d, dtype)
    check_forward(x, dtype, d ** -0.5, *run_forward(x, d ** -0.5))
    check_backward(x, dtype, d ** -0.5, run_backward(x, d ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hk,times,d", [(1, 1, 1, 64), (3, 2, 2, 64), (2, 3, 1, 48), (1, 2, 1, 7), (2, 1, 3, 128), (1, 1, 1, 1),
                                          (2, 2, 1, 30)])
def test_step(B, Hk, times, d, dtype):
    """float32 arithmetic: d products a sum, twice."""
    x = draw(d, B, 1, Hk, times, d, dtype)
    state = gpu(x["state"])
    out = mhla.delta_step(*(gpu(x[n]) for n in INPUTS), state, scale=0.3)
    torch.cuda.synchronize()
    q, k, v, g, beta, S = (f64(x[n]) for n in INPUTS + ("state",))
    o, end = oracle.delta(q, k, v, g, beta, 0.3, S)
    X = norm(S) + norm(v)
    assert norm(f64(state) - end) <= 4 * (d + 8) * 2.0 ** -24 * X
    assert (np.abs(f64(out) - o) <= HALF[dtype] * np.abs(o) + 4 * (d + 8) * 2.0 ** -24 * 0.3 * norm(q) * X).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_continue_the_forward(dtype):
    x = draw(9, 2, 80, 2, 2, 64, dtype)
    whole, end = run_forward(x, 0.125)
    cut = {n: (t[:, :70].contiguous() if n in INPUTS else t) for n, t in x.items()}
    _, state = run_forward(cut, 0.125)
    rows = [mhla.delta_step(*(gpu(x[n])[:, t:t + 1] for n in INPUTS), state, scale=0.125) for t in range(70, 80)]
    torch.cuda.synchronize()
    o, _, bound, E, _ = reference(x, dtype, 0.125)
    assert (np.abs(f64(torch.cat(rows, 1)) - o[:, 70:]) <= 2 * bound[:, 70:]).all()
    assert (np.sqrt((f64(state - end) ** 2).sum((-1, -2))) <= 2 * E).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_of_one_row(dtype):
    """q, k, v side by side in a projection's rows, gates and strengths side by side in another's, out and gradients too;
    what lies between and behind stays as it was."""
    B, N, H, d = 2, 150, 3, 40
    x = draw(11, B, N, H, 1, d, dtype)
    rows = torch.full((B, N + 2, 4, H, d), 7.0, dtype=DT[dtype], device=DEV)
    for i, n in enumerate(("q", "k", "v")):
        rows[:, :N, i] = x[n].to(DEV)
    gates = torch.stack((x["g"], x["beta"]), 2).to(DEV)
    args = [rows[:, :N, i] for i in range(3)] + [gates[:, :, 0], gates[:, :, 1]]
    out, last = mhla.delta_forward(*args, scale=0.2, state=gpu(x["state"]), out=rows[:, :N, 3])
    check_forward(x, dtype, 0.2, out, last)
    grads = torch.full((B, N, 3, H, d), 7.0, dtype=DT[dtype], device=DEV)
    dgates = torch.empty_like(gates)
    got = mhla.delta_backward(*args, gpu(x["dout"]), scale=0.2, state=gpu(x["state"]), dstate_out=gpu(x["dstate_out"]),
                              dq=grads[:, :, 0], dk=grads[:, :, 1], dv=grads[:, :, 2], dg=dgates[:, :, 0], dbeta=dgates[:, :, 1])
    torch.cuda.synchronize()
    check_backward(x, dtype, 0.2, got)
    assert (rows[:, N:] == 7).all()


def test_heads_in_front_and_odd_addresses():
    """[B, H, N, d] tensors seen as [B, N, H, d], and one that starts an element behind a 16-byte boundary."""
    x = draw(12, 2, 70, 2, 1, 64, "bf16")
    turned = {n: x[n].transpose(1, 2).contiguous().to(DEV).transpose(1, 2) for n in INPUTS}
    flat = torch.empty(x["k"].numel() + 1, dtype=torch.bfloat16, device=DEV)
    flat[1:] = x["k"].flatten().to(DEV)
    turned["k"] = flat[1:].view(x["k"].shape)
    out, last = mhla.delta_forward(*(turned[n] for n in INPUTS), scale=0.1, state=gpu(x["state"]))
    torch.cuda.synchronize()
    check_forward(x, "bf16", 0.1, out, last)


def test_broadcast_inputs():
    """One key row for every batch row and one strength for every token: strides of 0."""
    x = draw(13, 3, 90, 2, 1, 32, "f32")
    x["k"] = x["k"][:1].expand(3, -1, -1, -1)
    x["beta"] = x["beta"][:, :1].expand(-1, 90, -1)
    args = [gpu(x[n]) if n not in ("k", "beta") else None for n in INPUTS]
    args[1] = x["k"][:1].to(DEV).expand(3, -1, -1, -1)
    args[4] = x["beta"][:, :1].to(DEV).expand(-1, 90, -1)
    assert args[1].stride(0) == 0 and args[4].stride(1) == 0
    out, last = mhla.delta_forward(*args, scale=0.2, state=gpu(x["state"]))
    torch.cuda.synchronize()
    check_forward(x, "f32", 0.2, out, last)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_state_in_place_and_given_workspace(dtype):
    x = draw(14, 2, 100, 1, 2, 64, dtype)
    state = gpu(x["state"])
    ws = torch.empty(mhla.delta_workspace_size(gpu(x["q"]), gpu(x["v"])), dtype=torch.uint8, device=DEV)
    out, last = mhla.delta_forward(*(gpu(x[n]) for n in INPUTS), scale=0.1, state=state, state_out=state, workspace=ws)
    torch.cuda.synchronize()
    assert last is state
    check_forward(x, dtype, 0.1, out, state)
    ws = torch.full((mhla.delta_backward_workspace_size(gpu(x["q"]), gpu(x["v"])),), 255, dtype=torch.uint8, device=DEV)
    check_backward(x, dtype, 0.1, run_backward(x, 0.1, workspace=ws))   # what lay there before does not matter


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_closed_gates_pack_sequences(dtype):
    """A gate of -infinity starts afresh: two sequences in one row are the two by themselves."""
    x = draw(15, 1, 150, 2, 1, 64, dtype, state=False)
    x["g"][:, 77] = -torch.inf
    x["g"][:, 40] = -5000.0
    out, last = run_forward(x, 0.1)
    check_forward(x, dtype, 0.1, out, last)
    behind = {n: (t[:, 77:].contiguous() if t is not None else None) for n, t in x.items()}
    _, alone = run_forward(behind, 0.1)
    _, _, _, E, _ = reference(x, dtype, 0.1)
    assert (np.sqrt((f64(last - alone) ** 2).sum((-1, -2))) <= 2 * E).all()
    check_backward(x, dtype, 0.1, run_backward(x, 0.1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strong_decay(dtype):
    """Gates that sum far below what a product of decays from the chunk's start could hold."""
    x = draw(16, 1, 200, 2, 1, 64, dtype, remember=-30.0)
    check_forward(x, dtype, 0.1, *run_forward(x, 0.1))
    got = run_backward(x, 0.1)
    check_backward(x, dtype, 0.1, got)
    ref = oracle.delta_backward(*(f64(x[n]) for n in INPUTS + ("dout",)), 0.1, f64(x["state"]), f64(x["dstate_out"]))
    # each gate's gradient carries its own decay, about e^-30: no larger sum's rounding is left in it, but for the bf16
    # result's half step and as much again of the scores'
    assert np.abs(f64(got[3]) - ref[3]).max() <= 2.0 ** -6 * np.abs(ref[3]).max()


def test_padding_leaves_the_state():
    x = draw(17, 2, 130, 2, 1, 64, "f32")
    x["beta"][:, 100:] = 0
    x["g"][:, 100:] = 0
    _, last = run_forward(x, 0.1)
    cut = {n: (t[:, :100].contiguous() if n in INPUTS else t) for n, t in x.items()}
    _, short = run_forward(cut, 0.1)
    assert torch.equal(last, short) or (np.sqrt((f64(last - short) ** 2).sum((-1, -2))) <= 2 * reference(cut, "f32", 0.1)[3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_of_very_different_sizes(dtype):
    """Output gradients, queries and values over six decades from token to token: a token's dq is right for its own size.
    dq_t = scale S_t dout_t, so with dout_t exact and S_t known to a share r of X its error is below r scale X |dout_t|.  bf16
    calls: one rounding of the result, 2^-12 of the largest for each of a sum of d = 64 values of the state or of a chunk's w and k,
    of random sign: sqrt(64) 2^-12 = 2^-9 for either, r = 2^-8.  float32: E of the forward, with two fp16 (2^-22) a factor."""
    x = draw(51, 1, 200, 2, 1, 64, dtype)
    r = np.random.default_rng(52)
    for name in ("q", "v", "dout"):
        x[name] = (x[name].double() * torch.from_numpy(10.0 ** (-6 * r.random((1, 200, 2, 1))))).to(DT[dtype])
    out, last = run_forward(x, 0.125)
    check_forward(x, dtype, 0.125, out, last)
    got = run_backward(x, 0.125)
    check_backward(x, dtype, 0.125, got)
    q, k, v, g, beta, do, S, dS = (f64(x[n]) for n in INPUTS + ("dout", "state", "dstate_out"))
    ref = oracle.delta_backward(q, k, v, g, beta, do, 0.125, S, dS)[0]
    _, _, all_S, w = oracle.delta(q, k, v, g, beta, 0.125, S, steps=True)
    X = float(np.linalg.norm(all_S, axis=(-2, -1)).max()) + float(np.linalg.norm(w, axis=-1).max()) * CHUNK[dtype] ** 0.5
    share = 2.0 ** -8 if dtype == "bf16" else 16 * 2.0 ** -22 * 7
    each = np.linalg.norm(f64(got[0]) - ref, axis=-1)
    allowed = HALF[dtype] * np.linalg.norm(ref, axis=-1) + share * 0.125 * X * np.linalg.norm(do, axis=-1)
    assert (each <= allowed).all(), (each / allowed).max()


def test_offsets_beyond_32_bits():
    """Tokens 2^23 elements apart, the last ones behind 2^31: every tensor a view of rows of one array, the same bits as
    with its own."""
    B, N, H, d = 1, 300, 2, 64
    x = draw(41, B, N, H, 1, d, "bf16")
    want = run_forward(x, 0.125) + tuple(run_backward(x, 0.125))
    rows = torch.empty(N, 1 << 23, dtype=torch.bfloat16, device=DEV)
    assert (N - 1) * rows.stride(0) > 1 << 31
    views, at = {}, 0
    for name, width in [(n, H * d) for n in ("q", "k", "v", "dout", "out", "dq", "dk", "dv")] + [(n, H) for n in ("g", "beta", "dg", "dbeta")]:
        part = rows[:, at:at + width]
        views[name] = part.view(1, N, H, d) if width == H * d else part.view(1, N, H)
        at += width + 8
        if name in x:
            views[name].copy_(x[name])
    args = [views[n] for n in INPUTS]
    out, last = mhla.delta_forward(*args, scale=0.125, state=gpu(x["state"]), out=views["out"])
    grads = mhla.delta_backward(*args, views["dout"], scale=0.125, state=gpu(x["state"]), dstate_out=gpu(x["dstate_out"]),
                                **{n: views[n] for n in ("dq", "dk", "dv", "dg", "dbeta")})
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip((out, last) + tuple(grads), want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["k", "g", "beta", "v", "q"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite(what, value, dtype):
    """Earlier tokens and other heads are as they were; from the token on everything (v: its channel, q: its row) is NaN.
    A block of 16 rows or a chunk enters the tensor cores at the scale of its largest value, which a later token that no longer
    counts can change: an earlier token's result moves within its bound around the exact one, so by twice that at most."""
    x = draw(18, 2, 140, 2, 1, 48, dtype)
    clean, clean_last = run_forward(x, 0.1)
    _, _, bound, E, _ = reference(x, dtype, 0.1)
    at = 70
    if what in ("g", "beta"):
        x[what][1, at, 1] = value
    else:
        x[what][1, at, 1, 5] = value
    out, last = run_forward(x, 0.1)
    touched = torch.zeros_like(out, dtype=torch.bool)
    state = torch.zeros_like(last, dtype=torch.bool)
    if what == "q":
        touched[1, at, 1] = True
    elif what == "v":
        touched[1, at:, 1, 5] = True
        state[1, 1, :, 5] = True
    else:
        touched[1, at:, 1] = True
        state[1, 1] = True
    far = ~touched.clone()
    far[1, :, 1] = False
    assert torch.equal(out[far], clean[far]) and torch.equal(last[0], clean_last[0]) and torch.equal(last[1, 0], clean_last[1, 0])
    rest = (~touched).cpu().numpy()
    assert (np.abs(f64(out) - f64(clean)) <= 2 * bound)[rest].all()
    off = np.where(state.cpu().numpy(), 0, f64(last) - f64(clean_last))
    assert (np.sqrt((off ** 2).sum((-1, -2))) <= 2 * E).all()
    assert not out[touched].isfinite().any() and not last[state].isfinite().any()


def test_zero_length_work():
    z = lambda *s: torch.empty(*s, device=DEV)
    out, last = mhla.delta_forward(z(0, 5, 2, 32), z(0, 5, 2, 32), z(0, 5, 4, 32), z(0, 5, 4), z(0, 5, 4))
    assert out.shape == (0, 5, 4, 32) and last.shape == (0, 4, 32, 32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_every_time(dtype):
    x = draw(19, 2, 333, 2, 3, 64, dtype)
    a, b = run_backward(x, 0.1), run_backward(x, 0.1)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert all(torch.equal(s, t) for s, t in zip(run_forward(x, 0.1), run_forward(x, 0.1)))


def test_on_another_stream_and_captured():
    """Forward and gradients on a side stream, then captured and replayed on new values in the same tensors."""
    x = draw(20, 2, 150, 2, 2, 64, "bf16")
    args = [gpu(x[n]) for n in INPUTS]
    state, dout, dstate = gpu(x["state"]), gpu(x["dout"]), gpu(x["dstate_out"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, last = mhla.delta_forward(*args, scale=0.1, state=state, stream=side)
    got = mhla.delta_backward(*args, dout, scale=0.1, state=state, dstate_out=dstate, stream=side)
    side.synchronize()
    check_forward(x, "bf16", 0.1, out, last)
    check_backward(x, "bf16", 0.1, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, last = mhla.delta_forward(*args, scale=0.1, state=state)
        got = mhla.delta_backward(*args, dout, scale=0.1, state=state, dstate_out=dstate)
    y = draw(21, 2, 150, 2, 2, 64, "bf16")
    for t, n in zip(args, INPUTS):
        t.copy_(y[n])
    state.copy_(y["state"])
    dout.copy_(y["dout"])
    dstate.copy_(y["dstate_out"])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        check_forward(y, "bf16", 0.1, out, last)
        check_backward(y, "bf16", 0.1, got)


def test_gradients_by_differences():
    """Float32 gradients against central differences of the kernel's own forward, along random directions: both
    sides carry float32's rounding of the loss, about 2^-20 of it, over a step of 2^-5 each way."""
    x = draw(22, 1, 70, 1, 2, 32, "f32")
    got = dict(zip(INPUTS + ("state",), run_backward(x, 0.3)))
    r = np.random.default_rng(5)

    def loss(y):
        o, last = run_forward(y, 0.3)
        return (f64(o) * f64(y["dout"])).sum() + (f64(last) * f64(y["dstate_out"])).sum()

    size = abs(f64(x["dout"])).sum()
    for name, grad in got.items():
        way = torch.from_numpy(r.standard_normal(tuple(x[name].shape)).astype(np.float32))
        way = way / way.norm()
        h = 2.0 ** -5
        up, down = ({**x, name: x[name] + s * h * way} for s in (1, -1))
        want = (f64(grad) * f64(way)).sum()
        # the third derivative's part: h^2 of a loss that is smooth on the scale of 1
        assert abs((loss(up) - loss(down)) / (2 * h) - want) <= 2.0 ** -20 * size / h + h * h * max(abs(want), norm(f64(grad)))


def test_refusals():
    x = draw(23, 2, 20, 2, 2, 32, "bf16")
    args = [gpu(x[n]) for n in INPUTS]
    with pytest.raises(mhla.MhlaError):                          # 3 value heads on 2 key heads
        mhla.delta_forward(*args[:2], args[2][:, :, :3], args[3][:, :, :3], args[4][:, :, :3])
    with pytest.raises(mhla.MhlaError):
        mhla.delta_forward(*args[:4], args[4].float())
    with pytest.raises(ValueError):
        mhla.delta_forward(*args, state=torch.zeros(2, 4, 32, 31, device=DEV))
    with pytest.raises(ValueError):
        mhla.delta_forward(args[0].half(), *args[1:])
    with pytest.raises(ValueError):
        mhla.delta_forward(args[0].cpu(), *args[1:])
    with pytest.raises(mhla.MhlaError):
        mhla.delta_forward(*args, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(mhla.MhlaError):
        mhla.delta_step(*args, torch.zeros(2, 4, 32, 32, device=DEV))   # more than one token
    with pytest.raises(mhla.MhlaError):
        mhla.delta_forward(*args, out=args[2])
