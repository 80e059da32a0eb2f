"""The delta rule's digits: results against bounds made of the very terms that are summed for them (delta_bounds.py), so that a token, a
state or a head is held to its own size and not to the largest of the call."""

import numpy as np
import pytest
import torch

import oracle
import token_level_head_block_gb300 as mhla

from . import delta_bounds as db

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INPUTS = ("q", "k", "v", "g", "beta")
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dstate")


def draw(seed, B, N, Hk, times, d, dtype, state=True, remember=3.0):
    r = np.random.default_rng(seed)
    H = Hk * times
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))
    x = {"q": f(B, N, Hk, d), "k": f(B, N, Hk, d), "v": f(B, N, H, d), "dout": f(B, N, H, d)}
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


def doubles(x):
    return {n: f64(t) for n, t in x.items()}


def forward(x, scale):
    out, last = mhla.delta_forward(*(gpu(x[n]) for n in INPUTS), scale=scale, state=gpu(x["state"]))
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    return out, last


def steps(x, scale):
    """The same tokens one call each, from the same state."""
    B, N, H, d = x["v"].shape
    args = [gpu(x[n]) for n in INPUTS]
    state = torch.zeros(B, H, d, d, device=DEV) if x["state"] is None else gpu(x["state"])
    rows = [mhla.delta_step(*(t[:, i:i + 1] for t in args), state, scale=scale) for i in range(N)]
    torch.cuda.synchronize()
    return torch.cat(rows, 1), state


def check_forward(x, dtype, scale, out, last):
    want, end = db.chunk_form(doubles(x), dtype, scale)
    off, bound = db.over_axes(f64(out) - want.x, -1), db.out_bound(want, dtype)
    assert (off <= bound).all(), f"out: {(off / bound).max():.2f} of what is allowed"
    off, bound = db.over_axes(f64(last) - end.x, (-2, -1)), db.state_bound(end)
    assert (off <= bound).all(), f"state: {(off / bound).max():.2f} of what is allowed"
    return want, end


def check_backward(x, dtype, scale, got):
    for name, y, a in zip(GRADS, db.chunk_form(doubles(x), dtype, scale, back=True), got):
        bound, axes = db.grad_bound(name, y, dtype)
        off = db.over_axes(f64(a) - y.x, axes)
        assert np.isfinite(off).all() and (off <= bound).all(), f"{name}: {(off / bound).max():.2f} of what is allowed"


def backward(x, scale):
    got = mhla.delta_backward(*(gpu(x[n]) for n in INPUTS), gpu(x["dout"]), scale=scale, state=gpu(x["state"]),
                              dstate_out=gpu(x["dstate_out"]))
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    return got


# around the chunks of 32 and 64 tokens, several of them, head sizes on and off the tiles, shared keys, two tiles a CTA (24 heads
# and more of 64 channels)
SHAPES = [(1, 1, 1, 1, 64), (2, 64, 1, 2, 64), (1, 65, 1, 1, 128), (2, 129, 1, 3, 64), (1, 200, 2, 1, 48), (1, 130, 2, 1, 7),
          (2, 300, 1, 2, 100), (1, 700, 2, 1, 64), (1, 33, 1, 2, 32), (1, 260, 1, 2, 128), (3, 150, 7, 2, 64), (2, 70, 20, 1, 48)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("state", [True, False], ids=["state", "empty"])
def test_forward(shape, state, dtype):
    x = draw(sum(shape), *shape, dtype, state)
    check_forward(x, dtype, shape[4] ** -0.5, *forward(x, shape[4] ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("state", [True, False], ids=["state", "empty"])
def test_backward(shape, state, dtype):
    x = draw(sum(shape) + 1, *shape, dtype, state)
    check_backward(x, dtype, shape[4] ** -0.5, backward(x, shape[4] ** -0.5))


def fading(tokens, last, g, beta, dtype, d=64, state=False):
    """A chunk's tokens of full strength, then `last` ones that fade and write little."""
    x = draw(tokens + last, 1, tokens, 2, 1, d, dtype, state)
    x["g"][:, -last:] = g
    x["beta"][:, -last:] = beta
    return x


# a whole chunk of either type and a ragged one behind another; powers of two, so that a type's rounding does not matter
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [32, 64, 90])
@pytest.mark.parametrize("last,g,beta", [(8, -0.5, 0.0), (8, -1.0, 0.0), (12, -1.0, 0.0), (12, -1.0, 2.0 ** -13), (16, -1.0, 0.0),
                                         (16, -1.0, 2.0 ** -13), (16, -2.0, 0.0)])
def test_state_of_a_chunk_that_fades(last, g, beta, tokens, dtype):
    """What is left of a chunk's writes at its end is right for its own size, and the states that the gradients are formed
    with are those of the forward."""
    x = fading(tokens, last, g, beta, dtype)
    out, end = forward(x, 0.125)
    want, ref = check_forward(x, dtype, 0.125, out, end)
    assert (db.state_bound(ref) <= 1e-5 * db.over_axes(ref.x, (-2, -1))).all()
    _, one = steps(x, 0.125)
    assert (db.over_axes(f64(one) - f64(end), (-2, -1)) <= 2 * db.state_bound(ref)).all()
    check_backward(x, dtype, 0.125, backward(x, 0.125))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_behind_a_fading_chunk_read_what_is_left(dtype):
    """Chunks that end in fading, each read by tokens whose queries lift what is left to ordinary size."""
    x = draw(3, 1, 200, 2, 1, 64, dtype, False)
    for t in range(0, 200, 64):
        x["g"][:, t + 48:t + 64] = -1.0
        x["beta"][:, t + 48:t + 64] = 0.0
    check_forward(x, dtype, 0.125, *forward(x, 0.125))
    check_backward(x, dtype, 0.125, backward(x, 0.125))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [("v",), ("q", "v", "dout")], ids=["values", "all"])
def test_values_over_six_decades(what, dtype):
    """From token to token: each token's output is right for what that token and those before it put into it."""
    x = draw(5, 1, 200, 2, 1, 64, dtype, False)
    r = np.random.default_rng(6)
    for name in what:
        x[name] = (x[name].double() * torch.from_numpy(10.0 ** (-6 * r.random((1, 200, 2, 1))))).to(DT[dtype])
    check_forward(x, dtype, 0.125, *forward(x, 0.125))
    check_backward(x, dtype, 0.125, backward(x, 0.125))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_small_token_in_front_of_a_large_one(dtype):
    """The first token of a sequence, its value 1e-6 of the next one's: its output is w_0 (q . k) scale of its own value alone."""
    x = draw(7, 1, 16, 1, 1, 64, dtype, False)
    x["v"][:, 0] = (x["v"][:, 0].float() * 1e-6).to(DT[dtype])
    x["beta"][:, 0] = 1.0
    out, _ = forward(x, 0.125)
    y = doubles(x)
    score = 0.125 * (y["q"][0, 0, 0] @ y["k"][0, 0, 0])
    want = score * y["v"][0, 0, 0]
    # bf16: its score and its w as one fp16 each, the result's rounding; float32: three factors of 2^-22.  A channel of 16 tokens' w has one
    # scale: fp16's last bit, 2^-24 where the largest is at least 2^14, rounds by half of it, so 2^-39 of that largest
    share = 2 * 2.0 ** -11 + 2.0 ** -8 if dtype == "bf16" else 2.0 ** -17
    w = oracle.delta(*(y[n] for n in INPUTS), 0.125, steps=True)[3][0, :, 0]
    allowed = share * np.abs(want) + abs(score) * 2.0 ** -39 * np.abs(w).max(0)
    assert (np.abs(f64(out)[0, 0, 0] - want) <= allowed).all()
    assert np.linalg.norm(allowed) <= 0.01 * np.linalg.norm(want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-12, 1e-6, 1e6])
def test_gradients_of_every_size(size, dtype):
    """Gradients are linear in what comes back: dout and dstate_out a power of two times others give that times the bits, as long as
    no result leaves the type's normal range."""
    x = draw(9, 1, 150, 2, 2, 64, dtype)
    by = 2.0 ** round(np.log2(size))
    one = backward(x, 0.125)
    many = backward({**x, "dout": x["dout"] * by, "dstate_out": x["dstate_out"] * by}, 0.125)
    assert all(torch.equal(a.double() * by, b.double()) for a, b in zip(one, many))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_lies_around_the_results_stays(dtype):
    """Odd sizes and rows of their own length: nothing is written in front of, between or behind the results."""
    for B, N, Hk, times, d in [(2, 67, 1, 2, 33), (1, 1, 1, 1, 1), (1, 64, 2, 1, 7), (2, 130, 1, 3, 100)]:
        H = Hk * times
        x = draw(d, B, N, Hk, times, d, dtype)
        rooms = []

        def room(heads, width=None):
            """[B, N, heads(, width)] inside a larger array of sevens, and what is not of it."""
            shape = (B + 2, N + 2, heads + 1) + ((width + 3,) if width else ())
            whole = torch.full(shape, 7.0, dtype=DT[dtype], device=DEV)
            part = whole[1:B + 1, 1:N + 1, :heads, 1:width + 1] if width else whole[1:B + 1, 1:N + 1, :heads]
            mask = torch.ones(shape, dtype=torch.bool, device=DEV)
            (mask[1:B + 1, 1:N + 1, :heads, 1:width + 1] if width else mask[1:B + 1, 1:N + 1, :heads]).fill_(False)
            rooms.append((whole, mask))
            return part

        def square():
            whole = torch.full((B * H * d * d + 200,), 7.0, device=DEV)
            mask = torch.ones_like(whole, dtype=torch.bool)
            mask[100:-100] = False
            rooms.append((whole, mask))
            return whole[100:-100].view(B, H, d, d)

        args = [gpu(x[n]) for n in INPUTS]
        got = mhla.delta_forward(*args, scale=0.2, state=gpu(x["state"]), out=room(H, d), state_out=square())
        grads = mhla.delta_backward(*args, gpu(x["dout"]), scale=0.2, state=gpu(x["state"]), dstate_out=gpu(x["dstate_out"]),
                                    dq=room(Hk, d), dk=room(Hk, d), dv=room(H, d), dg=room(H), dbeta=room(H), dstate=square())
        state = square()
        state.copy_(gpu(x["state"]))
        one = mhla.delta_step(*(t[:, :1] for t in args), state, scale=0.2, out=room(H, d)[:, :1])
        torch.cuda.synchronize()
        assert all((whole[mask] == 7).all() for whole, mask in rooms)
        check_forward(x, dtype, 0.2, *got)
        check_backward(x, dtype, 0.2, grads)
        first, after = oracle.delta(*(f64(x[n][:, :1]) for n in INPUTS), 0.2, f64(x["state"]))
        assert np.abs(f64(one) - first).max() <= 2 * db.HALF[dtype] * np.abs(first).max() + 1e-5
        assert np.abs(f64(state) - after).max() <= 1e-5 * np.abs(after).max()


# two tiles of 16 columns a CTA, the widest heads, the narrowest, shared keys
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hk,times,d", [(3, 7, 2, 64), (4, 13, 1, 48), (1, 1, 2, 128), (1, 2, 1, 32), (2, 1, 3, 7)])
def test_fading_in_every_form_of_the_scan(B, Hk, times, d, dtype):
    x = draw(d, B, 100, Hk, times, d, dtype, False)
    for t in (20, 52, 88):                             # inside chunks of both types, the last one at the end
        x["g"][:, t:t + 12] = -1.0
        x["beta"][:, t:t + 12] = 0.0
    check_forward(x, dtype, d ** -0.5, *forward(x, d ** -0.5))
    check_backward(x, dtype, d ** -0.5, backward(x, d ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("beta", [1.0, 2.0])
def test_strengths_at_their_end(beta, dtype):
    """Unit keys written at full strength, and reflected (2): the state stays bounded, the triangular solve does not decay."""
    x = draw(31, 1, 150, 2, 1, 64, dtype)
    x["beta"][:] = beta
    check_forward(x, dtype, 0.125, *forward(x, 0.125))
    check_backward(x, dtype, 0.125, backward(x, 0.125))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what,value", [(w, float(x)) for w in ("k", "g", "beta", "v", "q") for x in ("nan", "inf")] + [("q", 1e30)])
def test_tokens_in_front_of_one_that_is_not_finite(what, value, dtype):
    """They keep their own digits, whatever stands behind them in their block of 16 or their chunk; so do other heads."""
    x = draw(33, 1, 70, 2, 1, 48, dtype)
    at, head = 21, 1
    want, _ = db.chunk_form(doubles(x), dtype, 0.2)
    if what in ("g", "beta"):
        x[what][0, at, head] = value
    else:
        x[what][0, at, head, 5] = value
    out, _ = forward(x, 0.2)
    off, bound = db.over_axes(f64(out) - want.x, -1), db.out_bound(want, dtype)
    assert (off <= bound)[:, :at].all() and (off <= bound)[:, :, 0].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["k", "beta"])
def test_keys_and_strengths_over_six_decades(what, dtype):
    """Tokens that write a millionth of what others do, and read as little of the state for it."""
    x = draw(41, 1, 200, 2, 1, 64, dtype)
    r = np.random.default_rng(42)
    by = torch.from_numpy(10.0 ** (-6 * r.random((1, 200, 2))))
    x[what] = (x[what].double() * (by[..., None] if what == "k" else by)).to(DT[dtype])
    check_forward(x, dtype, 0.125, *forward(x, 0.125))
    check_backward(x, dtype, 0.125, backward(x, 0.125))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_of_ordinary_size(dtype):
    """Rows padded in front and behind by tokens that are there but write nothing (beta = 0, g = 0), with any k of the others' size: out and
    state as without them; and the gradients of the tokens between."""
    N, front, behind, d = 90, 37, 21, 64
    x = draw(43, 1, front + N + behind, 2, 1, d, dtype)
    for cut in (slice(0, front), slice(front + N, None)):
        x["beta"][:, cut] = 0
        x["g"][:, cut] = 0
        x["dout"][:, cut] = 0
    mid = slice(front, front + N)
    short = {n: (t[:, mid].contiguous() if n in INPUTS + ("dout",) else t) for n, t in x.items()}
    out, last = forward(x, 0.125)
    check_forward(short, dtype, 0.125, out[:, mid], last)
    dq, dk, dv, dg, dbeta, dstate = backward(x, 0.125)
    check_backward(short, dtype, 0.125, (dq[:, mid], dk[:, mid], dv[:, mid], dg[:, mid], dbeta[:, mid], dstate))
    for cut in (slice(0, front), slice(front + N, None)):
        assert (dv[:, cut] == 0).all() and (dq[:, cut] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [(), ("v",), ("q", "v", "dout"), ("dout",), ("k",), ("beta",)], ids=lambda w: "_".join(w) or "alike")
@pytest.mark.parametrize("shape", [(1, 200, 2, 1, 64), (1, 150, 1, 2, 100)], ids=str)
def test_gradients_token_by_token(shape, what, dtype):
    """Inputs alike or over six decades: every token's own gradients are right for their own size (shared heads: dq and dk in sum)."""
    x = draw(51, *shape, dtype)
    r = np.random.default_rng(52)
    for name in what:
        by = torch.from_numpy(10.0 ** (-6 * r.random(x[name].shape[:3])))
        x[name] = (x[name].double() * (by if name == "beta" else by[..., None])).to(DT[dtype])
    got = backward(x, 0.125)
    for name, y, a in zip(GRADS[:5], db.chunk_form(doubles(x), dtype, 0.125, back=True), got):
        bound, size = db.token_bound(y, dtype)
        off = size(f64(a) - y.x)
        assert (off <= bound).all(), f"{name}: {(off / bound).max():.2f} of what is allowed"
        assert np.median(bound / size(y.x)) <= 0.05, name
