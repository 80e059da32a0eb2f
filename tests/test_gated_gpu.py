"""The gated recurrence, its gradients and its single-token form against the float64 oracle.

Tolerances.  The kernels keep sums and states in float32 and give the tensor
cores every factor as a sum of bf16 terms: bf16 runs use two terms for the decayed
scores and for the state that a query reads (each rounding leaves at most
2^-8 of what it rounds, so two leave 2^-16), three where the result is float32
(2^-24).  With A the same sum over absolute values, a bf16 result is within
  2^-8 |ref|          its own rounding
  + 2^-15 A           scores and state, 2^-16 each
and a float32 result within n 2^-24 A, where n counts the float32 operations in
a row that a term of the sum can meet: d of its dot product, 64 of its chunk, one or two per
later chunk, and 64 for the decay (an exponent's rounding, exp, and the products of terms dropped).
dg is a sum over later tokens of q.dq - k.dk: the bounds of dq and dk add up.
"""

import numpy as np
import pytest
import torch

import oracle
import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def draw(seed, B, N, H, d, dtype, state=True, remember=3.0):
    r = np.random.default_rng(seed)
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(DT[dtype])
    x = {n: f(B, N, H, d) for n in ("q", "k", "v", "dout")}
    x["g"] = torch.nn.functional.logsigmoid(f(B, N, H).float() + remember).to(DT[dtype])
    x["state"] = torch.from_numpy(r.standard_normal((B, H, d, d)).astype(np.float32)) if state else None
    x["dstate_out"] = torch.from_numpy(r.standard_normal((B, H, d, d)).astype(np.float32)) if state else None
    return x


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def gpu(t):
    return None if t is None else t.to(DEV)


def magnitude(x):
    return None if x is None else np.abs(x)


def slack(dtype, N, d):
    return 2.0 ** -15 if dtype == "bf16" else (d + 128 + 2 * (N // 64 + 1)) * 2.0 ** -24


def f32_slack(N, d):
    return (d + 128 + 2 * (N // 64 + 1)) * 2.0 ** -24


def within(name, got, ref, own, bound):
    got = f64(got)
    assert got.shape == ref.shape
    assert np.isfinite(got).all(), name
    over = np.abs(got - ref) - (own * np.abs(ref) + bound + 1e-30)
    assert over.max() <= 0, f"{name}: {np.abs(got - ref).max():.3e} off, {over.max():.3e} over its bound"


def check_forward(x, dtype, scale, out, last):
    q, k, v, g, S = (f64(x[n]) for n in ("q", "k", "v", "g", "state"))
    N, d = q.shape[1], q.shape[3]
    ref, end = oracle.gated(q, k, v, g, scale, S)
    size, size_end = oracle.gated(*(np.abs(a) for a in (q, k, v)), g, abs(scale), magnitude(S))
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    within("out", out, ref, u, slack(dtype, N, d) * size)
    within("state", last, end, 2.0 ** -24, f32_slack(N, d) * size_end)


def run_forward(x, scale, **kw):
    out, last = mhla.gated_forward(*(gpu(x[n]) for n in ("q", "k", "v", "g")), scale=scale, state=gpu(x["state"]), **kw)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    return out, last


# lengths of one token, around a chunk of 64 and around spans of chunks; head sizes on and off the tile sizes
SHAPES = [(1, 1, 1, 64), (2, 2, 3, 64), (1, 63, 2, 32), (2, 64, 2, 64), (1, 65, 1, 128), (2, 129, 3, 64),
          (1, 200, 2, 48), (1, 130, 2, 7), (1, 97, 1, 1), (2, 300, 2, 100), (1, 1000, 2, 64), (1, 2500, 1, 32),
          (40, 70, 9, 32)]


# bf16 on the tcgen05 kernel: more chunks than its stages, a last chunk of one token, few spans (joined by
# the scan) and more of them (joined apart), several waves, 32 and 64 channels whole and in part
TC_SHAPES = [(2, 769, 11, 64), (4, 1000, 6, 64), (1, 2300, 12, 40), (1, 5000, 4, 64), (10, 520, 8, 32), (10, 641, 8, 24),
             (16, 300, 10, 64), (20, 1030, 8, 8)]


@pytest.mark.parametrize("B,N,H,d", TC_SHAPES)
@pytest.mark.parametrize("state", [True, False], ids=["state", "empty"])
def test_forward_of_many_tokens(B, N, H, d, state):
    x = draw(N + H, B, N, H, d, "bf16", state)
    check_forward(x, "bf16", d ** -0.5, *run_forward(x, d ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,d", SHAPES)
@pytest.mark.parametrize("state", [True, False], ids=["state", "empty"])
def test_forward(B, N, H, d, dtype, state):
    x = draw(N + d, B, N, H, d, dtype, state)
    check_forward(x, dtype, d ** -0.5, *run_forward(x, d ** -0.5))


def check_backward(x, dtype, scale, got):
    q, k, v, g, do, S, dS = (f64(x[n]) for n in ("q", "k", "v", "g", "dout", "state", "dstate_out"))
    N, d = q.shape[1], q.shape[3]
    ref = oracle.gated_backward(q, k, v, g, do, scale, S, dS)
    size = oracle.gated_backward(*(np.abs(a) for a in (q, k, v)), g, np.abs(do), abs(scale), magnitude(S), magnitude(dS))
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    c = slack(dtype, N, d)
    for name, a, r, z in zip(("dq", "dk", "dv"), got, ref, size):
        within(name, a, r, u, c * z)
    # every step of the running sum brings the errors of a dq and a dk; its own float32 additions stay below
    # 2^-24 of what it has summed, at most N of them
    steps = (np.abs(q) * size[0]).sum(-1) + (np.abs(k) * size[1]).sum(-1)
    later = np.cumsum(steps[:, ::-1], axis=1)[:, ::-1]
    end = oracle.gated(*(np.abs(a) for a in (q, k, v)), g, 1.0, magnitude(S))[1]
    if dS is not None:
        later = later + (end * np.abs(dS)).sum((-1, -2))[:, None]
    within("dg", got[3], ref[3], u, (c + (d + N) * 2.0 ** -24) * later)
    within("dstate", got[4], ref[4], 2.0 ** -24, f32_slack(N, d) * size[4])


def run_backward(x, scale, **kw):
    got = mhla.gated_backward(*(gpu(x[n]) for n in ("q", "k", "v", "g", "dout")), scale=scale, state=gpu(x["state"]),
                              dstate_out=gpu(x["dstate_out"]), **kw)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,d", SHAPES)
@pytest.mark.parametrize("state", [True, False], ids=["state", "empty"])
def test_backward(B, N, H, d, dtype, state):
    x = draw(3 * N + d, B, N, H, d, dtype, state)
    check_backward(x, dtype, d ** -0.5, run_backward(x, d ** -0.5))


@pytest.mark.parametrize("B,N,H,d", [(1, 769, 4, 64), (2, 520, 6, 40), (1, 1500, 5, 64), (20, 1030, 8, 8), (7, 300, 8, 64)])
@pytest.mark.parametrize("state", [True, False], ids=["state", "empty"])
def test_backward_of_many_tokens(B, N, H, d, state):
    x = draw(N + H, B, N, H, d, "bf16", state)
    check_backward(x, "bf16", d ** -0.5, run_backward(x, d ** -0.5))


# the warp-level kernel over several spans: two slices of columns, float32 rows that 16-byte loads take and do not
@pytest.mark.parametrize("B,N,H,d,dtype", [(1, 900, 2, 128, "bf16"), (2, 700, 3, 72, "bf16"), (1, 900, 2, 128, "f32"),
                                           (2, 700, 3, 70, "f32"), (1, 1300, 3, 64, "f32"), (3, 600, 2, 36, "f32"),
                                           (12, 200, 9, 128, "f32")])
def test_spans_of_wide_heads_and_of_float32(B, N, H, d, dtype):
    x = draw(N + d, B, N, H, d, dtype)
    check_forward(x, dtype, d ** -0.5, *run_forward(x, d ** -0.5))
    check_backward(x, dtype, d ** -0.5, run_backward(x, d ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,d", [(2, 777, 12, 40), (1, 333, 3, 24), (3, 150, 5, 100), (10, 200, 6, 8)])
def test_what_an_earlier_launch_left_on_the_chip(B, N, H, d, dtype):
    """A call whose every value is NaN, then one with rows, channels and tokens behind its ends."""
    nan = draw(60, 4, 2048, 12, 128 if d > 64 else 64, dtype)
    nan = {n: torch.full_like(t, float("nan")) for n, t in nan.items()}
    x = draw(61, B, N, H, d, dtype)
    for _ in range(2):
        run_forward(nan, 1.0), run_backward(nan, 1.0)
        check_forward(x, dtype, d ** -0.5, *run_forward(x, d ** -0.5))
        run_forward(nan, 1.0), run_backward(nan, 1.0)
        check_backward(x, dtype, d ** -0.5, run_backward(x, d ** -0.5))


def test_backward_against_differences_of_the_forward():
    """Central differences of the framework's own forward, float32, along a direction per input.

    With x +- h dx, h = 2^-6, the loss is linear in each of q, k, v and the state, so only
    the gates leave a term in h^2: loss''' h^2 / 6, under 1e-3 of the derivative's size for |dg| <= 1
    over 70 tokens; each loss is a sum of B N H d outputs good to 1e-5 of A."""
    x = draw(11, 1, 70, 2, 16, "f32")
    scale, h = 0.25, 2.0 ** -6
    grads = dict(zip(("q", "k", "v", "g", "state"), run_backward(x, scale)))
    loss = lambda y: sum(float((a.double().cpu() * b.double()).sum())
                         for a, b in zip(run_forward(y, scale), (x["dout"], x["dstate_out"])))
    r = np.random.default_rng(12)
    for name in ("q", "k", "v", "g", "state"):
        step = torch.from_numpy(r.standard_normal(tuple(x[name].shape)).astype(np.float32))
        if name == "g":
            step = step * 0.05
        up, down = dict(x), dict(x)
        up[name], down[name] = x[name] + h * step, x[name] - h * step
        got = float((grads[name].cpu().double() * step.double()).sum())
        want = (loss(up) - loss(down)) / (2 * h)
        size = float((grads[name].cpu().double().abs() * step.double().abs()).sum())
        assert abs(got - want) <= 2e-3 * size, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_closed_gates_start_afresh(dtype):
    """Gates of -inf, of the type's lowest value, and ones so low that exp is zero: packed sequences."""
    x = draw(21, 2, 210, 2, 64, dtype)
    x["g"][:, 0, 1] = float("-inf")
    x["g"][0, 64] = float("-inf")
    x["g"][0, 127] = torch.finfo(DT[dtype]).min
    x["g"][1, 100:103] = -200.0
    x["g"][1, 180] = float("-inf")
    check_forward(x, dtype, 0.125, *run_forward(x, 0.125))
    check_backward(x, dtype, 0.125, run_backward(x, 0.125))


@pytest.mark.parametrize("dtype,H,d", [("f32", 1, 32), ("bf16", 11, 64)], ids=["f32", "bf16"])
@pytest.mark.parametrize("value", [0.0, -0.7, -2.0, -30.0])
def test_constant_gates_over_a_long_sequence(value, dtype, H, d):
    """No forgetting at all, short memories whose far pairs vanish, and almost none."""
    x = draw(22, 1, 1500, H, d, dtype)
    x["g"][:] = value
    check_forward(x, dtype, 1.0, *run_forward(x, 1.0))
    check_backward(x, dtype, 1.0, run_backward(x, 1.0))


def test_padding_tokens_leave_the_state():
    x = draw(23, 2, 150, 2, 64, "bf16")
    for n in ("k", "g"):
        x[n][:, 90:] = 0
    short = {n: (v[:, :90] if n in ("q", "k", "v", "g", "dout") else v) for n, v in x.items()}
    out, last = run_forward(x, 0.125)
    a, b = run_forward(short, 0.125)
    # the same sums in another grouping: both within the bound of the same oracle value
    check_forward(short, "bf16", 0.125, out[:, :90], last)
    check_forward(short, "bf16", 0.125, a, b)


@pytest.mark.parametrize("N", [5, 200, 5000])
def test_pieces_join(N):
    """A sequence cut at any point and carried on through its state, the state updated in place."""
    x = draw(24, 2, N, 2, 64, "f32")
    state = x["state"].clone().to(DEV)
    outs = []
    for a, b in ((0, N // 3), (N // 3, N // 3 + 1), (N // 3 + 1, N)):
        if a == b:
            continue
        cut = [x[n][:, a:b].to(DEV) for n in ("q", "k", "v", "g")]
        out, back = mhla.gated_forward(*cut, scale=0.125, state=state, state_out=state)
        assert back.data_ptr() == state.data_ptr()
        outs.append(out)
    torch.cuda.synchronize()
    check_forward(x, "f32", 0.125, torch.cat(outs, 1), state)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,d", [(1, 1, 64), (3, 5, 64), (2, 3, 128), (70, 12, 32), (2, 2, 48), (1, 2, 7), (1, 1, 1),
                                   (2, 3, 100)])
def test_step(B, H, d, dtype):
    x = draw(B + d, B, 1, H, d, dtype)
    state = x["state"].clone().to(DEV)
    out = mhla.gated_step(*(gpu(x[n]) for n in ("q", "k", "v", "g")), state, scale=0.3)
    torch.cuda.synchronize()
    check_forward(x, dtype, 0.3, out, state)


def test_steps_are_the_forward():
    x = draw(25, 3, 80, 2, 64, "bf16")
    state = x["state"].clone().to(DEV)
    outs = [mhla.gated_step(*(x[n][:, t:t + 1].to(DEV) for n in ("q", "k", "v", "g")), state, scale=0.125)
            for t in range(80)]
    torch.cuda.synchronize()
    check_forward(x, "bf16", 0.125, torch.cat(outs, 1), state)


def test_step_with_a_closed_gate_and_strides():
    x = draw(26, 4, 1, 3, 64, "bf16")
    x["g"][1] = float("-inf")
    x["g"][2, 0, 1] = -5000.0
    rows = torch.stack([x[n] for n in ("q", "k", "v")], 2).to(DEV)       # [B, 1, 3, H, d]
    state = x["state"].clone().to(DEV)
    out = mhla.gated_step(rows[:, :, 0], rows[:, :, 1], rows[:, :, 2], x["g"].to(DEV), state, scale=0.125)
    torch.cuda.synchronize()
    check_forward(x, "bf16", 0.125, out, state)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 40])
def test_views_of_one_projection(dtype, d):
    """q, k, v, out and the gradients as interleaved views; an odd element offset breaks 16-byte loads."""
    B, N, H = 2, 150, 3
    x = draw(27, B, N, H, d, dtype)
    for extra in (0, 1):
        row = 4 * H * d + extra
        buf = torch.full((B, N, row), float("nan"), dtype=DT[dtype], device=DEV)
        grads = torch.full((B, N, row), float("nan"), dtype=DT[dtype], device=DEV)
        view = lambda b, i: b[:, :, extra + i * H * d: extra + (i + 1) * H * d].unflatten(2, (H, d))
        q, k, v, o = (view(buf, i) for i in range(4))
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            t.copy_(x[n])
        out, last = mhla.gated_forward(q, k, v, gpu(x["g"]), scale=0.2, state=gpu(x["state"]), out=o)
        got = mhla.gated_backward(q, k, v, gpu(x["g"]), gpu(x["dout"]), scale=0.2, state=gpu(x["state"]),
                                  dstate_out=gpu(x["dstate_out"]), dq=view(grads, 0), dk=view(grads, 1), dv=view(grads, 2))
        torch.cuda.synchronize()
        check_forward(x, dtype, 0.2, out, last)
        check_backward(x, dtype, 0.2, got)
        if extra:
            assert buf[:, :, 0].isnan().all()
        assert grads[:, :, extra + 3 * H * d:].isnan().all()              # nothing written beside the views


def test_heads_that_share_keys_and_values():
    """Strides of zero: one key and value head for all query heads."""
    x = draw(28, 2, 100, 4, 64, "bf16")
    k, v = x["k"][:, :, :1].to(DEV).expand(-1, -1, 4, -1), x["v"][:, :, :1].to(DEV).expand(-1, -1, 4, -1)
    x["k"], x["v"] = k.cpu().contiguous(), v.cpu().contiguous()
    out, last = mhla.gated_forward(gpu(x["q"]), k, v, gpu(x["g"]), scale=0.1, state=gpu(x["state"]))
    torch.cuda.synchronize()
    check_forward(x, "bf16", 0.1, out, last)


def test_another_order_of_axes():
    """[B, H, N, d] memory seen as [B, N, H, d], a gate tensor of other strides."""
    x = draw(29, 2, 140, 3, 64, "bf16")
    turn = lambda t: t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    out = torch.empty(2, 3, 140, 64, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    got, last = mhla.gated_forward(*(turn(x[n]) for n in ("q", "k", "v", "g")), scale=0.1, state=gpu(x["state"]), out=out)
    torch.cuda.synchronize()
    check_forward(x, "bf16", 0.1, got, last)
    check_backward(x, "bf16", 0.1, mhla.gated_backward(*(turn(x[n]) for n in ("q", "k", "v", "g", "dout")), scale=0.1,
                                                        state=gpu(x["state"]), dstate_out=gpu(x["dstate_out"])))


def test_the_same_bits_every_time_and_on_another_stream():
    x = draw(30, 2, 3000, 3, 64, "bf16")
    a, b = run_forward(x, 0.125), run_backward(x, 0.125)
    c, d = run_forward(x, 0.125), run_backward(x, 0.125)
    args = [gpu(x[n]) for n in ("q", "k", "v", "g")]
    state, dout, ds = gpu(x["state"]), gpu(x["dout"]), gpu(x["dstate_out"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    e = mhla.gated_forward(*args, scale=0.125, state=state, stream=s)
    f = mhla.gated_backward(*args, dout, scale=0.125, state=state, dstate_out=ds, stream=s)
    torch.cuda.synchronize()
    for first, second in ((a, c), (b, d), (a, e), (b, f)):
        assert all(torch.equal(p, q) for p, q in zip(first, second))


def test_caller_workspace_holds_exactly_what_is_asked():
    x = draw(31, 1, 4000, 2, 64, "bf16")
    q = gpu(x["q"])
    for size, run in ((mhla.gated_workspace_size(q), run_forward), (mhla.gated_backward_workspace_size(q), run_backward)):
        buf = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device=DEV)   # stale contents, guarded end
        got, plain = run(x, 0.125, workspace=buf[:size]), run(x, 0.125)
        assert (buf[size:] == 0x5A).all()
        assert all(torch.equal(a, b) for a, b in zip(got, plain))


def test_captured_and_replayed_with_new_values():
    x, y = draw(32, 1, 700, 2, 64, "bf16"), draw(33, 1, 700, 2, 64, "bf16")
    buf = {n: gpu(v).clone() for n, v in x.items()}
    fwd = lambda: mhla.gated_forward(buf["q"], buf["k"], buf["v"], buf["g"], scale=0.125, state=buf["state"])
    bwd = lambda: mhla.gated_backward(buf["q"], buf["k"], buf["v"], buf["g"], buf["dout"], scale=0.125,
                                      state=buf["state"], dstate_out=buf["dstate_out"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd(), bwd()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grads = fwd(), bwd()
    for n, v in y.items():
        buf[n].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    check_forward(y, "bf16", 0.125, *out)
    check_backward(y, "bf16", 0.125, grads)


@pytest.mark.parametrize("B,N,H,d", [(4, 1024, 12, 64), (1, 9000, 12, 64), (3, 900, 2, 128)])
def test_calls_behind_one_another_that_share_a_workspace(B, N, H, d):
    """Each reads what the one in front wrote (its v, its state), the scan's launch starting before its spans' states are
    there; eagerly, and captured and replayed."""
    x = {n: gpu(t) for n, t in draw(62, B, N, H, d, "bf16").items()}
    size = max(mhla.gated_workspace_size(x["q"]), mhla.gated_backward_workspace_size(x["q"]))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)

    def chain(wait):
        got, v, state = [], x["v"].clone(), x["state"].clone()
        for _ in range(3):
            v = v * 1.0
            v, state = mhla.gated_forward(x["q"], x["k"], v, x["g"], scale=0.125, state=state, workspace=ws)
            wait()
            got += [v, state]
            got += mhla.gated_backward(x["q"], x["k"], v, x["g"], x["dout"], scale=0.125, state=state, workspace=ws)
            wait()
        return got

    one_by_one = chain(torch.cuda.synchronize)
    eager = chain(lambda: None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain(lambda: None)
    for t in captured:
        t.fill_(float("nan"))
    graph.replay(), graph.replay()
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    assert all(torch.isfinite(a).all() for a in one_by_one)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(one_by_one, eager, captured))


def test_nan_stays_in_its_head():
    x = draw(34, 2, 150, 2, 64, "bf16")
    x["v"][0, 70, 1, 3] = float("nan")
    out, last = run_forward(x, 0.125)
    out, last = f64(out), f64(last)
    assert np.isnan(out[0, 70:, 1, 3]).all() and np.isnan(last[0, 1, :, 3]).all()
    out[0, 70:, 1, 3] = last[0, 1, :, 3] = 0
    assert np.isfinite(out).all() and np.isfinite(last).all()   # no other channel, head or earlier token


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("N,H,d", [(60, 2, 32), (150, 2, 64), (1500, 11, 64), (150, 2, 100)])
def test_what_is_not_finite_reaches_no_earlier_token(N, H, d, bad):
    """One value of v: its channel from its token on; one of k: the channels of v from its token on."""
    at = N // 2 + 5
    for name in ("v", "k"):
        x = draw(35, 1, N, H, d, "bf16")
        plain, _ = run_forward(x, 0.125)
        x[name][0, at, 1, 3] = bad
        out, last = run_forward(x, 0.125)
        out, last, plain = f64(out), f64(last), f64(plain)
        touched = (slice(None), 1, 3) if name == "v" else (slice(None), 1)
        assert not np.isfinite(out[0, at:][touched]).any() and np.isfinite(out[0, :at]).all()
        assert np.isfinite(out[0, :, 0]).all() and np.isfinite(last[0, 0]).all() and not np.isfinite(last[0, 1, 3, 3])
        if name == "v":
            assert np.isfinite(np.delete(out[0, :, 1], 3, axis=1)).all() and np.isfinite(np.delete(last[0, 1], 3, axis=1)).all()
        # earlier tokens: the plain values, each side within 2^-8 of its own and 2^-15 of A of the exact one
        size = oracle.gated(*(np.abs(f64(x[n]))[:, :at] for n in "qkv"), f64(x["g"])[:, :at], 0.125, magnitude(f64(x["state"])))[0]
        assert (np.abs(out[:, :at] - plain[:, :at]) <= 2.0 ** -7 * np.abs(plain[:, :at]) + 2.0 ** -13 * size).all()


@pytest.mark.parametrize("bad", [0.0, float("nan")])
@pytest.mark.parametrize("N,H,d", [(150, 2, 64), (600, 40, 64), (1500, 11, 64), (700, 3, 32), (150, 2, 100), (6000, 4, 64)])
def test_a_state_updated_in_place(N, H, d, bad):
    """The same bits as with a state of its own, on a busy machine too (whose CTAs of one call start far apart)."""
    x = draw(40, 2, N, H, d, "bf16")
    x["v"][1, N // 3, 1, 3] = bad
    args = [gpu(x[n]) for n in ("q", "k", "v", "g")]
    out, last = mhla.gated_forward(*args, scale=0.125, state=gpu(x["state"]))
    torch.cuda.synchronize()
    other, load = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    for busy in (False, True, True, True):
        state = gpu(x["state"])
        torch.cuda.synchronize()
        if busy:
            with torch.cuda.stream(other):
                for _ in range(3):
                    load @ load
        o, s = mhla.gated_forward(*args, scale=0.125, state=state, state_out=state)
        torch.cuda.synchronize()
        assert torch.equal(o.nan_to_num(7.0), out.nan_to_num(7.0)) and torch.equal(s.nan_to_num(7.0), last.nan_to_num(7.0))


@pytest.mark.parametrize("N,H", [(150, 2), (1500, 4)])
def test_a_gradient_that_is_not_finite_reaches_no_later_token(N, H):
    """dout of one token: dk and dv of its token and earlier, dq of itself."""
    x = draw(36, 1, N, H, 64, "bf16")
    at = N // 2 + 5
    x["dout"][0, at, 1, 3] = float("nan")
    dq, dk, dv, dg, dstate = (f64(t) for t in run_backward(x, 0.125))
    assert np.isfinite(dk[0, at + 1:]).all() and np.isfinite(dv[0, at + 1:]).all() and np.isfinite(dg[0, at + 1:]).all()
    assert np.isnan(dv[0, :at + 1, 1, 3]).all() and np.isfinite(np.delete(dv[0, :, 1], 3, axis=1)).all()
    assert np.isfinite(np.delete(dq[0, :, 1], at, axis=0)).all() and np.isnan(dq[0, at, 1]).all()
    for t in (dq, dk, dv):
        assert np.isfinite(t[0, :, 0]).all()
    assert np.isfinite(dstate[0, 0]).all()


def test_a_gate_that_is_nan_reaches_no_earlier_token():
    for N, H in ((60, 2), (150, 2), (1500, 11)):
        x = draw(37, 1, N, H, 64, "bf16")
        at = N // 2 + 5
        x["g"][0, at, 1] = float("nan")
        out, last = (f64(t) for t in run_forward(x, 0.125))
        assert np.isfinite(out[0, :at]).all() and np.isnan(out[0, at:, 1]).all() and np.isfinite(out[0, :, 0]).all()
        assert np.isnan(last[0, 1]).all() and np.isfinite(last[0, 0]).all()


def raw_status():
    """(status, flags) of mhla_device_status without raising."""
    import ctypes
    flags = ctypes.c_uint32(0)
    st = mhla.lib().mhla_device_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream) or None,
                                       ctypes.byref(flags))
    return int(st), int(flags.value)


# the output warps: the ones whose waits outlast a first look (the hook acts on those alone)
@pytest.mark.parametrize("warp", [16, 23])
def test_a_wait_that_gives_up_is_reported_and_the_context_recovers(warp):
    x = draw(38, 4, 1000, 6, 64, "bf16")
    assert raw_status() == (0, 0)
    mhla.debug_stall_waits(warp, 1_000_000)
    try:
        mhla.gated_forward(*(gpu(x[n]) for n in ("q", "k", "v", "g")), scale=0.125, state=gpu(x["state"]))
        torch.cuda.synchronize()
        status, flags = raw_status()
    finally:
        mhla.debug_stall_waits(-1)
    assert status == 5 and flags & 1 and not flags & 2, (status, flags)
    assert raw_status() == (0, 0)
    check_forward(x, "bf16", 0.125, *run_forward(x, 0.125))
