"""The gradient of the log decays, dg_t = exp(g_t) <S_{t-1}, dS_t>, token by token.

Tolerance.  With A_t the same number for absolute values, exp(g_t) <|S_{t-1}|, |dS_t|>, whatever the gates: dg is a sum
of terms none of which is larger than A_t, so each rounding costs its share of A_t and not of some larger sum.  float32: both
states, or both dot products of a pair of tokens, each carry n 2^-24 (n float32 operations in a row: d of a dot product,
64 of a chunk, 64 of the decay, one or two per later chunk).  bf16 runs add 2^-15 (the state is read as two bf16
terms) and the result's own 2^-8.
"""

import numpy as np
import pytest
import torch

import oracle

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def draw(seed, B, N, H, d, dtype, state=True, remember=3.0):
    r = np.random.default_rng(seed)
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(DT[dtype])
    x = {n: f(B, N, H, d) for n in ("q", "k", "v", "dout")}
    x["g"] = torch.nn.functional.logsigmoid(f(B, N, H).float() + remember).to(DT[dtype])
    for n in ("state", "dstate_out"):
        x[n] = torch.from_numpy(r.standard_normal((B, H, d, d)).astype(np.float32)) if state else None
    return x


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def reference(x, scale, which=3):
    """(dg, A) in 64 bits."""
    q, k, v, g, do, S, dS = (f64(x[n]) for n in ("q", "k", "v", "g", "dout", "state", "dstate_out"))
    size = lambda a: None if a is None else np.abs(a)
    return (oracle.gated_backward(q, k, v, g, do, scale, S, dS)[which],
            oracle.gated_backward(size(q), size(k), size(v), g, size(do), abs(scale), size(S), size(dS))[which])


def over_bound(got, ref, A, dtype, d):
    """How far each value is over its bound."""
    N = ref.shape[1]
    own = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    slack = 2 * (d + 128 + 2 * (N // 64 + 1)) * 2.0 ** -24 + (2.0 ** -15 if dtype == "bf16" else 0.0)
    return np.abs(got - ref) - (own * np.abs(ref) + slack * A + 1e-30)


def check(x, dtype, scale, got):
    ref, A = reference(x, scale)
    got = f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all()
    over = over_bound(got, ref, A, dtype, x["q"].shape[3])
    assert over.max() <= 0, f"{(over > 0).mean():.1%} of the values over their bounds, by {over.max():.2e}"


# ------------------------------------------------------------------ what the bound sees (no GPU)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [None, -2.0, -8.0, -30.0])
def test_the_bound_refuses_what_is_wrong(gate, dtype):
    """Zeros, a sum that lost what lies behind one border of the sequence, and one carried in float32 over all tokens."""
    x = draw(1, 1, 400, 2, 16, dtype, remember=6.0)
    if gate is not None:
        x["g"][:] = gate
    ref, A = reference(x, 1.0)
    bad = lambda got: over_bound(got, ref, A, dtype, 16) > 0
    assert not bad(ref).any()
    rounded = f64(torch.from_numpy(ref).to(DT[dtype]))
    assert not bad(rounded).any()
    assert bad(np.zeros_like(ref)).mean() > 0.95
    q, k, v, g, do, S, dS = (f64(x[n]) for n in ("q", "k", "v", "g", "dout", "state", "dstate_out"))
    cut = oracle.gated_backward(q[:, 200:], k[:, 200:], v[:, 200:], g[:, 200:], do[:, 200:], 1.0, None, dS)[3]
    at = 1 if gate is not None else 10                                   # as far as the memory reaches
    assert bad(np.concatenate((ref[:, :200], cut), 1))[:, 200:200 + at].mean() > 0.9
    if gate is not None and gate <= -8:
        dq, dk = oracle.gated_backward(q, k, v, g, do, 1.0, S, dS)[:2]
        step = ((q * dq).sum(-1) - (k * dk).sum(-1)).astype(np.float32)
        end = (oracle.gated(q, k, v, g, 1.0, S)[1] * dS).sum((-1, -2)).astype(np.float32)
        run = np.cumsum(step[:, ::-1], axis=1, dtype=np.float32)[:, ::-1] + end[:, None]
        assert bad(run).mean() > (0.9 if gate <= -15 else 0.0)            # an error of a sum of ones, a value of e^gate


# ------------------------------------------------------------------ the kernels

gpu = pytest.mark.gpu


def dev(t):
    return None if t is None else t.cuda()


def run(x, scale, **kw):
    import token_level_head_block_gb300 as mhla
    got = mhla.gated_backward(*(dev(x[n]) for n in ("q", "k", "v", "g", "dout")), scale=scale, state=dev(x["state"]),
                              dstate_out=dev(x["dstate_out"]), **kw)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    return got


# (B, N, H, d): lengths around a block of 16 tokens, a chunk and several spans, head sizes on and off the tile sizes, one
# wave of CTAs and several; bf16 takes both kernels
SHAPES = [(1, 1, 1, 64), (2, 2, 3, 64), (1, 15, 2, 16), (2, 17, 2, 32), (1, 63, 2, 32), (2, 64, 2, 64), (1, 65, 1, 128),
          (2, 129, 3, 64), (1, 200, 2, 48), (1, 130, 2, 7), (1, 97, 1, 1), (2, 300, 2, 100), (1, 2500, 1, 32), (40, 70, 9, 32),
          (1, 900, 2, 128), (2, 700, 3, 70), (3, 600, 2, 36), (2, 700, 3, 72),
          (1, 769, 4, 64), (2, 520, 6, 40), (1, 1500, 5, 64), (20, 1030, 8, 8), (7, 300, 8, 64), (1, 385, 8, 24)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,d", SHAPES)
@pytest.mark.parametrize("state", [True, False], ids=["state", "empty"])
def test_every_token(B, N, H, d, dtype, state):
    x = draw(5 * N + d, B, N, H, d, dtype, state)
    check(x, dtype, d ** -0.5, run(x, d ** -0.5)[3])


@gpu
@pytest.mark.parametrize("dtype,B,N,H,d", [("f32", 1, 1500, 1, 32), ("bf16", 1, 1500, 11, 64), ("bf16", 1, 700, 2, 96),
                                           ("bf16", 6, 1100, 10, 32)])
@pytest.mark.parametrize("gate", [0.0, -2.0, -5.0, -8.0, -12.0, -15.0, -30.0, -60.0])
def test_gates_that_forget(gate, dtype, B, N, H, d):
    x = draw(6, B, N, H, d, dtype)
    x["g"][:] = gate
    check(x, dtype, 1.0, run(x, 1.0)[3])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,d", [(2, 500, 2, 64), (2, 900, 9, 64), (1, 400, 3, 128)])
def test_a_few_strong_gates_among_mild_ones(B, N, H, d, dtype):
    """At the edges of blocks and chunks, side by side, at the first and the last token."""
    x = draw(7, B, N, H, d, dtype, remember=6.0)
    for i, t in enumerate((0, 1, 15, 16, 31, 32, 63, 64, 65, 127, 128, 200, 255, 256, 257, N - 1)):
        x["g"][i % B, t] = (-8.0, -20.0, -60.0)[i % 3]
    check(x, dtype, 0.125, run(x, 0.125)[3])


CUTS = (0, 1, 40, 64, 200, 300, 301, 384)


@gpu
@pytest.mark.parametrize("dtype,H", [("bf16", 3), ("bf16", 40), ("f32", 3)])
@pytest.mark.parametrize("loud", [None, 2, 5])
def test_packed_sequences_are_apart(dtype, H, loud):
    """Closed gates (-inf, and below -1000) start a sequence: their dg is 0, and every sequence has the dg it has alone,
    also beside one whose values are 10^4 times larger."""
    N, d = 500, 32
    x = draw(8, 1, N, H, d, dtype, state=False)
    ends = CUTS[1:] + (N,)
    for i, t in enumerate(CUTS):
        x["g"][:, t] = float("-inf") if i % 2 else -2000.0
    if loud is not None:
        for n in ("q", "k", "v", "dout"):
            x[n][:, CUTS[loud]:ends[loud]] *= 1e4
    dg = run(x, 1.0)[3]
    assert (dg[:, list(CUTS)] == 0).all()
    for a, b in zip(CUTS, ends):
        alone = {n: (t[:, a:b] if t is not None else None) for n, t in x.items()}
        check(alone, dtype, 1.0, dg[:, a:b])


@gpu
@pytest.mark.parametrize("dtype,H", [("bf16", 2), ("bf16", 24), ("f32", 2)])
def test_an_empty_state_has_no_gradient(dtype, H):
    """Tokens in front of which nothing was added to the state, and ones behind which nothing is read."""
    N = 700
    x = draw(9, 1, N, H, 64, dtype, state=False)
    x["k"][:, :150] = 0
    x["dout"][:, 400:] = 0
    dg = run(x, 0.125)[3]
    assert (dg[:, :151] == 0).all() and (dg[:, 400:] == 0).all()
    check(x, dtype, 0.125, dg)


@gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,N,H,d", [("bf16", 60, 2, 32), ("bf16", 150, 2, 64), ("bf16", 1500, 11, 64), ("bf16", 150, 2, 100),
                                         ("f32", 300, 2, 48)])
def test_what_is_not_finite_stays_on_its_side(dtype, N, H, d, bad):
    """k and v of a token enter dg of later tokens alone, q and dout of it and earlier ones alone."""
    at = N // 2 + 5
    x = draw(10, 1, N, H, d, dtype)
    ref, A = reference(x, 0.125)
    for name in ("q", "k", "v", "dout"):
        y = {n: (t.clone() if t is not None else None) for n, t in x.items()}
        y[name][0, at, 1, 3] = bad
        dg = f64(run(y, 0.125)[3])
        apart = slice(0, at + 1) if name in "kv" else slice(at + 1, N)
        touched = slice(at + 1, N) if name in "kv" else slice(0, at + 1)
        assert not np.isfinite(dg[0, touched, 1]).any(), name
        keep = np.ones((N, H), bool)
        keep[touched, 1] = False
        assert np.isfinite(dg[0][keep]).all(), name
        assert over_bound(dg, ref, A, dtype, d)[0][keep].max() <= 0, name
        assert keep[apart, 1].all()


@gpu
def test_nothing_beside_the_gradients_is_written():
    """dg as a strided view; rows behind and beside it as they were."""
    x = draw(11, 2, 333, 3, 64, "bf16")
    buf = torch.full((2, 340, 7), 5.0, dtype=torch.bfloat16, device="cuda")
    dg = buf[:, :333, 2:5]
    got = run(x, 0.125, dg=dg)
    assert got[3].data_ptr() == dg.data_ptr()
    check(x, "bf16", 0.125, dg)
    assert (buf[:, 333:] == 5).all() and (buf[:, :, :2] == 5).all() and (buf[:, :, 5:] == 5).all()


@gpu
@pytest.mark.parametrize("dtype,B,N,H,d", [("bf16", 2, 300, 3, 80), ("bf16", 2, 300, 3, 100), ("f32", 1, 300, 2, 72), ("f32", 2, 130, 3, 40),
                                           ("f32", 1, 200, 2, 17), ("bf16", 6, 1100, 10, 24), ("bf16", 1, 1500, 11, 40), ("f32", 2, 64, 3, 64)])
def test_the_workspace_is_what_was_asked_for(dtype, B, N, H, d):
    """Stale contents in it, a guard behind it; the same bits as with the library's own."""
    import token_level_head_block_gb300 as mhla
    x = draw(12, B, N, H, d, dtype)
    size = mhla.gated_backward_workspace_size(x["q"].cuda())
    buf = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")      # NaN as floats
    got, plain = run(x, 0.125, workspace=buf[:size]), run(x, 0.125)
    assert (buf[size:] == 0xFF).all()
    assert all(torch.equal(a, b) for a, b in zip(got, plain))
    check(x, dtype, 0.125, got[3])
