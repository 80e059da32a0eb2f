"""The query/key norm with rotation and its gradients against the float64 oracle.

Tolerances.  float32 arithmetic on exact inputs: mean of squares (d additions, so d 2^-24), its root and
reciprocal, two products and the turn, all below (d + 16) 2^-24 of the pair's size |a| + |b|; a bf16 result adds
its own 2^-8.  A weight's gradient sums n rows in float32: n 2^-24 of the sum of absolute values.
"""

import numpy as np
import pytest
import torch

import oracle
import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def f64(t):
    return t.detach().cpu().double().numpy()


def draw(seed, B, N, H, Hk, d, dtype, pairs=None, positions=False, rows=None):
    r = np.random.default_rng(seed)
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))
    pairs = d // 2 if pairs is None else pairs
    rows = rows or N + 7
    x = {"q": f(B, N, H, d).to(DT[dtype]), "k": (3 * f(B, N, Hk, d)).to(DT[dtype]),
         "dq_out": f(B, N, H, d).to(DT[dtype]), "dk_out": f(B, N, Hk, d).to(DT[dtype]),
         "q_weight": 1 + 0.3 * f(d), "k_weight": 1 + 0.3 * f(d),
         "table": torch.from_numpy(mhla.init_rotation((1, rows), (0, pairs), 100.0)) if pairs else None,
         "positions": torch.from_numpy(r.integers(0, rows, (B, N)).astype(np.int32)) if positions else None}
    return x


def options(x, layout, on_gpu):
    pick = (lambda t: None if t is None else t.to(DEV)) if on_gpu else (lambda t: None if t is None else t.numpy())
    o = {"table": pick(x["table"]), "positions": pick(x["positions"]), "layout": layout, "eps": EPS}
    if not on_gpu and o["table"] is not None:
        o["table"] = o["table"].astype(np.float64)
    return o


def pair_size(y, pairs, layout):
    """|a| + |b| of each channel's pair."""
    y = np.abs(y)
    a, b = (np.arange(pairs), np.arange(pairs) + pairs) if layout == "half" else (2 * np.arange(pairs),
                                                                                 2 * np.arange(pairs) + 1)
    s = y.copy()
    s[..., a] = s[..., b] = y[..., a] + y[..., b]
    return s


def within(name, got, ref, own, bound):
    got = f64(got)
    assert got.shape == ref.shape
    bad = np.isnan(ref)
    assert np.array_equal(np.isnan(got), bad), name
    over = np.where(bad, 0, np.abs(got - ref) - (own * np.abs(ref) + bound + 1e-30))
    assert over.size == 0 or over.max() <= 0, f"{name}: {over.max():.3e} over its bound"


def check_forward(x, layout, dtype, q, k):
    o = options(x, layout, False)
    u, d = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24), x["q"].shape[3]
    pairs = 0 if x["table"] is None else x["table"].shape[1]
    for name, got in (("q", q), ("k", k)):
        a, w = f64(x[name]), None if x[name + "_weight"] is None else f64(x[name + "_weight"])
        size = pair_size(oracle.qk_norm(a, w, EPS), pairs, layout)
        within(name, got, oracle.qk_norm(a, w, **o), u, (d + 16) * 2.0 ** -24 * size)


def run_forward(x, layout, **kw):
    w = [None if x[n] is None else x[n].to(DEV) for n in ("q_weight", "k_weight")]
    got = mhla.qk_norm(x["q"].to(DEV), x["k"].to(DEV), *w, **options(x, layout, True), **kw)
    torch.cuda.synchronize()
    return got


def check_backward(x, layout, dtype, got):
    o = options(x, layout, False)
    u, d = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24), x["q"].shape[3]
    pairs = 0 if x["table"] is None else x["table"].shape[1]
    for i, name in enumerate("qk"):
        a, dz = f64(x[name]), f64(x["d%s_out" % name])
        w = None if x[name + "_weight"] is None else f64(x[name + "_weight"])
        dx, dw = oracle.qk_norm_backward(a, dz, w, **o)
        r = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + EPS)
        unit = np.abs(a) * r
        dy = pair_size(dz, pairs, layout)
        m = dy if w is None else dy * np.abs(w)
        size = r * (m + unit * (m * unit).mean(-1, keepdims=True))
        within("d" + name, got[i], dx, u, 2 * (d + 16) * 2.0 ** -24 * size)
        rows = a.shape[0] * a.shape[1] * a.shape[2]
        within("d%s_weight" % name, got[2 + i], dw, 2.0 ** -24,
               (min(rows, 2048 + rows // 256) + d + 16) * 2.0 ** -24 * (dy * unit).sum((0, 1, 2)))


def run_backward(x, layout, **kw):
    w = [None if x[n] is None else x[n].to(DEV) for n in ("q_weight", "k_weight")]
    got = mhla.qk_norm_backward(*(x[n].to(DEV) for n in ("q", "k", "dq_out", "dk_out")), *w, **options(x, layout, True),
                                **kw)
    torch.cuda.synchronize()
    return got


# (B, N, H, Hk, d, pairs): head sizes on and off the vector sizes, fewer key heads, whole, partial and no rotation
SHAPES = [(1, 1, 1, 1, 64, 32), (2, 37, 3, 3, 64, 32), (3, 50, 4, 1, 128, 64), (2, 20, 5, 2, 32, 16),
          (1, 33, 2, 2, 64, 16), (2, 11, 3, 1, 40, 9), (1, 13, 2, 2, 7, 3), (1, 9, 1, 1, 1, 0), (2, 16, 2, 2, 64, 0),
          (1, 700, 12, 12, 64, 32), (1, 21, 3, 2, 96, 48), (2, 15, 2, 1, 16, 8), (2, 15, 33, 1, 8, 4), (5, 3, 2, 7, 80, 20)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,N,H,Hk,d,pairs", SHAPES)
def test_forward_and_backward(B, N, H, Hk, d, pairs, layout, dtype):
    x = draw(N + d, B, N, H, Hk, d, dtype, pairs, positions=(N % 2 == 1) and pairs > 0)
    check_forward(x, layout, dtype, *run_forward(x, layout))
    check_backward(x, layout, dtype, run_backward(x, layout))


# more tokens than a launch's groups hold at once (they go on from round to round, over the ends of sequences) and,
# in the last two, more heads than it has groups
LONG = [(7, 1999, 2, 1, 64, 32), (3, 2503, 3, 2, 128, 64), (4001, 3, 2, 1, 64, 8), (5, 2777, 1, 3, 40, 9),
        (1, 1, 34000, 1, 64, 32), (1, 2, 50000, 3, 64, 16)]


@pytest.mark.parametrize("dtype,layout", [("bf16", "half"), ("f32", "interleaved")])
@pytest.mark.parametrize("B,N,H,Hk,d,pairs", LONG)
def test_many_rounds(B, N, H, Hk, d, pairs, layout, dtype):
    x = draw(N + H, B, N, H, Hk, d, dtype, pairs, positions=B % 2 == 1)
    if x["positions"] is not None:
        x["positions"][:, ::5] = -1
    x["k"] = x["k"].transpose(1, 2).contiguous().transpose(1, 2)     # heads outside tokens
    check_forward(x, layout, dtype, *run_forward(x, layout))
    check_backward(x, layout, dtype, run_backward(x, layout))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_what_an_earlier_launch_left_in_shared_memory(layout, dtype):
    """A call whose every value is NaN, then a narrower head, some of whose lanes hold no channel."""
    nan = draw(50, 8, 1999, 3, 3, 64, dtype, positions=True)
    for n in ("q", "k", "dq_out", "dk_out"):
        nan[n].fill_(float("nan"))
    nan["positions"].fill_(10 ** 6)                                  # past the table
    x = draw(51, 3, 517, 5, 2, 40, dtype, 8)
    for _ in range(3):
        run_forward(nan, layout), run_backward(nan, layout)
        check_forward(x, layout, dtype, *run_forward(x, layout))
        run_backward(nan, layout)
        check_backward(x, layout, dtype, run_backward(x, layout))


@pytest.mark.parametrize("d", [64, 40])
def test_without_weights(d):
    x = draw(41, 2, 30, 2, 3, d, "bf16")
    x["q_weight"] = x["k_weight"] = None
    check_forward(x, "half", "bf16", *run_forward(x, "half"))
    check_backward(x, "half", "bf16", run_backward(x, "half"))


@pytest.mark.parametrize("d", [64, 40])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_padding_and_positions_past_the_table(d, layout):
    x = draw(42, 2, 12, 2, 1, d, "f32", pairs=8, positions=True)
    x["positions"][0, 3:6] = -1                                      # padding: normed, not rotated
    x["positions"][1, 2] = x["table"].shape[0]                       # past the table: NaN in the rotated channels
    x["positions"][1, 4] = 2 ** 31 - 1
    x["positions"][1, 5] = -2 ** 31
    q, k = run_forward(x, layout)
    check_forward(x, layout, "f32", q, k)
    assert torch.isnan(q[1, 2, 0, :16]).all() and torch.isfinite(q[1, 2, 0, 16:]).all()
    assert torch.isfinite(q[0]).all() and torch.isfinite(k[0]).all()


def test_zero_rows_and_large_values():
    x = draw(43, 1, 6, 2, 2, 64, "f32")
    x["q"][0, 2] = 0                                                 # 0 / sqrt(eps): zero, its gradient finite
    x["k"][0, 3] *= 1e15                                             # squares to 1e30
    check_forward(x, "half", "f32", *run_forward(x, "half"))
    check_backward(x, "half", "f32", run_backward(x, "half"))


@pytest.mark.parametrize("d", [64, 40, 7])
def test_no_eps(d):
    """eps = 0: a row that is not there (the lanes behind the last one) leaves no 0 / 0 in the sums."""
    x = draw(49, 1, 3, 3, 1, d, "f32", pairs=0)
    got = mhla.qk_norm_backward(*(x[n].to(DEV) for n in ("q", "k", "dq_out", "dk_out", "q_weight", "k_weight")), eps=0.0)
    torch.cuda.synchronize()
    for i, name in enumerate("qk"):
        dx, dw = oracle.qk_norm_backward(f64(x[name]), f64(x["d%s_out" % name]), f64(x[name + "_weight"]), 0.0)
        assert np.abs(f64(got[i]) - dx).max() <= 1e-5 * np.abs(dx).max()
        assert np.abs(f64(got[2 + i]) - dw).max() <= 1e-5 * np.abs(dw).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra", [0, 1])
def test_in_place_on_a_projection(dtype, extra):
    """q, k (and v untouched) as views of one projection's rows; an odd offset breaks 16-byte loads."""
    B, N, H, Hk, d = 2, 19, 4, 2, 64
    x = draw(44, B, N, H, Hk, d, dtype)
    row = (H + 2 * Hk) * d + extra
    buf = torch.full((B, N, row), 7.0, dtype=DT[dtype], device=DEV)
    q = buf[:, :, extra:extra + H * d].unflatten(2, (H, d))
    k = buf[:, :, extra + H * d:extra + (H + Hk) * d].unflatten(2, (Hk, d))
    q.copy_(x["q"]), k.copy_(x["k"])
    w = [x[n].to(DEV) for n in ("q_weight", "k_weight")]
    mhla.qk_norm(q, k, *w, **options(x, "half", True), q_out=q, k_out=k)
    torch.cuda.synchronize()
    check_forward(x, "half", dtype, q, k)
    assert (buf[:, :, extra + (H + Hk) * d:] == 7).all() and (buf[:, :, :extra] == 7).all()
    q.copy_(x["dq_out"]), k.copy_(x["dk_out"])                       # the gradients, in place too
    got = mhla.qk_norm_backward(x["q"].to(DEV), x["k"].to(DEV), q, k, *w, **options(x, "half", True), dq=q, dk=k)
    torch.cuda.synchronize()
    check_backward(x, "half", dtype, got)


def test_a_head_shared_by_stride_zero_and_another_order():
    x = draw(45, 2, 25, 3, 3, 64, "bf16")
    q = x["q"][:, :, :1].to(DEV).expand(-1, -1, 3, -1)
    x["q"] = q.cpu().contiguous()
    k = x["k"].transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    got = mhla.qk_norm(q, k, x["q_weight"].to(DEV), x["k_weight"].to(DEV), **options(x, "half", True))
    torch.cuda.synchronize()
    check_forward(x, "half", "bf16", *got)


def test_no_key_heads():
    x = draw(46, 2, 25, 3, 1, 64, "bf16")
    x["k"], x["dk_out"] = x["k"][:, :, :0], x["dk_out"][:, :, :0]
    q, k = run_forward(x, "half")
    assert k.shape == (2, 25, 0, 64)
    dq, dk, dwq, dwk = run_backward(x, "half")
    assert (dwk == 0).all()
    x["k"] = torch.zeros(2, 25, 1, 64, dtype=torch.bfloat16)
    x["dk_out"] = torch.zeros_like(x["k"])
    check_forward(x, "half", "bf16", q, torch.zeros(2, 25, 1, 64))
    check_backward(x, "half", "bf16", (dq, torch.zeros(2, 25, 1, 64), dwq, dwk))


def test_empty_batch_gives_zero_weight_gradients():
    x = draw(47, 1, 5, 2, 2, 64, "bf16")
    e = {n: x[n][:0].to(DEV) for n in ("q", "k", "dq_out", "dk_out")}
    got = mhla.qk_norm_backward(e["q"], e["k"], e["dq_out"], e["dk_out"], table=x["table"].to(DEV),
                                dq_weight=torch.full((64,), 3.0, device=DEV))
    torch.cuda.synchronize()
    assert (got[2] == 0).all() and (got[3] == 0).all() and got[0].shape[0] == 0


def test_the_same_bits_another_stream_and_a_replayed_graph():
    x = draw(48, 2, 500, 6, 2, 64, "bf16", positions=True)
    a, b = run_forward(x, "half") + run_backward(x, "half"), run_forward(x, "half") + run_backward(x, "half")
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    dev = {n: t.to(DEV) for n, t in x.items()}
    o = options(x, "half", True)
    w = (dev["q_weight"], dev["k_weight"])
    run = lambda stream=None: mhla.qk_norm(dev["q"], dev["k"], *w, **o, stream=stream) + mhla.qk_norm_backward(
        dev["q"], dev["k"], dev["dq_out"], dev["dk_out"], *w, **o, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = run(s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = run()
    for n in ("q", "k"):
        dev[n].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d[0], -a[0]) and torch.equal(d[3], a[3]) and torch.equal(d[4], -a[4])


def test_grid_rotation_turns_by_rows_and_columns():
    """A 2-D grid: with q and k alike everywhere, products depend on the offset of row and column alone."""
    grid, d = (5, 7), 32
    table = torch.from_numpy(mhla.init_rotation(grid, (8, 8))).to(DEV)
    r = torch.randn(2, 1, 1, 1, d, generator=torch.Generator().manual_seed(5))
    q, k = (t.expand(1, 35, 1, d).contiguous().to(DEV) for t in r)
    q, k = mhla.qk_norm(q, k, table=table)
    p = f64((q[0, :, 0] @ k[0, :, 0].T).double()).reshape(5, 7, 5, 7)
    for dy in range(-4, 5):
        for dx in range(-6, 7):
            got = [p[y, x, y + dy, x + dx] for y in range(5) for x in range(7) if 0 <= y + dy < 5 and 0 <= x + dx < 7]
            assert np.ptp(got) <= 1e-3 * d                           # torch's product may round its factors to 11 bits
