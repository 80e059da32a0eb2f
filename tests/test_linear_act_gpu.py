"""The linear layer with activation and residual, and its gradients, against the float64 oracle.

Tolerances.  The tensor core adds products to float32 sums, each addition off by at most a step, 2^-23 of the
largest sum, so z is within K 2^-23 A, A = sum |x||w| + |bias| (float32 operands: their three terms' remainder, 2^-24 each and
the dropped products', is covered by twice that).  An activation passes at most 1.2 times an error on; its own
arithmetic is good to 2^-18 (bf16 calls; their result is rounded to 2^-8) or 2^-21 of |z| + 1.  Gradients: dz is rounded to the type
(half a step of |dz|) and summed the same way.
"""

import numpy as np
import pytest
import torch

import oracle
import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
OWN = {"bf16": 2.0 ** -18, "f32": 2.0 ** -21}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]

# rows, k, n: one of each, few rows (a kernel of their own) to its limits, around the tiles of 128 and 64, odd sizes, K in parts
SHAPES = [(1, 1, 1), (1, 768, 520), (3, 7, 5), (8, 40, 33), (9, 264, 64), (33, 72, 50), (64, 136, 200), (65, 136, 200), (65, 77, 130),
          (128, 64, 64), (129, 65, 65), (300, 200, 136), (1000, 33, 17), (257, 1032, 72), (70, 2000, 260), (520, 192, 640), (1500, 264, 520),
          (700, 4100, 136), (3000, 72, 1288)]


def draw(seed, rows, k, n, dtype):
    r = np.random.default_rng(seed)
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))
    x = {"x": f(rows, k), "w": f(n, k) / k ** 0.5, "bias": f(n), "residual": f(rows, n), "dout": f(rows, n)}
    return {name: t.to(DT[dtype]) for name, t in x.items()}


def f64(t):
    return t.detach().cpu().double().numpy()


def within(name, got, ref, bound):
    got = f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    over = np.abs(got - ref) - bound
    assert over.max() <= 0, f"{name}: {np.abs(got - ref).max():.3e} off, {over.max():.3e} over"


def check(x, dtype, act, bias, residual, out, pre=None):
    a, w = f64(x["x"]), f64(x["w"])
    b, s = f64(x["bias"]) if bias else None, f64(x["residual"]) if residual else None
    ref, z = oracle.linear_act(a, w, b, act, s)
    A = np.abs(a) @ np.abs(w).T + (np.abs(b) if bias else 0)
    off = 2 * (a.shape[1] + 4) * 2.0 ** -23 * A
    y = np.abs(ref) if s is None else np.abs(ref) + np.abs(s)
    within("out", out, ref, HALF[dtype] * np.abs(ref) + 1.2 * off + OWN[dtype] * (np.abs(z) + 1) * (act != "none") + 2.0 ** -23 * y + 1e-30)
    if pre is not None:
        within("pre", pre, z, HALF[dtype] * np.abs(z) + off + 1e-30)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act,bias,residual,keep", [("silu", True, False, True), ("none", False, True, False), ("gelu_tanh", True, True, True)])
def test_forward(shape, dtype, act, bias, residual, keep):
    x = draw(sum(shape), *shape, dtype)
    g = {n: t.to(DEV) for n, t in x.items()}
    # what lies behind the results stays
    room = torch.full((2, shape[0] * shape[2] + 64), 7.0, dtype=DT[dtype], device=DEV)
    out, pre = (room[i, :shape[0] * shape[2]].view(shape[0], shape[2]) for i in range(2)) if room.stride(0) % 8 == 0 else (
        torch.empty(shape[0], shape[2], dtype=DT[dtype], device=DEV) for _ in range(2))
    got = mhla.linear_act(g["x"], g["w"], g["bias"] if bias else None, act, g["residual"] if residual else None, out=out,
                          pre=pre if keep else None)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0 and got is out
    check(x, dtype, act, bias, residual, out, pre if keep else None)
    assert (room[:, shape[0] * shape[2]:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [5, 200])
@pytest.mark.parametrize("act", ACTS)
def test_activations(act, rows, dtype):
    """Over their whole range: x of one column, so that z is what the test sets."""
    z = torch.linspace(-40, 40, rows * 8).view(rows, 8).to(DT[dtype])
    x = {"x": torch.eye(8).repeat(rows // 8 + 1, 1)[:rows].to(DT[dtype]), "w": torch.zeros(24, 8, dtype=DT[dtype])}
    x["w"][:8] = z[:8, :8] if rows >= 8 else torch.linspace(-40, 40, 64).view(8, 8).to(DT[dtype])
    x["w"][8:16] = torch.linspace(-6, 6, 64).view(8, 8).to(DT[dtype])
    x["w"][16:] = torch.linspace(-0.5, 0.5, 64).view(8, 8).to(DT[dtype])
    out = mhla.linear_act(x["x"].to(DEV), x["w"].to(DEV), activation=act)
    torch.cuda.synchronize()
    check(x, dtype, act, False, False, out)


def check_backward(x, dtype, act, pre, got, bias=True):
    a, w, do = f64(x["x"]), f64(x["w"]), f64(x["dout"])
    dx, dw, db = oracle.linear_act_backward(a, w, do, act, None if pre is None else f64(pre))
    dz = np.abs(do) if act == "none" else np.abs(do * oracle.activation(f64(pre), act)[1])
    # slope: a share of 1 + |z| on the way, then the rounding of dz
    own = 0.0 if act == "none" else 2.0 ** -20 * np.abs(do) * (1 + np.abs(f64(pre)))
    e = (HALF[dtype] if act != "none" or dtype == "f32" else 0.0) * dz + own
    for name, g, ref, A, E, K in (("dx", got[0], dx, dz @ np.abs(w), e @ np.abs(w), w.shape[0]),
                                  ("dw", got[1], dw, dz.T @ np.abs(a), e.T @ np.abs(a), a.shape[0]),
                                  ("dbias", got[2], db, dz.sum(0), own.sum(0) if act != "none" else 0.0, a.shape[0])):
        if name == "dbias" and not bias:
            assert g is None
            continue
        within(name, g, ref, HALF[dtype] * np.abs(ref) + 2 * (K + 4) * 2.0 ** -23 * A + E + 1e-30)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act,bias", [("gelu", True), ("none", True), ("silu", False)])
def test_backward(shape, dtype, act, bias):
    x = draw(sum(shape) + 1, *shape, dtype)
    g = {n: t.to(DEV) for n, t in x.items()}
    pre = torch.empty(shape[0], shape[2], dtype=DT[dtype], device=DEV)
    mhla.linear_act(g["x"], g["w"], g["bias"], act, pre=pre)
    got = mhla.linear_act_backward(g["x"], g["w"], g["dout"], act, None if act == "none" else pre, bias=bias)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    check_backward(x, dtype, act, pre, got, bias)


# what the small ones above do not reach: pairs of CTAs on tiles of 256 rows, each width of tile, the long axis in parts
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(300, 768, 8192), (700, 200, 4096), (300, 200, 8192), (129, 65536, 200), (129, 65536, 192),
                                   (129, 65536, 100), (257, 65536, 256), (65, 65536, 384), (65, 65536, 1000), (65, 65536, 192)], ids=str)
def test_forward_of_every_cutting(shape, dtype):
    x = draw(sum(shape), *shape, dtype)
    g = {n: t.to(DEV) for n, t in x.items()}
    pre = torch.empty(shape[0], shape[2], dtype=DT[dtype], device=DEV)
    out = mhla.linear_act(g["x"], g["w"], g["bias"], "silu", g["residual"], pre=pre)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    check(x, dtype, "silu", True, True, out, pre)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(300, 8192, 768), (129, 8192, 8), (768, 8192, 300), (129, 192, 65536), (65536, 192, 129),
                                   (65536, 100, 129), (65536, 256, 257)], ids=str)
def test_backward_of_every_cutting(shape, dtype):
    x = draw(sum(shape) + 1, *shape, dtype)
    g = {n: t.to(DEV) for n, t in x.items()}
    got = mhla.linear_act_backward(g["x"], g["w"], g["dout"])
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    check_backward(x, dtype, "none", None, got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "gelu_tanh"])
def test_slopes(act, dtype):
    """x = 1 and w = 1 of one column each: dx is the slope times dout."""
    z = torch.cat((torch.linspace(-40, 40, 161), torch.linspace(-2, 2, 161), torch.tensor([0.0, 1e30, -1e30]))).to(DT[dtype])
    rows = z.numel()
    x = {"x": torch.ones(rows, 1, dtype=DT[dtype]), "w": torch.ones(1, 1, dtype=DT[dtype]), "dout": torch.ones(rows, 1, dtype=DT[dtype])}
    got = mhla.linear_act_backward(*(x[n].to(DEV) for n in ("x", "w", "dout")), act, z[:, None].to(DEV))
    torch.cuda.synchronize()
    ref = oracle.activation(np.clip(f64(z), -100, 100), act)[1][:, None]
    within("dx", got[0], ref, 2 * HALF[dtype] * np.abs(ref) + 2.0 ** -18)


@pytest.mark.parametrize("rows", [3, 90, 700])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_residual_in_place_and_leading_axes(rows, dtype):
    x = draw(rows, rows, 96, 72, dtype)
    g = {n: t.to(DEV) for n, t in x.items()}
    out = g["residual"].clone().view(1, rows, 72)
    got = mhla.linear_act(g["x"].view(1, rows, 96), g["w"], g["bias"], "silu", residual=out, out=out)
    torch.cuda.synchronize()
    assert got is out and got.shape == (1, rows, 72)
    check(x, dtype, "silu", True, True, out[0])


def test_same_result_as_linear():
    """Without activation and residual: the sums of mhla_linear, each rounded once (its tiles add in another order)."""
    x = draw(5, 400, 192, 384, "bf16")
    g = {n: t.to(DEV) for n, t in x.items()}
    a, b = mhla.linear_act(g["x"], g["w"], g["bias"]), mhla.linear(g["x"], g["w"], g["bias"])
    torch.cuda.synchronize()
    check(x, "bf16", "none", True, False, a)
    check(x, "bf16", "none", True, False, b)


def test_same_bits_every_time():
    x = draw(6, 2000, 200, 136, "f32")
    g = {n: t.to(DEV) for n, t in x.items()}
    pre = torch.empty(2000, 136, device=DEV)
    one, two = (mhla.linear_act(g["x"], g["w"], g["bias"], "gelu", pre=pre) for _ in range(2))
    a, b = (mhla.linear_act_backward(g["x"], g["w"], g["dout"], "gelu", pre) for _ in range(2))
    torch.cuda.synchronize()
    assert torch.equal(one, two) and all(torch.equal(s, t) for s, t in zip(a, b))


def test_not_finite_stays_in_its_row():
    for rows in (6, 200):
        x = draw(7, rows, 64, 48, "bf16")
        x["x"][4, 3] = float("inf")
        x["x"][5, 0] = float("nan")
        out = mhla.linear_act(x["x"].to(DEV), x["w"].to(DEV), activation="relu")
        torch.cuda.synchronize()
        assert out[5].isnan().all() and not out[4].isfinite().all()
        x["x"][4:6] = 0
        ref = mhla.linear_act(x["x"].to(DEV), x["w"].to(DEV), activation="relu")
        rest = [r for r in range(rows) if r not in (4, 5)]
        assert torch.equal(out[rest], ref[rest])


def test_stream_workspace_and_capture():
    x = draw(8, 300, 100, 60, "f32")
    g = {n: t.to(DEV) for n, t in x.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pre = torch.empty(300, 60, device=DEV)
    ws = torch.full((mhla.linear_act_workspace_size(300, 100, 60, "f32"),), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    out = mhla.linear_act(g["x"], g["w"], g["bias"], "silu", pre=pre, workspace=ws, stream=side)
    got = mhla.linear_act_backward(g["x"], g["w"], g["dout"], "silu", pre, stream=side)
    side.synchronize()
    check(x, "f32", "silu", True, False, out, pre)
    check_backward(x, "f32", "silu", pre, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mhla.linear_act(g["x"], g["w"], g["bias"], "silu", pre=pre)
        got = mhla.linear_act_backward(g["x"], g["w"], g["dout"], "silu", pre)
    y = draw(9, 300, 100, 60, "f32")
    for n in ("x", "w", "bias", "dout"):
        g[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    check(y, "f32", "silu", True, False, out, pre)
    check_backward(y, "f32", "silu", pre, got)


def test_gradients_by_differences():
    """Along random directions; the loss is smooth and the step 2^-6: the third derivative's part is h^2 of it."""
    x = draw(10, 40, 24, 20, "f32")
    g = {n: t.to(DEV) for n, t in x.items()}
    pre = torch.empty(40, 20, device=DEV)
    mhla.linear_act(g["x"], g["w"], g["bias"], "gelu_tanh", pre=pre)
    grads = dict(zip(("x", "w", "bias"), mhla.linear_act_backward(g["x"], g["w"], g["dout"], "gelu_tanh", pre)))
    loss = lambda y: (f64(mhla.linear_act(y["x"], y["w"], y["bias"], "gelu_tanh")) * f64(y["dout"])).sum()
    size = np.abs(f64(x["dout"])).sum()
    for n, grad in grads.items():
        way = torch.randn(g[n].shape, generator=torch.Generator().manual_seed(1)).to(DEV)
        way /= way.norm()
        h = 2.0 ** -6
        want = (loss({**g, n: g[n] + h * way}) - loss({**g, n: g[n] - h * way})) / (2 * h)
        assert abs((f64(grad) * f64(way)).sum() - want) <= 2.0 ** -20 * size / h + 4 * h * h * float(grad.norm())


def test_offsets_beyond_32_bits():
    """Results and gradients of more than 2^31 elements: their last rows, and sums over all rows (of ones: exact in float32)."""
    rows, k, n = (1 << 20) + 77, 24, 2056
    x = torch.ones(rows, k, dtype=torch.bfloat16, device=DEV)
    w = draw(3, 1, k, n, "bf16")["w"].to(DEV)
    assert rows * n > 1 << 31
    tail = draw(4, 500, k, n, "bf16")
    x[-500:] = tail["x"].to(DEV)
    pre = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)
    out = mhla.linear_act(x, w, activation="silu", pre=pre)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    check({"x": tail["x"], "w": w.cpu()}, "bf16", "silu", False, False, out[-500:], pre[-500:])
    x[-500:] = 1
    pre.fill_(1.0)                                                       # where the slope of relu is one
    dx, dw, db = mhla.linear_act_backward(x, w, pre, "relu", pre)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    # rows ones added exactly or each partial sum rounded (2^-24 of it, 2 rows / 64 additions); bf16 rounds the result
    for got in (dw, db):
        assert (got.double() - rows).abs().max() <= (2.0 ** -8 + rows / 32 * 2.0 ** -24) * rows
    want = f64(w).sum(0)
    assert (np.abs(f64(dx[-500:]) - want) <= 2.0 ** -8 * np.abs(want) + 2 * (n + 4) * 2.0 ** -23 * np.abs(f64(w)).sum(0)).all()


def test_no_rows():
    x, w = torch.empty(0, 16, device=DEV), torch.ones(8, 16, device=DEV)
    assert mhla.linear_act(x, w).shape == (0, 8)
    dx, dw, db = mhla.linear_act_backward(x, w, torch.empty(0, 8, device=DEV))
    torch.cuda.synchronize()
    assert dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()


def test_refusals():
    x = draw(11, 20, 32, 24, "bf16")
    g = {n: t.to(DEV) for n, t in x.items()}
    with pytest.raises(ValueError):
        mhla.linear_act(g["x"], g["w"], activation="tanh")
    with pytest.raises(ValueError):
        mhla.linear_act(g["x"], g["w"][:, :16])
    with pytest.raises(ValueError):
        mhla.linear_act(g["x"], g["w"].t().contiguous().t())
    with pytest.raises(ValueError):
        mhla.linear_act(g["x"], g["w"], bias=g["bias"].float())
    with pytest.raises(ValueError):
        mhla.linear_act(g["x"], g["w"], residual=g["residual"][:10])
    with pytest.raises(ValueError):
        mhla.linear_act(x["x"], x["w"])
    with pytest.raises(ValueError):
        mhla.linear_act_backward(g["x"], g["w"], g["dout"], "silu")        # without pre
    with pytest.raises(mhla.MhlaError):
        mhla.linear_act(g["x"].flatten()[4:4 + 18 * 32].view(18, 32), g["w"])   # 8 bytes behind a boundary of 16
    with pytest.raises(mhla.MhlaError):
        mhla.linear_act(g["x"], g["w"], out=g["dout"], pre=g["dout"])
