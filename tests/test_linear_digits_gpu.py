"""The linear layer where nothing may be off: sums of whole numbers, which float32 holds exactly however K is cut, the activations'
tails relative to their own size, and what lies around the results."""

import math

import numpy as np
import pytest
import torch

import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}

# around every kernel, width of tile and number of parts of K: few rows, one CTA, pairs, long K
SHAPES = [(1, 1, 1), (1, 768, 520), (8, 40, 33), (9, 264, 64), (33, 72, 50), (64, 136, 200), (65, 77, 130), (129, 65, 65), (257, 1032, 72),
          (70, 2000, 260), (700, 4100, 136), (3000, 72, 1288), (300, 768, 8192), (700, 200, 4096), (129, 65536, 200), (129, 65536, 192),
          (129, 65536, 100), (257, 65536, 256), (65, 65536, 384), (65, 65536, 1000)]
BACK = SHAPES[:12] + [(300, 8192, 768), (129, 8192, 8), (768, 8192, 300), (129, 192, 65536), (65536, 192, 129), (65536, 100, 129),
                      (65536, 256, 257), (20000, 768, 2304)]


def whole(seed, rows, cols, dtype):
    """-1, 0 and 1."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-1, 2, (rows, cols), generator=g, device=DEV).to(DT[dtype])


def exact(a, b):
    return a.double() @ b.double()


class Rooms:
    """Results that each lie inside an array of sevens, on a boundary of 16 bytes."""

    def __init__(self, dtype):
        self.dtype, self.all = DT[dtype], []

    def __call__(self, *shape):
        n = math.prod(shape)
        flat = torch.full((64 + n + 67,), 7.0, dtype=self.dtype, device=DEV)
        self.all.append((flat, n))
        return flat[64:64 + n].view(shape)

    def untouched(self):
        return all((f[:64] == 7).all() and (f[64 + n:] == 7).all() for f, n in self.all)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rest", [False, True], ids=["alone", "bias_residual_pre"])
def test_sums_of_whole_numbers(shape, rest, dtype):
    """Every sum is below 2^24: float32 has it exactly in any order, and a result is its one rounding."""
    rows, k, n = shape
    x, w = whole(1, rows, k, dtype), whole(2, n, k, dtype)
    room = Rooms(dtype)
    out, pre = room(rows, n), room(rows, n) if rest else None
    bias, residual = (whole(3, 1, n, dtype)[0], whole(4, rows, n, dtype)) if rest else (None, None)
    mhla.linear_act(x, w, bias, residual=residual, out=out, pre=pre)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0 and room.untouched()
    z = exact(x, w.t()) + (bias.double() if rest else 0)
    if rest:
        assert torch.equal(pre, z.to(DT[dtype]))
        z = z + residual.double()
    assert torch.equal(out, z.to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", BACK, ids=str)
@pytest.mark.parametrize("act", ["none", "relu"])
def test_gradients_of_whole_numbers(shape, act, dtype):
    """The slope of relu is 0 or 1, so dz stays whole."""
    rows, k, n = shape
    x, w, dout = whole(5, rows, k, dtype), whole(6, n, k, dtype), whole(7, rows, n, dtype)
    pre = whole(8, rows, n, dtype) if act == "relu" else None
    dz = dout * (pre > 0) if act == "relu" else dout
    room = Rooms(dtype)
    dx, dw, dbias = room(rows, k), room(n, k), room(n)
    mhla.linear_act_backward(x, w, dout, act, pre, dx=dx, dw=dw, dbias=dbias)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0 and room.untouched()
    assert torch.equal(dx, exact(dz, w).to(DT[dtype]))
    assert torch.equal(dw, exact(dz.t(), x).to(DT[dtype]))
    assert torch.equal(dbias, dz.double().sum(0).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(129, 65536, 200), (65, 65536, 384), (700, 4100, 136)], ids=str)
def test_long_sums_of_random_values(shape, dtype):
    """K products, each addition off by at most a step of the running sum (2^-23 of it, towards zero): the sums
    themselves walk at random, sqrt(K) |x_i w_i|, and what the K additions lose has one sign as long as the sum has: 2^-23 of sqrt(K)
    of those, K times.  Chunks of 16 of K enter with one addition.  The result is many times larger than that."""
    rows, k, n = shape
    g = torch.Generator(device=DEV).manual_seed(9)
    x, w = torch.randn(rows, k, generator=g, device=DEV).to(DT[dtype]), (torch.randn(n, k, generator=g, device=DEV) / k ** 0.5).to(DT[dtype])
    out = mhla.linear_act(x, w)
    torch.cuda.synchronize()
    ref = exact(x, w.t())
    bound = HALF[dtype] * ref.abs() + 4 * (k / 16 + 16) * 2.0 ** -23 * (x.double() ** 2 @ w.double().t() ** 2).sqrt()
    assert ((out.double() - ref).abs() <= bound).all()
    assert bound.max() < 0.02 * ref.std()


# ------------------------------------------------------------------ tails


def column(z, dtype, rows):
    """x and w with x w^T = z in the first of `rows` rows or more, exactly: one channel of eight is not zero."""
    x = torch.zeros(rows, 8, dtype=DT[dtype], device=DEV)
    x[:, 0] = 1
    w = torch.zeros(z.numel(), 8, dtype=DT[dtype], device=DEV)
    w[:, 0] = z.to(DEV)
    return x, w


def tail(kind, z):
    """act(z) and act'(z) of a float64 z < 0 without cancellation."""
    erfc = np.vectorize(math.erfc, otypes=[np.float64])
    if kind == "gelu":
        half = erfc(-z / math.sqrt(2)) / 2
        return z * half, half + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = z if kind == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    du = 1.0 if kind == "silu" else math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + np.exp(-u))
    return z * p, p + z * p * (1 - p) * du


# rows: the kernels of few rows, the product's finish, and its bulk stores
@pytest.mark.parametrize("rows", [3, 20, 200, 700])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_tails_of_activations(kind, dtype, rows):
    """For z from -9 to -4 the result's own digits.  The argument of what falls (erfc, or an exponential: 41 and, in tanh's form, 66 at
    most) is known to 1.5 half steps of itself and enters as 1.5 times 2 41 (66) of them: 2^-17; what the functions themselves lose is no
    more: 2^-16."""
    z = torch.linspace(-9, -4, 1024).to(DT[dtype])
    x, w = column(z, dtype, rows)
    out = mhla.linear_act(x, w, activation=kind)
    torch.cuda.synchronize()
    want = tail(kind, z.double().numpy())[0]
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= (HALF[dtype] + 2.0 ** -16) * np.abs(want)).all(), np.abs(got / want - 1).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_tails_of_slopes(kind, dtype):
    """dz = dout act'(z) as dw of one row of ones: rounded to the type (bf16: once more as the result, the same value), float32: three
    terms.  The two parts of gelu's slope differ by z^2 - 1 >= 15 there, so little cancels; 2^-16 as above, doubled."""
    z = torch.linspace(-9, -4, 1024).to(DT[dtype])
    x, w = column(z, dtype, 1)
    ones = torch.ones(1, z.numel(), dtype=DT[dtype], device=DEV)
    _, _, dbias = mhla.linear_act_backward(x, w, ones, kind, z[None].to(DEV))
    torch.cuda.synchronize()
    want = tail(kind, z.double().numpy())[1]
    got = dbias.double().cpu().numpy()
    assert (np.abs(got - want) <= (HALF[dtype] + 2.0 ** -15) * np.abs(want)).all(), np.abs(got / want - 1).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gelu_on_both_sides(dtype):
    """On both sides and around 0, z Phi(z): erfc's argument is off by 1.5 half steps (a constant and a product), which is 1.5 z^2 of
    them in a tail; erfc itself by 8 half steps (4 steps), two products by one each."""
    z = torch.cat((torch.linspace(-4, 10, 1000), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e30, 3e38, 60.0, -60.0]))).to(DT[dtype])
    x, w = column(z, dtype, 200)
    out = mhla.linear_act(x, w, activation="gelu")
    torch.cuda.synchronize()
    d = z.double().numpy()
    want = tail("gelu", d)[0]
    got = out.double().cpu().numpy()
    share = HALF[dtype] + (1.5 * np.minimum(d, 0.0) ** 2 + 10) * 2.0 ** -24
    assert (np.abs(got - want) <= np.where(want == 0, 0.0, share * np.abs(want) + 1e-38)).all()
