"""The linear layer's digits: the activations' tails relative to their own size."""

import math

import numpy as np
import pytest
import torch

import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


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
