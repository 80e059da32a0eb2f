"""The sequence operators together, as a decoder layer runs them.

One layer: qkv = x W_qkv^T, q and k normed and turned in place in qkv's rows, the gated recurrence over q, k and
v of those rows, y = o W_out^T.  The stages pass bf16 rows on; the reference takes the same stages in float64 on the
bf16 values each stage was given, so each stage answers for itself and the whole for the handing over.
"""

import numpy as np
import pytest
import torch

import oracle
import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
H, D = 6, 64
C = H * D


def f64(t):
    return t.detach().cpu().double().numpy()


class Layer:
    def __init__(self, seed, rows):
        r = np.random.default_rng(seed)
        bf = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(torch.bfloat16).to(DEV)
        self.qkv_weight, self.gate_weight, self.out_weight = bf(3 * C, C) / C ** 0.5, bf(8, C) / C ** 0.5, bf(C, C) / C ** 0.5
        self.q_weight, self.k_weight = (1 + 0.1 * bf(D).float() for _ in range(2))
        self.table = torch.from_numpy(mhla.init_rotation((1, rows), (0, D // 2))).to(DEV)

    def rows(self, x, positions=None):
        """q, k (normed and turned), v as views of the projection's rows, and the gates."""
        B, N = x.shape[:2]
        qkv = mhla.linear(x, self.qkv_weight).view(B, N, 3, H, D)
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
        raw = qkv.clone()
        mhla.qk_norm(q, k, self.q_weight, self.k_weight, table=self.table, positions=positions, q_out=q, k_out=k)
        gates = torch.nn.functional.logsigmoid(mhla.linear(x, self.gate_weight)[..., :H] + 3)
        return q, k, v, gates, raw

    def prefill(self, x):
        q, k, v, g, _ = self.rows(x)
        o, state = mhla.gated_forward(q, k, v, g, scale=D ** -0.5)
        return mhla.linear(o.flatten(2), self.out_weight), state

    def decode(self, x, position, state):
        q, k, v, g, _ = self.rows(x, torch.full((x.shape[0], 1), position, dtype=torch.int32, device=DEV))
        o = mhla.gated_step(q, k, v, g, state, scale=D ** -0.5)
        return mhla.linear(o.flatten(2), self.out_weight)


def tokens(seed, B, N):
    return torch.randn(B, N, C, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("B,N", [(2, 50), (2, 200), (4, 1200)])
def test_prefill_matches_the_reference_stage_by_stage(B, N):
    layer, x = Layer(1, N), tokens(2, B, N)
    q, k, v, g, raw = layer.rows(x)
    o, state = mhla.gated_forward(q, k, v, g, scale=D ** -0.5)
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    table = f64(layer.table)
    for i, (got, w) in enumerate(((q, layer.q_weight), (k, layer.k_weight))):
        ref = oracle.qk_norm(f64(raw[:, :, i]), f64(w), table=table)
        # bf16's half step, and float32's (d + 16) 2^-24 of a pair, here below 8
        assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 4e-5).all()
    assert torch.equal(v, raw[:, :, 2])                                  # the rows' third part is as it was
    args = [f64(t) for t in (q, k, v, g)]
    ref, end = oracle.gated(*args, D ** -0.5)
    size, size_end = oracle.gated(*(np.abs(t) for t in args[:3]), args[3], D ** -0.5)
    assert (np.abs(f64(o) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * size).all()
    assert (np.abs(f64(state) - end) <= (D + 128 + N // 32 + 3) * 2.0 ** -24 * size_end).all()


def test_decoding_token_by_token_continues_the_prefill():
    """Prefill and single steps give the same rows: each stage rounds to bf16 the same way wherever its
    float32 values agree to 2^-15, so rows differ by a few bf16 steps of what the layer sums."""
    B, N, cut = 3, 140, 120
    layer, x = Layer(3, N), tokens(4, B, N)
    whole, end = layer.prefill(x)
    first, state = layer.prefill(x[:, :cut].contiguous())
    steps = [layer.decode(x[:, t:t + 1].contiguous(), t, state) for t in range(cut, N)]
    got = torch.cat([first] + steps, 1)
    torch.cuda.synchronize()
    # o of both ways is off by at most half a step each, a step of bf16 apart: 2^-7 of |o| W, C terms of random sign
    o = whole.float()
    assert (got.float() - o).norm() <= 2.0 ** -7 * o.norm()
    assert (state - end).norm() <= 2.0 ** -14 * end.norm()


def test_gradients_through_norm_and_recurrence():
    """d loss / d (qkv rows) of norm, rotation and recurrence against float64 automatic differentiation of the
    same formulas, the recurrence differentiated at the bf16 rows that the norm handed over."""
    B, N = 2, 90
    layer, x = Layer(5, N), tokens(6, B, N)
    q, k, v, g, raw = layer.rows(x)
    dout = tokens(7, B, N).view(B, N, H, D)
    dq, dk, dv, dg, _ = mhla.gated_backward(q, k, v, g, dout, scale=D ** -0.5)
    got = mhla.qk_norm_backward(raw[:, :, 0], raw[:, :, 1], dq, dk, layer.q_weight, layer.k_weight, table=layer.table,
                                dq=dq, dk=dk)
    torch.cuda.synchronize()

    t64 = lambda t: t.detach().cpu().double()
    raw64 = [t64(raw[:, :, i]).requires_grad_(i < 2) for i in range(3)]
    gate64 = t64(g).requires_grad_()
    v64 = raw64[2].clone().requires_grad_()
    weights = [t64(w).requires_grad_() for w in (layer.q_weight, layer.k_weight)]
    table = t64(layer.table)
    normed = []
    for t, w in zip(raw64[:2], weights):
        y = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a, b = y[..., :D // 2], y[..., D // 2:]
        c, s = table[None, :, None, :, 0], table[None, :, None, :, 1]
        normed.append(torch.cat((a * c - b * s, a * s + b * c), -1))
    # the recurrence sees the rounded rows; the rounding passes the gradient on
    q64, k64 = (n + (t64(r) - n).detach() for n, r in zip(normed, (q, k)))
    S, loss = torch.zeros(B, H, D, D, dtype=torch.float64), 0.0
    for t in range(N):
        S = gate64[:, t].exp()[..., None, None] * S + k64[:, t, :, :, None] * v64[:, t, :, None, :]
        loss = loss + (D ** -0.5 * (q64[:, t, :, :, None] * S).sum(-2) * t64(dout[:, t])).sum()
    loss.backward()
    want = [raw64[0].grad, raw64[1].grad, weights[0].grad, weights[1].grad]
    # dq and dk go through bf16 once on the way (2^-8) and once at the end
    for a, b in list(zip(got, want)) + [(dv, v64.grad), (dg, gate64.grad)]:
        assert float((t64(a) - b).norm()) <= 2.0 ** -7 * float(b.norm())
