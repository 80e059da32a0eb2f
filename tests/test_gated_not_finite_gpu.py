"""Gradients of the gated recurrence beside a gate that is not a number.

dS_i holds the gates behind token i alone and S_i those up to it, so a NaN gate at t leaves dk and dv of t and later tokens,
and dq of earlier ones, as they are: the values of a call in which that gate is a number.  dg needs all gates.
Tolerance: both calls are within 2^-8 |ref| + 2^-15 A (bf16) or n 2^-24 A (float32) of the exact value, A the sum over absolute values.
"""

import numpy as np
import pytest
import torch

import oracle
import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("dtype,N,H,d", [("bf16", 60, 2, 32), ("bf16", 150, 2, 64), ("bf16", 1500, 11, 64), ("bf16", 700, 24, 32),
                                         ("bf16", 200, 2, 100), ("f32", 150, 2, 48), ("f32", 150, 1, 128)])
@pytest.mark.parametrize("where", [0, 1, 2, 3])
def test_a_gate_that_is_nan(where, dtype, N, H, d):
    at = (0, N // 2 + 5, 33, N - 1)[where]
    r = np.random.default_rng(N + where)
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(DT[dtype])
    q, k, v, dout = (f(1, N, H, d) for _ in range(4))
    g = torch.nn.functional.logsigmoid(f(1, N, H).float() + 3).to(DT[dtype])
    S, dS = (torch.from_numpy(r.standard_normal((1, H, d, d)).astype(np.float32)) for _ in range(2))
    ref = oracle.gated_backward(*(f64(t) for t in (q, k, v, g, dout)), 0.125, f64(S), f64(dS))
    size = oracle.gated_backward(*(np.abs(f64(t)) for t in (q, k, v)), f64(g), np.abs(f64(dout)), 0.125, np.abs(f64(S)),
                                 np.abs(f64(dS)))
    g[0, at, 0] = float("nan")
    got = mhla.gated_backward(*(t.cuda() for t in (q, k, v, g, dout)), scale=0.125, state=S.cuda(), dstate_out=dS.cuda())
    torch.cuda.synchronize()
    assert mhla.device_status() == 0
    own = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    slack = 2.0 ** -15 if dtype == "bf16" else (d + 128 + 2 * (N // 64 + 1)) * 2.0 ** -24
    touched = {"dq": slice(at, N), "dk": slice(0, at), "dv": slice(0, at)}
    for name, a, want, A in zip(("dq", "dk", "dv"), got, ref, size):
        a = f64(a)
        keep = np.ones((N, H), bool)
        keep[touched[name], 0] = False
        assert np.isnan(a[0][~keep]).all(), name
        assert np.isfinite(a[0][keep]).all(), name
        assert (np.abs(a - want) <= own * np.abs(want) + slack * A)[0][keep].all(), name
    dg, dstate = f64(got[3]), f64(got[4])
    assert np.isnan(dg[0, :, 0]).all() and np.isfinite(dg[0, :, 1:]).all()
    assert np.isnan(dstate[0, 0]).all() and np.isfinite(dstate[0, 1:]).all()
