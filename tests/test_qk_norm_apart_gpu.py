"""Channels that the rotation does not turn keep to themselves: what is not finite in one stays in it.

Behind the rotated pairs, and in every channel of a token without a position, a NaN or infinite weight or gradient
reaches its own channel alone; a turned pair shares it.  The values' tolerance is (d + 16) 2^-24 of the pair's size for float32
and 2^-8 of the value beside it for bf16 (inputs of magnitude below 8, weights below 3).
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


def same(name, got, ref, dtype, size):
    got = f64(got)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), name
    ok = np.isfinite(ref)
    own = 2.0 ** -8 if dtype == "bf16" else 0.0
    assert (np.abs(got[ok] - ref[ok]) <= own * np.abs(ref[ok]) + 144 * 2.0 ** -24 * size).all(), name


# head sizes and pairs that the vector path takes, and two that it does not
@pytest.mark.parametrize("layout,d,pairs", [("half", 64, 16), ("half", 32, 4), ("half", 128, 32), ("interleaved", 64, 16),
                                            ("interleaved", 64, 13), ("interleaved", 40, 9), ("half", 40, 9), ("half", 64, 0),
                                            ("interleaved", 16, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_unturned_channels_are_apart(bad, dtype, layout, d, pairs):
    B, N, H = 2, 23, 3
    r = np.random.default_rng(d + pairs)
    f = lambda *s: torch.from_numpy(np.clip(r.standard_normal(s), -4, 4).astype(np.float32))
    x, dz = f(B, N, H, d).to(DT[dtype]), f(B, N, H, d).to(DT[dtype])
    table = torch.from_numpy(mhla.init_rotation((1, N), (0, pairs), 100.0)) if pairs else None
    positions = torch.from_numpy(r.integers(1, N, (B, N)).astype(np.int32))
    positions[:, ::4] = -1
    o = {"eps": 1e-6, "layout": layout, "table": table.numpy().astype(np.float64) if pairs else None,
         "positions": positions.numpy()}
    on = {"eps": 1e-6, "layout": layout, "table": table.cuda() if pairs else None, "positions": positions.cuda() if pairs else None}
    for at in sorted({d - 1, 2 * pairs, 0, min(2 * pairs + 1, d - 1)}):
        if at >= d:
            continue
        w = 1 + 0.3 * f(d)
        w[at] = bad
        got = mhla.qk_norm(x.cuda(), x.cuda(), w.cuda(), w.cuda(), **on)
        with np.errstate(invalid="ignore"):
            ref = oracle.qk_norm(f64(x), f64(w), **o)
        for g in got:
            same(f"weight {at}", g, ref, dtype, 64.0)
        w[at] = 1.0
        z = dz.clone()
        z[0, 0, 1, at] = bad                                              # of a token without a position
        z[1, 2, 0, at] = bad
        got = mhla.qk_norm_backward(x.cuda(), x.cuda(), z.cuda(), z.cuda(), w.cuda(), w.cuda(), **on)
        with np.errstate(invalid="ignore"):
            dx, dw = oracle.qk_norm_backward(f64(x), f64(z), f64(w), **o)
        keep = np.ones((B, N, H), bool)                                   # a row's mean spreads it over the row
        keep[0, 0, 1] = keep[1, 2, 0] = False
        for g in got[:2]:
            same(f"gradient {at}", g.cpu()[torch.from_numpy(keep)], dx[keep], dtype, 64.0)
            assert not np.isfinite(f64(g)[~keep]).any()
        for g in got[2:]:
            assert np.array_equal(np.isfinite(f64(g)), np.isfinite(dw)), at
