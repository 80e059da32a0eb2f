"""The same call gives the same bits: gradients that reuse every tile of shared memory many times.

In the tcgen05 scan a tile is loaded by TMA, rewritten by ordinary stores with the rows that go out, and loaded again; the
order of the two kinds of writes shows, if anywhere, as bits that differ from call to call.
"""

import pytest
import torch

import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


# whole heads and heads of 32 channels (the second half of whose output warps has no channel), one wave of CTAs and several
@pytest.mark.parametrize("B,N,H,d", [(4, 4096, 12, 64), (2, 4096, 70, 32), (1, 2304, 60, 24), (3, 1111, 20, 40)])
def test_gradients_repeat_bit_by_bit(B, N, H, d):
    gen = torch.Generator(device=DEV).manual_seed(N + H)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    q, k, v, dout = (normal(B, N, H, d).bfloat16() for _ in range(4))
    g = torch.nn.functional.logsigmoid(normal(B, N, H) + 3).bfloat16()
    load, other = normal(4096, 4096), torch.cuda.Stream()
    first = None
    for turn in range(8):
        torch.cuda.synchronize()
        if turn % 2:
            with torch.cuda.stream(other):
                load @ load
        got = mhla.gated_backward(q, k, v, g, dout, scale=d ** -0.5)
        torch.cuda.synchronize()
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got)), turn
    assert mhla.device_status() == 0
    assert all(torch.isfinite(t).all() for t in first)
