"""Rotation tables that cannot be meant are refused before anything is queued: no GPU is used."""

import ctypes

import pytest
import torch

import token_level_head_block_gb300 as mhla

UNSUPPORTED = 3
FAKE = 1 << 40          # never dereferenced


def test_a_table_without_rows():
    """Without rows there is no cosine to turn by: not the same as no table."""
    x = torch.zeros(1, 3, 2, 64)
    with pytest.raises(ValueError, match="rows"):
        mhla.qk_norm(x, x, table=torch.zeros(0, 16, 2), positions=torch.zeros(1, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="rows"):
        mhla.qk_norm_backward(x, x, x, x, table=torch.zeros(0, 16, 2))


@pytest.mark.parametrize("rows", [(1 << 40) + 1, 1 << 58, (1 << 63) - 1])
def test_more_rows_than_memory_has(rows):
    """Their size in bytes would not fit 64 bits, and the check for overlaps needs it."""
    L = mhla.lib()
    t = lambda i: mhla.tensor_desc(FAKE + (i << 30), "bf16", (1, 3, 2, 64), (384, 128, 64))
    rot = mhla.Rotation(FAKE + (9 << 30), FAKE + (10 << 30), rows, 32, 0)
    d = [ctypes.byref(t(i)) for i in range(6)]
    assert L.mhla_qk_norm(d[0], d[1], None, None, 1e-6, rot, d[2], d[3], None) == UNSUPPORTED
    assert L.mhla_qk_norm_backward(d[0], d[1], None, None, 1e-6, rot, d[2], d[3], d[4], d[5], None, None, None, 0,
                                   None) == UNSUPPORTED
