"""Rotation tables that cannot be meant are refused before anything is queued: no GPU is used."""

import pytest
import torch

import token_level_head_block_gb300 as mhla


def test_a_table_without_rows():
    """Without rows there is no cosine to turn by: not the same as no table."""
    x = torch.zeros(1, 3, 2, 64)
    with pytest.raises(ValueError, match="rows"):
        mhla.qk_norm(x, x, table=torch.zeros(0, 16, 2), positions=torch.zeros(1, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="rows"):
        mhla.qk_norm_backward(x, x, x, x, table=torch.zeros(0, 16, 2))
