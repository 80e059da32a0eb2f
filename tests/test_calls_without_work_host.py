"""Calls with nothing to compute, and arguments that a call does not use: host checks, no kernel is launched."""

import ctypes

import pytest

import token_level_head_block_gb300 as mhla

OK, INVALID, SHAPE, UNSUPPORTED, CUDA, TIMEOUT, WORKSPACE = range(7)
FAKE = 1 << 40          # never dereferenced
STEP = 1 << 32


@pytest.fixture(scope="module")
def L():
    return mhla.lib()


def at(i, off=0):
    return FAKE + i * STEP + off


def test_gradients_of_keys_that_no_value_head_reads_are_refused(L):
    """dq and dk have elements, nothing would write them; the forward has nothing to leave unwritten."""
    def t(i, heads, d=64):
        return mhla.tensor_desc(at(i), "bf16", (2, 5, heads, d), (5 * max(heads, 1) * d, max(heads, 1) * d, d))

    keys, none = lambda i: ctypes.byref(t(i, 2)), lambda i, d=64: ctypes.byref(t(i, 0, d))
    args = (keys(0), keys(1), none(2), none(3, 1), none(4, 1))
    assert L.mhla_delta_forward(*args, 1.0, None, none(5), None, None, 0, None) == OK
    assert L.mhla_delta_backward(*args, none(5), 1.0, None, None, keys(6), keys(7), none(8), none(9, 1), none(10, 1), None, None, 0,
                                 None) == SHAPE


def test_gradients_of_no_sequences_have_nothing_to_write(L):
    """B = 0: dq and dk have no elements whatever the heads."""
    t = lambda heads, d=64: ctypes.byref(mhla.tensor_desc(0, "bf16", (0, 5, heads, d), (1, 1, 1)))
    args = (t(2), t(2), t(0), t(0, 1), t(0, 1))
    assert L.mhla_delta_backward(*args, t(0), 1.0, None, None, t(2), t(2), t(0), t(0, 1), t(0, 1), None, None, 0, None) == OK


def test_pre_is_not_looked_at_without_an_activation(L):
    """With MHLA_ACT_NONE it may be anything, the place of a result too: the checks end at the workspace, made too small here."""
    n = ctypes.c_size_t()
    assert L.mhla_linear_act_backward_workspace_size(300, 64, 96, 0, 0, ctypes.byref(n)) == OK and n.value > 0
    for pre in (None, at(3), at(3, 8), at(4), at(5), at(6)):
        got = L.mhla_linear_act_backward(at(0), at(1), at(2), pre, 0, at(4), at(5), at(6), 300, 64, 96, 0, at(9), n.value - 1, None)
        assert got == WORKSPACE
    assert L.mhla_linear_act_backward(at(0), at(1), at(2), at(4), 4, at(4), at(5), at(6), 300, 64, 96, 0, at(9), 16, None) == INVALID
