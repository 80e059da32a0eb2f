"""Host-side checks of the linear layer with activation and residual: no GPU, no kernel is launched."""

import ctypes

import pytest

import token_level_head_block_gb300 as mhla

OK, INVALID, SHAPE, UNSUPPORTED, CUDA, TIMEOUT, WORKSPACE = range(7)
FAKE = 1 << 40
STEP = 1 << 32


@pytest.fixture(scope="module")
def L():
    return mhla.lib()


def at(i, off=0):
    return FAKE + i * STEP + off


def forward(L, x=at(0), w=at(1), bias=at(2), act=4, residual=at(3), pre=at(4), out=at(5), rows=300, k=64, n=96, dtype=0, ws=None,
            ws_bytes=0):
    return L.mhla_linear_act(x, w, bias, act, residual, pre, out, rows, k, n, dtype, ws, ws_bytes, None)


def backward(L, x=at(0), w=at(1), dout=at(2), pre=at(3), act=4, dx=at(4), dw=at(5), dbias=at(6), rows=300, k=64, n=96, dtype=0,
             ws=None, ws_bytes=0):
    return L.mhla_linear_act_backward(x, w, dout, pre, act, dx, dw, dbias, rows, k, n, dtype, ws, ws_bytes, None)


def test_sizes(L):
    for call in (forward, backward):
        for kw in (dict(rows=-1), dict(k=0), dict(n=0), dict(dtype=2), dict(act=5), dict(act=-1)):
            assert call(L, **kw) == INVALID
        for kw in (dict(rows=1 << 31), dict(k=(1 << 20) + 1), dict(n=(1 << 20) + 1)):
            assert call(L, **kw) == UNSUPPORTED


def test_forward_pointers(L):
    for name in ("x", "w", "out"):
        assert forward(L, **{name: None}) == INVALID
    for i, name in enumerate(("x", "w", "bias", "residual", "pre", "out")):
        assert forward(L, **{name: at(i, 8)}) == INVALID          # not on a boundary of 16 bytes
    for i in (0, 1, 2, 3, 4):
        assert forward(L, out=at(i, 16)) == INVALID               # out over another
    for i in (0, 1, 2, 3):
        assert forward(L, pre=at(i)) == INVALID
    assert forward(L, pre=at(3), residual=at(3)) == INVALID       # pre may not be residual
    assert forward(L, out=at(3), residual=at(3), pre=at(3)) == INVALID


def test_backward_pointers(L):
    for name in ("x", "w", "dout", "pre"):
        assert backward(L, **{name: None}) == INVALID
    for i, name in enumerate(("x", "w", "dout", "pre", "dx", "dw", "dbias")):
        assert backward(L, **{name: at(i, 4)}) == INVALID
    for name in ("dx", "dw", "dbias"):
        for i in range(4):
            assert backward(L, **{name: at(i)}) == INVALID
    assert backward(L, dw=at(4)) == INVALID
    assert backward(L, dbias=at(5)) == INVALID
    assert backward(L, dx=None, dw=None, dbias=None) == OK         # nothing wanted


def test_workspace(L):
    n = ctypes.c_size_t(7)
    assert L.mhla_linear_act_workspace_size(0, 64, 96, 0, ctypes.byref(n)) == OK and n.value == 0
    assert L.mhla_linear_act_workspace_size(8, 64, 96, 1, ctypes.byref(n)) == OK and n.value == 0
    assert L.mhla_linear_act_workspace_size(300, 64, 96, 1, ctypes.byref(n)) == OK and n.value > 0 and n.value % 256 == 0
    need = n.value
    assert forward(L, dtype=1, ws=None, ws_bytes=16) == WORKSPACE
    assert forward(L, dtype=1, ws=at(9), ws_bytes=need - 1) == WORKSPACE
    assert forward(L, dtype=1, ws=at(9, 64), ws_bytes=need + 256) == WORKSPACE
    assert L.mhla_linear_act_backward_workspace_size(300, 64, 96, 0, 4, ctypes.byref(n)) == OK and n.value > 0
    assert backward(L, ws=at(9), ws_bytes=n.value - 1) == WORKSPACE
    assert L.mhla_linear_act_workspace_size(300, 64, 96, 0, None) == INVALID
    assert L.mhla_linear_act_workspace_size(300, 64, 96, 3, ctypes.byref(n)) == INVALID
    assert L.mhla_linear_act_backward_workspace_size(300, 64, 96, 0, 9, ctypes.byref(n)) == INVALID


def test_no_rows(L):
    assert forward(L, x=None, w=None, out=None, bias=None, residual=None, pre=None, rows=0) == OK
