"""Host-side checks of the gated recurrence and of the query/key norm: no GPU, no kernel is launched.

Every malformed request is rejected with its documented status before anything
is queued; empty calls and planning calls work without a GPU.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import token_level_head_block_gb300 as mhla

OK, INVALID, SHAPE, UNSUPPORTED, CUDA, TIMEOUT, WORKSPACE = range(7)
FAKE = 1 << 40          # never dereferenced
STEP = 1 << 30
B, N, H, D = 2, 300, 3, 64


@pytest.fixture(scope="module")
def L():
    return mhla.lib()


def t(i, shape=(B, N, H, D), dtype="bf16", strides=None, base=None):
    b, n, h, d = shape
    return mhla.tensor_desc(FAKE + i * STEP if base is None else base, dtype, shape,
                            strides or (n * h * d, h * d, d))


def gate(i, shape=(B, N, H), dtype="bf16"):
    b, n, h = shape
    return mhla.tensor_desc(FAKE + i * STEP, dtype, (b, n, h, 1), (n * h, h, 1))


def ref(*xs):
    return [ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in xs]


def forward(L, q=None, k=None, v=None, g=None, scale=1.0, s_in=None, out=None, s_out=None, ws=None, n=0):
    q, k, v, g, out = q or t(0), k or t(1), v or t(2), g or gate(3), out or t(4)
    return L.mhla_gated_forward(*ref(q, k, v, g, scale, s_in, out, s_out, ws, n, None))


def test_forward_refusals(L):
    assert forward(L, k=t(1, (B, N, H, 32))) == SHAPE
    assert forward(L, v=t(2, (B, N - 1, H, D))) == SHAPE
    assert forward(L, k=t(1, dtype="f32")) == SHAPE
    assert forward(L, g=gate(3, (B, N, H + 1))) == SHAPE
    assert forward(L, g=gate(3, dtype="f32")) == SHAPE
    assert forward(L, g=t(3)) == SHAPE                                    # a gate of d values
    assert forward(L, out=t(4, (B, N, H, 32))) == SHAPE
    for bad in (float("nan"), float("inf")):
        assert forward(L, scale=bad) == INVALID
    assert forward(L, out=t(0)) == INVALID                                # out is q
    assert forward(L, out=t(4, base=FAKE + 3 * STEP)) == INVALID          # out over the gates
    assert forward(L, out=t(4, strides=(N * H * D, H * D, 32))) == INVALID   # heads of out overlap
    assert forward(L, s_out=FAKE + 4 * STEP + 64) == INVALID              # the state inside out
    assert forward(L, s_out=FAKE) == INVALID                              # the state inside q
    assert forward(L, s_in=FAKE + 8 * STEP, s_out=FAKE + 8 * STEP + 64) == INVALID   # states overlap, not equal
    assert forward(L, s_in=FAKE + 8 * STEP + 2) == INVALID                # misaligned float32
    big = (B, N, H, 129)
    assert forward(L, *(t(i, big) for i in range(3)), out=t(4, big)) == INVALID
    assert forward(L, t(0, (B, 0, H, D)), t(1, (B, 0, H, D)), t(2, (B, 0, H, D)), gate(3, (B, 0, H)),
                   out=t(4, (B, 0, H, D))) == INVALID                     # no tokens
    assert forward(L, q=t(0, base=0)) == INVALID
    assert L.mhla_gated_forward(None, None, None, None, 1.0, None, None, None, None, 0, None) == INVALID


def test_workspace_refusals(L):
    n = ctypes.c_size_t()
    shape = (1, 65536, 2, 64)
    q, k, v, out, g = t(0, shape), t(1, shape), t(2, shape), t(4, shape), gate(3, shape[:3])
    assert L.mhla_gated_workspace_size(*ref(q), ctypes.byref(n)) == OK and n.value % 256 == 0
    need = n.value
    assert forward(L, q, k, v, g, out=out, ws=None, n=16) == WORKSPACE
    assert forward(L, q, k, v, g, out=out, ws=FAKE + 9 * STEP + 8, n=need + 256) == WORKSPACE
    if need:
        assert forward(L, q, k, v, g, out=out, ws=FAKE + 9 * STEP, n=need - 1) == WORKSPACE
    assert L.mhla_gated_backward_workspace_size(*ref(q), ctypes.byref(n)) == OK and n.value % 256 == 0
    assert L.mhla_gated_workspace_size(*ref(q), None) == INVALID
    assert L.mhla_gated_workspace_size(None, ctypes.byref(n)) == INVALID
    assert L.mhla_qk_norm_backward_workspace_size(*ref(q), ctypes.byref(n)) == OK and n.value % 256 == 0


def test_empty_calls(L):
    for shape in ((0, N, H, D), (B, N, 0, D)):
        z = [mhla.tensor_desc(0, "bf16", shape, (1, 1, 1)) for _ in range(9)]
        z[3] = mhla.tensor_desc(0, "bf16", shape[:3] + (1,), (1, 1, 1))
        z[8] = mhla.tensor_desc(0, "bf16", shape[:3] + (1,), (1, 1, 1))
        assert forward(L, *z[:4], out=z[4]) == OK
        assert backward(L, *z) == OK
        n = ctypes.c_size_t(7)
        assert L.mhla_gated_workspace_size(*ref(z[0]), ctypes.byref(n)) == OK and n.value == 0
    one = [mhla.tensor_desc(0, "bf16", (0, 1, H, D), (1, 1, 1)) for _ in range(4)]
    g = mhla.tensor_desc(0, "bf16", (0, 1, H, 1), (1, 1, 1))
    assert L.mhla_gated_step(*ref(*one[:3], g, 1.0, None, one[3], None)) == OK
    assert L.mhla_qk_norm(*ref(*one[:2]), None, None, 1e-6, None, *ref(*one[2:]), None) == OK


def backward(L, q, k, v, g, do, dq, dk, dv, dg, s_in=None, ds_out=None, ds_in=None):
    return L.mhla_gated_backward(*ref(q, k, v, g, do, 1.0, s_in, ds_out, dq, dk, dv, dg, ds_in, None, 0, None))


def test_backward_refusals(L):
    base = [t(0), t(1), t(2), gate(3), t(4), t(5), t(6), t(7), gate(8)]

    def call(i, x, **kw):
        a = list(base)
        a[i] = x
        return backward(L, *a, **kw)

    assert call(4, t(4, dtype="f32")) == SHAPE
    assert call(5, t(5, (B, N, H, 32))) == SHAPE
    assert call(8, gate(8, (B, N, 1))) == SHAPE
    for i in (5, 6, 7):
        assert call(i, t(4)) == INVALID                    # over dout
        assert call(i, t(0)) == INVALID                    # over q
        assert call(i, t(i, strides=(0, H * D, D))) == INVALID
    assert call(6, t(5)) == INVALID                        # dk is dq
    assert call(8, gate(3)) == INVALID                     # dg is g
    far = FAKE + 12 * STEP
    assert backward(L, *base, ds_out=far, ds_in=far) == INVALID
    assert backward(L, *base, s_in=far, ds_in=far + 64) == INVALID
    assert backward(L, *base, ds_in=FAKE + 5 * STEP) == INVALID
    assert backward(L, *base, ds_in=FAKE + 1 * STEP) == INVALID


def test_step_refusals(L):
    one = (B, 1, H, D)
    q, k, v, out, g, state = t(0, one), t(1, one), t(2, one), t(4, one), gate(3, (B, 1, H)), FAKE + 8 * STEP
    call = lambda *a: L.mhla_gated_step(*ref(*a, None))
    assert call(t(0), t(1), t(2), gate(3), 1.0, state, t(4)) == SHAPE      # more than one token
    assert call(q, k, v, g, 1.0, None, out) == INVALID
    assert call(q, k, v, g, 1.0, FAKE, out) == INVALID                     # the state over q
    assert call(q, k, v, g, 1.0, FAKE + 4 * STEP, out) == INVALID          # the state over out
    assert call(q, k, v, g, 1.0, state, q) == INVALID
    assert call(q, k, v, g, float("inf"), state, out) == INVALID


def rot(rows=N, pairs=32, layout=0, table=FAKE + 20 * STEP, positions=None):
    return mhla.Rotation(table, positions, rows, pairs, layout)


def norm(L, q=None, k=None, eps=1e-6, r=None, qo=None, ko=None, wq=None, wk=None):
    hk = (B, N, 1, D)
    return L.mhla_qk_norm(*ref(q or t(0), k or t(1, hk)), wq, wk, eps, *ref(r or rot()), *ref(qo or t(2), ko or t(3, hk)),
                          None)


def test_qk_norm_refusals(L):
    assert norm(L, k=t(1, (B, N + 1, 1, D))) == SHAPE
    assert norm(L, k=t(1, (B, N, 1, 32))) == SHAPE
    assert norm(L, k=t(1, (B, N, 1, D), "f32")) == SHAPE
    assert norm(L, qo=t(2, (B, N, 1, D))) == SHAPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(L, eps=eps) == INVALID
    assert norm(L, r=rot(pairs=33)) == SHAPE               # more channels than the head has
    assert norm(L, r=rot(rows=N - 1)) == SHAPE             # token n without a row
    assert norm(L, r=rot(pairs=-1)) == INVALID
    assert norm(L, r=rot(layout=2)) == INVALID
    assert norm(L, r=rot(table=FAKE + 4)) == INVALID       # cos, sin read together
    assert norm(L, r=rot(positions=FAKE + 2)) == INVALID
    assert norm(L, qo=t(1)) == INVALID                     # over k
    assert norm(L, qo=t(0, base=FAKE + 2 * D)) == INVALID  # q, shifted by a head
    assert norm(L, qo=t(3)) == INVALID                     # over k_out
    assert norm(L, ko=t(0, (B, N, 1, D))) == INVALID       # over q
    assert norm(L, qo=t(20)) == INVALID                    # over the table
    assert norm(L, wq=FAKE + 2 * STEP) == INVALID          # the weight inside q_out
    hk = (B, N, 1, D)
    back = lambda **kw: L.mhla_qk_norm_backward(
        *ref(t(0), t(1, hk)), None, None, 1e-6, *ref(rot()), *ref(t(2), t(3, hk), kw.get("dq") or t(4), t(5, hk)),
        kw.get("wq"), kw.get("wk"), kw.get("ws"), kw.get("n", 0), None)
    assert back(dq=t(0)) == INVALID                        # dq over q
    assert back(dq=t(3)) == INVALID                        # dq over dk_out
    assert back(dq=t(4, (B, N, 2, D))) == SHAPE
    assert back(wq=FAKE + 6 * STEP, wk=FAKE + 6 * STEP) == INVALID
    assert back(wq=FAKE) == INVALID
    assert back(n=8) == WORKSPACE
    assert back(ws=FAKE + 9 * STEP, n=8) == WORKSPACE


def test_elements_at_odd_addresses_are_refused(L):
    odd = lambda i, *a: t(i, *a, base=FAKE + i * STEP + 1)
    hk = (B, N, 1, D)
    for i, name in enumerate(("q", "k", "v")):
        assert forward(L, **{name: odd(i)}) == INVALID
    assert forward(L, out=odd(4)) == INVALID
    g = gate(3)
    g.data = FAKE + 3 * STEP + 1
    assert forward(L, g=g) == INVALID
    assert norm(L, q=odd(0)) == INVALID and norm(L, k=odd(1, hk)) == INVALID and norm(L, qo=odd(2)) == INVALID
    f32 = t(0, dtype="f32", base=FAKE + 2)
    assert forward(L, f32, *(t(i, dtype="f32") for i in (1, 2)), g=gate(3, dtype="f32"), out=t(4, dtype="f32")) == INVALID


def test_weight_gradients_over_the_rotation_are_refused(L):
    hk = (B, N, 1, D)
    back = lambda r, wq: L.mhla_qk_norm_backward(*ref(t(0), t(1, hk)), None, None, 1e-6, *ref(r),
                                                 *ref(t(2), t(3, hk), t(4), t(5, hk)), wq, None, None, 8, None)
    table, positions = FAKE + 20 * STEP, FAKE + 30 * STEP
    r = rot(positions=positions)
    assert back(r, FAKE + 40 * STEP) == WORKSPACE           # all but the workspace given here is in order
    assert back(r, table + N * 32 * 8 - 4) == INVALID
    assert back(r, table - 4 * D + 4) == INVALID
    assert back(r, positions + 4 * B * N - 4) == INVALID


def test_views_of_one_projection_pass_the_overlap_checks(L):
    """Interleaved views share no element: only the workspace given here is refused."""
    st = (N * 4 * H * D, 4 * H * D, D)
    q, k, v, o = (t(0, strides=st, base=FAKE + 2 * i * H * D) for i in range(4))
    assert forward(L, q, k, v, out=o, ws=None, n=16) == WORKSPACE
    st = (N * 4 * H * D, 4 * H * D, 4 * D)                 # interleaved head by head
    q, k, v, o = (t(0, strides=st, base=FAKE + 2 * i * D) for i in range(4))
    assert forward(L, q, k, v, out=o, ws=None, n=16) == WORKSPACE
    o = t(0, strides=st, base=FAKE + 2 * (2 * D + 1))      # one element into v's neighbour
    assert forward(L, q, k, v, out=o, ws=None, n=16) == INVALID
    st = (N * 2 * H * D, 2 * H * D, D)                     # rows of two, the third runs into the next token
    q, k, o = (t(0, strides=st, base=FAKE + 2 * i * H * D) for i in range(3))
    assert forward(L, q, k, k, out=o, ws=None, n=16) == INVALID


def test_init_rotation(L):
    for grid, pairs in (((1, 50), (0, 7)), ((4, 6), (3, 2)), ((2, 3, 4), (1, 2, 0))):
        got = mhla.init_rotation(grid, pairs, 500.0)
        assert got.shape == (int(np.prod(grid)), sum(pairs), 2)
        # both sides round a double once; libm's cos and sin may differ in the last bit of the double
        assert np.abs(got - oracle.rotation_table(grid, pairs, 500.0)).max() <= 2.0 ** -24
    assert mhla.init_rotation((1, 5), (0, 0)).shape == (5, 0, 2)
    buf = (ctypes.c_float * 64)()
    call = lambda grid, pairs, base, cap, p=buf: L.mhla_init_rotation(
        ctypes.byref(mhla.shape3(grid)), (ctypes.c_int32 * 3)(*pairs), base, p, cap)
    assert call((4, 4), (1, 1), 10.0, 64) == OK
    assert call((4, 4), (1, 1), 10.0, 63) == INVALID
    assert call((4, 4), (1, -1), 10.0, 64) == INVALID
    assert call((4, 4), (1, 1), 0.0, 64) == INVALID
    assert call((4, 4), (1, 1), float("nan"), 64) == INVALID
    assert call((4, 0), (1, 1), 10.0, 64) == SHAPE
    assert call((1 << 40, 1 << 40), (1, 1), 10.0, 64) == INVALID
    assert call((4, 4), (1, 1), 10.0, 64, None) == INVALID


def test_binding_refusals():
    q = torch.zeros(1, 4, 2, 8)
    g = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError):
        mhla.gated_forward(q, q, q, g)                                   # not on a GPU
    with pytest.raises(ValueError):
        mhla.gated_forward(q.half(), q, q, g)
    with pytest.raises(ValueError):
        mhla.gated_forward(q, q, q, g, state=torch.zeros(1, 2, 8, 7))
    with pytest.raises(ValueError):
        mhla.gated_forward(q, q, q, g, state=torch.zeros(1, 2, 8, 8, dtype=torch.float64))
    with pytest.raises(ValueError):
        mhla.gated_step(q[:, :1], q[:, :1], q[:, :1], g[:, :1], torch.zeros(2, 1, 8, 8).transpose(0, 1)[:, :1])
    with pytest.raises(ValueError):
        mhla.gated_forward(q.transpose(2, 3), q, q, g)                   # channels not contiguous
    with pytest.raises(ValueError):
        mhla.qk_norm(q, q, q_weight=torch.ones(7))
    with pytest.raises(ValueError):
        mhla.qk_norm(q, q, table=torch.zeros(4, 4))
    with pytest.raises(ValueError):
        mhla.qk_norm(q, q, table=torch.zeros(4, 4, 2), positions=torch.zeros(1, 4, dtype=torch.int64))
    with pytest.raises(ValueError):
        mhla.qk_norm(q, q, table=torch.zeros(4, 4, 2), layout="pairs")
    with pytest.raises(ValueError):
        mhla.init_rotation((1, 4), (1,))
