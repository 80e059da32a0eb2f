"""Host-side checks of the gated delta rule: no GPU, no kernel is launched."""

import ctypes

import pytest

import token_level_head_block_gb300 as mhla

OK, INVALID, SHAPE, UNSUPPORTED, CUDA, TIMEOUT, WORKSPACE = range(7)
FAKE = 1 << 40          # never dereferenced
STEP = 1 << 30
B, N, HK, H, D = 2, 300, 2, 4, 64


@pytest.fixture(scope="module")
def L():
    return mhla.lib()


def t(i, heads=H, shape=(B, N, D), dtype="bf16", strides=None, base=None):
    b, n, d = shape
    return mhla.tensor_desc(FAKE + i * STEP if base is None else base, dtype, (b, n, heads, d), strides or (n * heads * d, heads * d, d))


def gate(i, heads=H, shape=(B, N), dtype="bf16"):
    return t(i, heads, shape + (1,), dtype)


def ref(*xs):
    return [ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in xs]


def forward(L, s_in=None, s_out=None, ws=None, n=0, scale=1.0, **kw):
    x = dict(q=t(0, HK), k=t(1, HK), v=t(2), g=gate(3), beta=gate(4), out=t(5))
    x.update(kw)
    return L.mhla_delta_forward(*ref(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, s_in, x["out"], s_out, ws, n, None))


def test_forward_refusals(L):
    assert forward(L, k=t(1, H)) == SHAPE                                 # q and k differ
    assert forward(L, q=t(0, 3), k=t(1, 3)) == SHAPE                      # 4 heads on 3
    assert forward(L, q=t(0, 8), k=t(1, 8)) == SHAPE                      # fewer values than keys
    assert forward(L, v=t(2, shape=(B, N - 1, D))) == SHAPE
    assert forward(L, v=t(2, dtype="f32")) == SHAPE
    assert forward(L, g=gate(3, HK)) == SHAPE
    assert forward(L, beta=gate(4, HK)) == SHAPE
    assert forward(L, beta=gate(4, dtype="f32")) == SHAPE
    assert forward(L, beta=t(4)) == SHAPE
    assert forward(L, out=t(5, HK)) == SHAPE
    for bad in (float("nan"), float("inf")):
        assert forward(L, scale=bad) == INVALID
    for i in range(5):
        assert forward(L, out=t(i)) == INVALID                            # out over an input
    assert forward(L, out=t(5, strides=(N * H * D, H * D, 32))) == INVALID
    assert forward(L, s_out=FAKE + 5 * STEP + 64) == INVALID
    assert forward(L, s_out=FAKE + 4 * STEP) == INVALID
    assert forward(L, s_in=FAKE + 8 * STEP, s_out=FAKE + 8 * STEP + 64) == INVALID
    assert forward(L, s_in=FAKE + 8 * STEP + 2) == INVALID
    assert forward(L, v=t(2, base=FAKE + 2 * STEP + 1)) == INVALID        # half an element
    assert forward(L, q=t(0, HK, base=0)) == INVALID
    big = (B, N, 129)
    assert forward(L, q=t(0, HK, big), k=t(1, HK, big), v=t(2, shape=big), out=t(5, shape=big)) == INVALID
    assert L.mhla_delta_forward(*([None] * 5), 1.0, None, None, None, None, 0, None) == INVALID


def test_too_many_chunks(L):
    many = (1 << 12, 1 << 25)
    kw = {n: t(i, h, many + (D,), strides=(0, 0, 0)) for i, (n, h) in enumerate((("q", HK), ("k", HK), ("v", H)))}
    g = {n: t(i, H, many + (1,), strides=(0, 0, 0)) for i, n in ((3, "g"), (4, "beta"))}
    assert forward(L, **kw, **g) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert L.mhla_delta_workspace_size(*ref(kw["q"], kw["v"]), ctypes.byref(n)) == UNSUPPORTED


def test_workspace(L):
    n = ctypes.c_size_t()
    q, v = t(0, HK), t(2)
    assert L.mhla_delta_workspace_size(*ref(q, v), ctypes.byref(n)) == OK and n.value > 0 and n.value % 256 == 0
    need = n.value
    assert forward(L, ws=None, n=16) == WORKSPACE
    assert forward(L, ws=FAKE + 9 * STEP + 8, n=need + 256) == WORKSPACE
    assert forward(L, ws=FAKE + 9 * STEP, n=need - 1) == WORKSPACE
    assert L.mhla_delta_backward_workspace_size(*ref(q, v), ctypes.byref(n)) == OK and n.value > need
    assert L.mhla_delta_workspace_size(*ref(q, v), None) == INVALID
    assert L.mhla_delta_workspace_size(*ref(q), None, ctypes.byref(n)) == INVALID
    assert L.mhla_delta_workspace_size(*ref(t(0, 3), v), ctypes.byref(n)) == SHAPE


def backward(L, s_in=None, ds_out=None, ds_in=None, **kw):
    x = dict(q=t(0, HK), k=t(1, HK), v=t(2), g=gate(3), beta=gate(4), dout=t(5), dq=t(6, HK), dk=t(7, HK), dv=t(8), dg=gate(9),
             dbeta=gate(10))
    x.update(kw)
    return L.mhla_delta_backward(*ref(*list(x.values())[:6], 1.0, s_in, ds_out, *list(x.values())[6:], ds_in, None, 0, None))


def test_backward_refusals(L):
    assert backward(L, dout=t(5, HK)) == SHAPE
    assert backward(L, dq=t(6, H)) == SHAPE
    assert backward(L, dk=t(7, H)) == SHAPE
    assert backward(L, dv=t(8, HK)) == SHAPE
    assert backward(L, dg=gate(9, HK)) == SHAPE
    assert backward(L, dbeta=gate(10, dtype="f32")) == SHAPE
    for name in ("dq", "dk"):
        for i in range(6):
            assert backward(L, **{name: t(i, HK)}) == INVALID
    assert backward(L, dk=t(6, HK)) == INVALID                            # over dq
    assert backward(L, dv=t(5)) == INVALID                                # over dout
    assert backward(L, dbeta=gate(9)) == INVALID                          # over dg
    assert backward(L, ds_in=FAKE + 8 * STEP) == INVALID                  # inside dv
    assert backward(L, s_in=FAKE + 12 * STEP, ds_in=FAKE + 12 * STEP) == INVALID


def test_step_refusals(L):
    one = (B, 1, D)
    x = [t(0, HK, one), t(1, HK, one), t(2, shape=one), gate(3, shape=(B, 1)), gate(4, shape=(B, 1))]
    step = lambda a, state, out: L.mhla_delta_step(*ref(*a, 1.0, state, out, None))
    assert step(x, None, t(5, shape=one)) == INVALID
    assert step(x, FAKE + 7 * STEP + 1, t(5, shape=one)) == INVALID
    assert step(x, FAKE + 5 * STEP, t(5, shape=one)) == INVALID           # the state inside out
    assert step(x, FAKE, t(5, shape=one)) == INVALID                      # inside q
    assert step(x, FAKE + 7 * STEP, t(5, HK, one)) == SHAPE
    two = [t(0, HK, (B, 2, D)), t(1, HK, (B, 2, D)), t(2, shape=(B, 2, D)), gate(3, shape=(B, 2)), gate(4, shape=(B, 2))]
    assert step(two, FAKE + 7 * STEP, t(5, shape=(B, 2, D))) == SHAPE


def test_empty_calls(L):
    z = lambda heads, d=D, b=0: mhla.tensor_desc(0, "bf16", (b, 5, heads, d), (1, 1, 1))
    kw = dict(q=z(HK), k=z(HK), v=z(H), g=z(H, 1), beta=z(H, 1), out=z(H))
    assert forward(L, **kw) == OK
    none = dict(q=z(0, b=2), k=z(0, b=2), v=z(0, b=2), g=z(0, 1, 2), beta=z(0, 1, 2), out=z(0, b=2))
    assert forward(L, **none) == OK
    assert forward(L, **{**none, "v": t(2, shape=(2, 5, D))}) == SHAPE      # values without keys
    del kw["out"]
    assert backward(L, **kw, dout=z(H), dq=z(HK), dk=z(HK), dv=z(H), dg=z(H, 1), dbeta=z(H, 1)) == OK
    n = ctypes.c_size_t(7)
    assert L.mhla_delta_workspace_size(*ref(z(HK), z(H)), ctypes.byref(n)) == OK and n.value == 0
