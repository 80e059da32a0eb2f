"""Pins of the gated-recurrence and query/key-norm oracle against closed forms, none comparing it with itself."""

import numpy as np
import pytest

import oracle


def draw(seed, B=2, N=9, H=2, d=3):
    r = np.random.default_rng(seed)
    q, k, v, do = (r.standard_normal((B, N, H, d)) for _ in range(4))
    return q, k, v, -np.abs(r.standard_normal((B, N, H))), do, r.standard_normal((B, H, d, d)), \
        r.standard_normal((B, H, d, d))


def test_no_decay_is_running_sum_of_outer_products():
    q, k, v, g, *_ = draw(1)
    o, S = oracle.gated(q, k, v, 0 * g)
    kv = np.cumsum(np.einsum("bnhr,bnhc->bnhrc", k, v), axis=1)
    assert np.allclose(o, np.einsum("bnhr,bnhrc->bnhc", q, kv), rtol=0, atol=1e-12)
    assert np.allclose(S, kv[:, -1], rtol=0, atol=1e-12)


def test_recurrence_is_the_dense_form():
    q, k, v, g, *_ = draw(2)
    assert np.allclose(oracle.gated(q, k, v, g, 0.3)[0], oracle.gated_dense(q, k, v, g, 0.3), rtol=0, atol=1e-12)


def test_one_token_from_a_state_by_hand():
    q, k, v = (np.array(x, dtype=float).reshape(1, 1, 1, 2) for x in ([1, 2], [3, 5], [7, 11]))
    S = np.array([[1.0, 2.0], [4.0, 8.0]]).reshape(1, 1, 2, 2)
    o, last = oracle.gated(q, k, v, np.log(np.full((1, 1, 1), 0.5)), 2.0, S)
    want = np.array([[0.5 + 21, 1 + 33], [2 + 35, 4 + 55]])
    assert np.allclose(last[0, 0], want) and np.allclose(o[0, 0, 0], 2 * (want[0] + 2 * want[1]))


def test_a_closed_gate_starts_afresh():
    q, k, v, g, _, S, _ = draw(3)
    g[:, 4] = -np.inf
    o, last = oracle.gated(q, k, v, g, 1.0, S)
    fresh, end = oracle.gated(q[:, 4:], k[:, 4:], v[:, 4:], np.where(np.isinf(g[:, 4:]), 0, g[:, 4:]))
    assert np.allclose(o[:, 4:], fresh) and np.allclose(last, end)


def test_cutting_a_sequence_changes_nothing():
    q, k, v, g, _, S, _ = draw(4)
    o, last = oracle.gated(q, k, v, g, 0.7, S)
    a, mid = oracle.gated(q[:, :5], k[:, :5], v[:, :5], g[:, :5], 0.7, S)
    b, end = oracle.gated(q[:, 5:], k[:, 5:], v[:, 5:], g[:, 5:], 0.7, mid)
    assert np.allclose(o, np.concatenate((a, b), 1)) and np.allclose(last, end)


@pytest.mark.parametrize("which", ["q", "k", "v", "g", "state"])
def test_gradients_by_central_differences(which):
    q, k, v, g, do, S, dS = draw(5, B=1, N=5, H=1, d=2)
    x = {"q": q, "k": k, "v": v, "g": g, "state": S}

    def loss():
        o, last = oracle.gated(q, k, v, g, 0.6, S)
        return (o * do).sum() + (last * dS).sum()

    got = dict(zip(("q", "k", "v", "g", "state"), oracle.gated_backward(q, k, v, g, do, 0.6, S, dS)))[which]
    a = x[which]
    for i in np.ndindex(a.shape):
        keep, h = a[i], 1e-5
        a[i] = keep + h
        up = loss()
        a[i] = keep - h
        down = loss()
        a[i] = keep
        assert abs((up - down) / (2 * h) - got[i]) < 1e-7


def test_norm_of_a_known_row_and_its_rotation():
    x = np.array([3.0, 4.0]).reshape(1, 1, 1, 2)          # mean square 12.5
    y = oracle.qk_norm(x, np.array([2.0, 1.0]), eps=3.5)   # / 4
    assert np.allclose(y[0, 0, 0], [1.5, 1.0])
    quarter = np.array([[[0.0, 1.0]]])                     # 90 degrees: (a, b) -> (-b, a)
    z = oracle.qk_norm(x, None, eps=3.5, table=quarter)
    assert np.allclose(z[0, 0, 0], [-1.0, 0.75])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_keeps_lengths_and_sees_only_distances(layout):
    r = np.random.default_rng(6)
    x, y = r.standard_normal((2, 1, 1, 1, 8))
    table = oracle.rotation_table((1, 40), (0, 3))
    at = lambda v, n: oracle.qk_norm(v, None, 0.0, table, np.array([[n]]), layout)[0, 0, 0]
    assert np.allclose(np.linalg.norm(at(x, 0)), np.linalg.norm(at(x, 17)))
    assert np.allclose(at(x, 9) @ at(y, 4), at(x, 30) @ at(y, 25))
    assert np.allclose(at(x, 9)[6:], at(x, 0)[6:])         # channels behind the pairs stay


def test_rotation_table_axes_by_hand():
    t = oracle.rotation_table((2, 3), (1, 2), base=100.0)
    assert t.shape == (6, 3, 2)
    assert np.allclose(t[5, :, 0], np.cos([1.0, 2.0, 0.2])) and np.allclose(t[5, :, 1], np.sin([1.0, 2.0, 0.2]))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_gradients_by_central_differences(layout):
    r = np.random.default_rng(7)
    x, dz = r.standard_normal((2, 1, 3, 2, 6))
    w, table = r.standard_normal(6), oracle.rotation_table((1, 9), (0, 2))
    pos = np.array([[4, -1, 8]])
    loss = lambda: (dz * oracle.qk_norm(x, w, 0.1, table, pos, layout)).sum()
    dx, dw = oracle.qk_norm_backward(x, dz, w, 0.1, table, pos, layout)
    for a, got in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            keep, h = a[i], 1e-5
            a[i] = keep + h
            up = loss()
            a[i] = keep - h
            down = loss()
            a[i] = keep
            assert abs((up - down) / (2 * h) - got[i]) < 1e-7
