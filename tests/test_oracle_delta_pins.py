"""Pins of the delta-rule and linear-layer oracle against closed forms and differences, none comparing it with itself."""

import math

import numpy as np
import pytest

import oracle


def draw(seed, B=2, N=7, H=4, Hk=2, d=3):
    r = np.random.default_rng(seed)
    q, k = (r.standard_normal((B, N, Hk, d)) for _ in range(2))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    v, do = (r.standard_normal((B, N, H, d)) for _ in range(2))
    g, beta = -np.abs(r.standard_normal((B, N, H))), r.uniform(0, 1, (B, N, H))
    S, dS = (r.standard_normal((B, H, d, d)) for _ in range(2))
    return q, k, v, g, beta, do, S, dS


def test_recurrence_is_the_product_of_transitions():
    q, k, v, g, beta, *_ = draw(1)
    assert np.allclose(oracle.delta(q, k, v, g, beta, 0.3)[0], oracle.delta_dense(q, k, v, g, beta, 0.3), rtol=0, atol=1e-12)


def test_full_strength_stores_the_value_under_its_key():
    """beta = 1 and unit keys: reading the state with the key just written gives the value, whatever was there."""
    q, k, v, g, beta, _, S, _ = draw(2)
    o, _ = oracle.delta(k, k, v, g, np.ones_like(beta), 1.0, S)
    assert np.allclose(o, v, rtol=0, atol=1e-12)


def test_without_strength_the_state_only_fades():
    q, k, v, g, beta, _, S, _ = draw(3)
    _, last = oracle.delta(q, k, v, g, 0 * beta, 1.0, S)
    assert np.allclose(last, np.exp(g.sum(1))[..., None, None] * S)


def test_orthogonal_keys_are_the_gated_recurrence():
    """Keys orthogonal to one another and to the state's rows: nothing to correct."""
    q, _, v, g, beta, *_ = draw(4, N=3)
    k = np.broadcast_to(np.eye(3)[None, :, None, :], q.shape)
    o, S = oracle.delta(q, k, v, g, beta)
    rep = lambda x: np.repeat(x, 2, axis=2)
    want, last = oracle.gated(rep(q), rep(k) * beta[..., None], v, g)
    assert np.allclose(o, want) and np.allclose(S, last)


def test_cutting_a_sequence_changes_nothing():
    q, k, v, g, beta, _, S, _ = draw(5)
    x = (q, k, v, g, beta)
    o, last = oracle.delta(*x, 0.7, S)
    a, mid = oracle.delta(*(t[:, :4] for t in x), 0.7, S)
    b, end = oracle.delta(*(t[:, 4:] for t in x), 0.7, mid)
    assert np.allclose(o, np.concatenate((a, b), 1)) and np.allclose(last, end)


@pytest.mark.parametrize("which", ["q", "k", "v", "g", "beta", "state"])
def test_gradients_by_central_differences(which):
    q, k, v, g, beta, do, S, dS = draw(6, B=1, N=4, H=2, Hk=1, d=2)
    x = {"q": q, "k": k, "v": v, "g": g, "beta": beta, "state": S}

    def loss():
        o, last = oracle.delta(q, k, v, g, beta, 0.6, S)
        return (o * do).sum() + (last * dS).sum()

    got = dict(zip(("q", "k", "v", "g", "beta", "state"), oracle.delta_backward(q, k, v, g, beta, do, 0.6, S, dS)))[which]
    a = x[which]
    for i in np.ndindex(a.shape):
        keep, h = a[i], 1e-6
        a[i] = keep + h
        up = loss()
        a[i] = keep - h
        down = loss()
        a[i] = keep
        assert abs(got[i] - (up - down) / (2 * h)) < 1e-7


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_activations_and_their_slopes(kind):
    z = np.array([-3.0, -0.7, 0.4, 2.5])
    y, slope = oracle.activation(z, kind)
    h = 1e-6
    assert np.allclose(slope, (oracle.activation(z + h, kind)[0] - oracle.activation(z - h, kind)[0]) / (2 * h), atol=1e-8)
    if kind == "silu":
        assert math.isclose(y[3], 2.5 / (1 + math.exp(-2.5)))
    if kind == "gelu":
        assert math.isclose(y[2], 0.4 * 0.5 * math.erfc(-0.4 / math.sqrt(2)))
    if kind == "gelu_tanh":   # the approximation is within 5e-4 of the exact form
        assert np.abs(y - oracle.activation(z, "gelu")[0]).max() < 5e-4


def test_linear_layer_gradients_by_central_differences():
    r = np.random.default_rng(8)
    x, w, b, do = r.standard_normal((3, 4)), r.standard_normal((2, 4)), r.standard_normal(2), r.standard_normal((3, 2))
    dx, dw, db = oracle.linear_act_backward(x, w, do, "silu", oracle.linear_act(x, w, b)[1])
    for a, got in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(a.shape):
            keep, h = a[i], 1e-6
            a[i] = keep + h
            up = (oracle.linear_act(x, w, b, "silu")[0] * do).sum()
            a[i] = keep - h
            down = (oracle.linear_act(x, w, b, "silu")[0] * do).sum()
            a[i] = keep
            assert abs(got[i] - (up - down) / (2 * h)) < 1e-7
