"""The bounds that the delta rule's GPU tests use, on the CPU: the chunk form is the recurrence, factors that are really rounded stay
within them, and a term that is missing, turned round or rounded to too few bits does not."""

import numpy as np
import pytest

import oracle

from . import delta_bounds as db

GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dstate")
SHAPES = [(2, 64, 1, 2, 64), (1, 200, 2, 1, 48), (1, 129, 1, 2, 100), (1, 97, 1, 1, 7)]


def draw(seed, B, N, Hk, times, d, state=True):
    r = np.random.default_rng(seed)
    H = Hk * times
    f = r.standard_normal
    x = {"q": f((B, N, Hk, d)), "k": f((B, N, Hk, d)), "v": f((B, N, H, d)), "dout": f((B, N, H, d)),
         "g": -np.log1p(np.exp(-(f((B, N, H)) + 3))), "beta": 1 / (1 + np.exp(-f((B, N, H)))),
         "state": f((B, H, d, d)) if state else None, "dstate_out": f((B, H, d, d)) if state else None}
    x["k"] /= np.linalg.norm(x["k"], axis=-1, keepdims=True)
    return x


def args(x):
    return [x[n] for n in ("q", "k", "v", "g", "beta")]


def failing(x, dtype, scale, got):
    """Names of the gradients that the bounds refuse."""
    names = []
    for name, y, z in zip(GRADS, db.chunk_form(x, dtype, scale, back=True), got):
        bound, axes = db.grad_bound(name, y, dtype)
        if not (db.over_axes(z - y.x, axes) <= bound).all():
            names.append(name)
    return names


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_the_chunk_form_is_the_recurrence(shape, dtype):
    x = draw(1, *shape)
    out, last = db.chunk_form(x, dtype, 0.3)
    o, end = oracle.delta(*args(x), 0.3, x["state"])
    assert np.allclose(out.x, o, rtol=0, atol=1e-11) and np.allclose(last.x, end, rtol=0, atol=1e-11)
    ref = oracle.delta_backward(*args(x), x["dout"], 0.3, x["state"], x["dstate_out"])
    for y, r in zip(db.chunk_form(x, dtype, 0.3, back=True), ref):
        assert np.abs(y.x - r).max() <= 1e-11 * np.abs(r).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("state", [True, False])
def test_rounded_factors_stay_within(shape, state, dtype):
    """Every factor off by a random share up to the whole of u; and no bound allows a tenth of what it bounds."""
    x = draw(2, *shape, state)
    exact = db.chunk_form(x, dtype, 0.3)
    out, last = db.chunk_form(x, dtype, 0.3, rng=np.random.default_rng(3))
    assert (db.over_axes(out.x - exact[0].x, -1) <= db.out_bound(exact[0], dtype)).all()
    assert (db.over_axes(last.x - exact[1].x, (-2, -1)) <= db.state_bound(exact[1])).all()
    assert (db.state_bound(exact[1]) <= 1e-4 * db.over_axes(exact[1].x, (-2, -1))).all()
    got = db.chunk_form(x, dtype, 0.3, back=True, rng=np.random.default_rng(4))
    assert failing(x, dtype, 0.3, [y.x for y in got]) == []
    for name, y in zip(GRADS, db.chunk_form(x, dtype, 0.3, back=True)):
        bound, axes = db.grad_bound(name, y, dtype)
        assert (bound <= 0.1 * db.over_axes(y.x, axes)).all(), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("term,seen", [("reads", "dq"), ("A K", "dq"), ("A^T Q", "dk"), ("L K", "dk"), ("L^T K", "dk"), ("recalls", "dk"),
                                       ("writes", "dk"), ("e^b K S", "dbeta"), ("rows", "dbeta"), ("pairs", "dg"), ("enters", "dg"),
                                       ("leaves", "dg"), ("through", "dg")])
def test_a_missing_term_of_a_gradient_is_seen(term, seen, dtype):
    x = draw(5, 1, 200, 1, 2, 64)
    got = db.chunk_form(x, dtype, 0.3, back=True, drop=(term,))
    assert failing(x, dtype, 0.3, [y.x for y in got]) == [seen]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zeros_and_turned_signs_are_seen(dtype):
    x = draw(6, 1, 150, 2, 1, 100)
    ref = [y.x for y in db.chunk_form(x, dtype, 0.3, back=True)]
    assert failing(x, dtype, 0.3, ref) == []
    assert failing(x, dtype, 0.3, [0 * r for r in ref]) == list(GRADS) == failing(x, dtype, 0.3, [-r for r in ref])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("term", ["recall", "scores", "write"])
def test_a_missing_term_of_the_forward_is_seen(term, dtype):
    x = draw(7, 1, 150, 2, 1, 64)
    out, last = db.chunk_form(x, dtype, 0.3)
    bad, end = db.chunk_form(x, dtype, 0.3, drop=(term,))
    first = db.CHUNK[dtype] if term == "write" else 1   # a chunk's own tokens read what it writes through their scores
    assert (db.over_axes(bad.x - out.x, -1) > db.out_bound(out, dtype))[:, first:].mean() > 0.9
    assert term == "scores" or (db.over_axes(end.x - last.x, (-2, -1)) > db.state_bound(last)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_state_of_too_few_bits_is_seen(dtype):
    """Two bf16 terms (2^-16) or one of fp16 (2^-11) on the way to the state."""
    x = draw(8, 1, 300, 2, 1, 64)
    _, last = db.chunk_form(x, dtype, 0.3)
    for u in (2.0 ** -16, 2.0 ** -11):
        _, bad = db.chunk_form(x, dtype, 0.3, rng=np.random.default_rng(9), u_state=u)
        assert (db.over_axes(bad.x - last.x, (-2, -1)) > db.state_bound(last)).all()
