"""Plain float64 CPU oracle of gated causal linear attention and of the query/key norm with rotation.

TEST INFRASTRUCTURE ONLY, like ``mhla_oracle``.  Written from the definitions:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t

``gated`` and ``gated_backward`` walk the tokens; ``gated_dense`` is the explicit
N x N form.  ``qk_norm`` norms every head by its root mean square and turns
pairs of channels; ``qk_norm_backward`` is its chain rule.
"""

from __future__ import annotations

import numpy as np

LOWEST_GATE = -1000.0


def gated(q, k, v, g, scale=1.0, state=None):
    """(o [B, N, H, d], last state [B, H, d, d]) of float64 arrays [B, N, H, d], g [B, N, H]."""
    B, N, H, d = q.shape
    S = np.zeros((B, H, d, d)) if state is None else np.array(state, dtype=np.float64)
    o = np.empty((B, N, H, d))
    a = np.exp(np.maximum(g, LOWEST_GATE))
    for t in range(N):
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * np.einsum("bhr,bhrc->bhc", q[:, t], S)
    return o, S


def gated_dense(q, k, v, g, scale=1.0):
    """The N x N form from an empty state: A[t, s] = exp(sum of g over s < u <= t) (q_t . k_s), s <= t."""
    N = q.shape[1]
    c = np.cumsum(g, axis=1)
    A = np.einsum("bthr,bshr->bhts", q, k)
    for t in range(N):
        for s in range(N):
            A[:, :, t, s] *= np.exp(c[:, t] - c[:, s]) if s <= t else 0.0
    return scale * np.einsum("bhts,bshc->bthc", A, v)


def gated_backward(q, k, v, g, dout, scale=1.0, state=None, dstate_out=None):
    """(dq, dk, dv, dg, dstate) of sum(dout * o) + sum(dstate_out * S_last)."""
    B, N, H, d = q.shape
    S = np.zeros((N + 1, B, H, d, d))
    if state is not None:
        S[0] = state
    a = np.exp(np.maximum(g, LOWEST_GATE))
    for t in range(N):
        S[t + 1] = a[:, t, :, None, None] * S[t] + k[:, t, :, :, None] * v[:, t, :, None, :]
    dS = np.zeros((B, H, d, d)) if dstate_out is None else np.array(dstate_out, dtype=np.float64)
    dq, dk, dv, dg = (np.empty_like(x) for x in (q, k, v, g))
    for t in range(N - 1, -1, -1):
        dq[:, t] = scale * np.einsum("bhrc,bhc->bhr", S[t + 1], dout[:, t])
        dS = dS + scale * q[:, t, :, :, None] * dout[:, t, :, None, :]
        dk[:, t] = np.einsum("bhrc,bhc->bhr", dS, v[:, t])
        dv[:, t] = np.einsum("bhrc,bhr->bhc", dS, k[:, t])
        dS = a[:, t, :, None, None] * dS
        dg[:, t] = (dS * S[t]).sum((-2, -1))
    return dq, dk, dv, dg, dS


def rotation_table(grid, pairs, base=10000.0):
    """cos and sin of every token's angles, float64 [N, sum(pairs), 2]."""
    rows = []
    for index in np.ndindex(*grid):
        angles = [x * base ** (-i / p) for x, p in zip(index, pairs) for i in range(p)]
        rows.append([(np.cos(a), np.sin(a)) for a in angles])
    return np.array(rows, dtype=np.float64).reshape(int(np.prod(grid)), sum(pairs), 2)


def _channels(pairs, layout):
    i = np.arange(pairs)
    return (i, i + pairs) if layout == "half" else (2 * i, 2 * i + 1)


def _turn(x, table, positions, layout, sign):
    """x [B, N, H, d] with every pair turned by its token's row (negative position: left alone)."""
    if table is None or table.shape[1] == 0:
        return x
    x = x.copy()
    a, b = _channels(table.shape[1], layout)
    B, N = x.shape[:2]
    pos = np.broadcast_to(np.arange(N), (B, N)) if positions is None else positions
    for i in range(B):
        for n in range(N):
            if pos[i, n] < 0:
                continue
            if pos[i, n] >= table.shape[0]:
                x[i, n][:, np.concatenate((a, b))] = np.nan
                continue
            c, s = table[pos[i, n], :, 0], sign * table[pos[i, n], :, 1]
            lo, hi = x[i, n][:, a], x[i, n][:, b]
            x[i, n][:, a], x[i, n][:, b] = lo * c - hi * s, lo * s + hi * c
    return x


def qk_norm(x, weight=None, eps=1e-6, table=None, positions=None, layout="half"):
    """One of the two sides: x [B, N, H, d] normed per head and turned."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    return _turn(y, table, positions, layout, 1.0)


def qk_norm_backward(x, dz, weight=None, eps=1e-6, table=None, positions=None, layout="half"):
    """(dx, dweight) of sum(dz * qk_norm(x))."""
    dy = _turn(dz, table, positions, layout, -1.0)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r
    dweight = (dy * u).sum((0, 1, 2))
    m = dy if weight is None else dy * weight
    return r * (m - u * (m * u).mean(-1, keepdims=True)), dweight
