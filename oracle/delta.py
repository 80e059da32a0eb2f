"""Plain float64 CPU oracle of the gated delta rule and of the linear layer with activation and residual.

TEST INFRASTRUCTURE ONLY, like ``mhla_oracle``.  Written from the definitions:

    S'_t = exp(g_t) S_{t-1},  w_t = beta_t (v_t - S'_t^T k_t),  S_t = S'_t + k_t w_t^T,  o_t = scale * S_t^T q_t

``delta`` and ``delta_backward`` walk the tokens; ``delta_dense`` forms the product
of all tokens' transitions.  q and k have Hk heads, v, g and beta H; head h
reads key head h // (H / Hk).
"""

from __future__ import annotations

import math

import numpy as np

from .gated import LOWEST_GATE


def _heads(x, H):
    return np.repeat(x, H // x.shape[2], axis=2)


def delta(q, k, v, g, beta, scale=1.0, state=None, steps=False):
    """(o [B, N, H, d], last state [B, H, d, d]) of float64 arrays; steps: also every S_t
    [N, B, H, d, d] and w_t [B, N, H, d]."""
    B, N, H, d = v.shape
    q, k = _heads(q, H), _heads(k, H)
    S = np.zeros((B, H, d, d)) if state is None else np.array(state, dtype=np.float64)
    o, w, all_S = np.empty((B, N, H, d)), np.empty((B, N, H, d)), []
    a = np.exp(np.maximum(g, LOWEST_GATE))
    for t in range(N):
        S = a[:, t, :, None, None] * S
        w[:, t] = beta[:, t, :, None] * (v[:, t] - np.einsum("bhrc,bhr->bhc", S, k[:, t]))
        S = S + k[:, t, :, :, None] * w[:, t, :, None, :]
        o[:, t] = scale * np.einsum("bhr,bhrc->bhc", q[:, t], S)
        if steps:
            all_S.append(S)
    return (o, S, np.array(all_S), w) if steps else (o, S)


def delta_dense(q, k, v, g, beta, scale=1.0):
    """The explicit form from an empty state: S_t = sum_s (prod of u from t down to s + 1 of
    exp(g_u) (1 - beta_u k_u k_u^T)) beta_s k_s v_s^T."""
    B, N, H, d = v.shape
    q, k = _heads(q, H), _heads(k, H)
    o = np.zeros((B, N, H, d))
    for b in range(B):
        for h in range(H):
            for t in range(N):
                A, S = np.eye(d), np.zeros((d, d))
                for s in range(t, -1, -1):
                    S = S + A @ (beta[b, s, h] * np.outer(k[b, s, h], v[b, s, h]))
                    A = A @ (math.exp(g[b, s, h]) * (np.eye(d) - beta[b, s, h] * np.outer(k[b, s, h], k[b, s, h])))
                o[b, t, h] = scale * S.T @ q[b, t, h]
    return o


def delta_backward(q, k, v, g, beta, dout, scale=1.0, state=None, dstate_out=None, steps=False):
    """(dq, dk, dv, dg, dbeta, dstate) of sum(dout * o) + sum(dstate_out * S_last); steps: also the
    largest norm of a dS_t."""
    B, N, H, d = v.shape
    Hk = q.shape[2]
    _, _, all_S, w = delta(q, k, v, g, beta, 1.0, state, steps=True)
    q, k = _heads(q, H), _heads(k, H)
    start = np.zeros((B, H, d, d)) if state is None else np.array(state, dtype=np.float64)
    a = np.exp(np.maximum(g, LOWEST_GATE))
    dS = np.zeros((B, H, d, d)) if dstate_out is None else np.array(dstate_out, dtype=np.float64)
    dq, dk, dv = (np.empty((B, N, H, d)) for _ in range(3))
    dg, dbeta = np.empty((B, N, H)), np.empty((B, N, H))
    largest = np.linalg.norm(dS)
    for t in range(N - 1, -1, -1):
        before = all_S[t - 1] if t else start
        M = a[:, t, :, None, None] * before
        dq[:, t] = scale * np.einsum("bhrc,bhc->bhr", all_S[t], dout[:, t])
        dS = dS + scale * q[:, t, :, :, None] * dout[:, t, :, None, :]
        largest = max(largest, np.linalg.norm(dS))
        dw = np.einsum("bhrc,bhr->bhc", dS, k[:, t])
        dv[:, t] = beta[:, t, :, None] * dw
        dbeta[:, t] = (dw * (v[:, t] - np.einsum("bhrc,bhr->bhc", M, k[:, t]))).sum(-1)
        dk[:, t] = np.einsum("bhrc,bhc->bhr", dS, w[:, t]) - np.einsum("bhrc,bhc->bhr", M, dv[:, t])
        dM = dS - k[:, t, :, :, None] * dv[:, t, :, None, :]
        dg[:, t] = (dM * M).sum((-2, -1))
        dS = a[:, t, :, None, None] * dM
    share = lambda x: x.reshape(B, N, Hk, H // Hk, d).sum(3)
    out = (share(dq), share(dk), dv, dg, dbeta, dS)
    return out + (largest,) if steps else out


def _erf(x):
    return np.vectorize(math.erf, otypes=[np.float64])(x)


def activation(z, kind):
    """act(z) and its slope."""
    if kind == "none":
        return z, np.ones_like(z)
    if kind == "relu":
        return np.where(z > 0, z, 0.0), (z > 0).astype(np.float64)
    if kind == "silu":
        p = 1 / (1 + np.exp(-z))
        return z * p, p + z * p * (1 - p)
    if kind == "gelu":
        p = (1 + _erf(z / math.sqrt(2))) / 2
        return z * p, p + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = np.tanh(a * (z + 0.044715 * z ** 3))
        return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) / 2 * a * (1 + 3 * 0.044715 * z * z)
    raise ValueError(f"unknown activation {kind!r}")


def linear_act(x, w, bias=None, kind="none", residual=None):
    """(act(x w^T + bias) + residual, x w^T + bias)."""
    z = x @ w.T + (0.0 if bias is None else bias)
    return activation(z, kind)[0] + (0.0 if residual is None else residual), z


def linear_act_backward(x, w, dout, kind="none", pre=None):
    """(dx, dw, dbias)."""
    dz = dout if kind == "none" else dout * activation(pre, kind)[1]
    return dz @ w, dz.T @ x, dz.sum(0)
