"""How far the delta rule's results may be off, from the terms that are summed for them.

The chunk form is evaluated in float64 (C tokens a chunk, S the state that enters, D the gradient of the one that leaves):
  T = (1 + beta G)^-1, G = tril(K K^T . decay, -1);  W = T beta V - K^ S, K^ = T beta e^b K
  O = scale e^b Q S + P W, P = scale tril(Q K^T . decay);  S <- e^B S + (e^{B-b} K)^T W
  dW = P^T do + e^{B-b} K D;  dR = T^T dW;  D <- e^B D + (scale e^b Q)^T do - K^^T dW
  A = scale (do W^T) . decay, L = -beta (dR W^T) . decay (strict)
  dq = scale e^b do S^T + A K;  dk = A^T Q + L K + L^T K - beta e^b dR S^T + e^{B-b} W D^T;  dv = beta dR
  dbeta = dR . (V - e^b K S) - rows of (dR W^T . G);  dg: pairs of A (q k) + L (k k) around the gate, what reads S
  behind it, what writes D in front of it, e^B <S, D>
Every value carries an error: a factor that enters the tensor cores is off by a share u of itself, each by itself, so the error of a
product is the root of the summed squares of its terms' errors, and later steps pass it on.  u is 2^-22 (pairs of fp16) on the way to the
state and its gradient and throughout float32 calls, 2^-11 (one fp16) for what only feeds bf16 results; a block's scale ends
2^-39 below its largest value.  What the float32 sums, powers of two and decays add is 2^-22 of their terms at most, counted as another share of the products.  A bound is
MARGIN times that error and half a step of the result's type.
"""

import numpy as np

from oracle.gated import LOWEST_GATE

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
CHUNK = {"bf16": 64, "f32": 32}
FINE = 2.0 ** -22                                     # of what reaches the state
COARSE = {"bf16": 2.0 ** -11, "f32": 2.0 ** -22}      # of what only reaches results of the type
MARGIN = 4                                            # u is the largest rounding: 7 of its standard deviations


class Off:
    """An array and the error of each element."""

    def __init__(self, x, e=None):
        self.x = np.asarray(x, dtype=np.float64)
        self.e = np.zeros_like(self.x) if e is None else e

    @property
    def T(self):
        return Off(np.swapaxes(self.x, -1, -2), np.swapaxes(self.e, -1, -2))

    def __add__(self, o):
        return Off(self.x + o.x, np.hypot(self.e, o.e))

    def __neg__(self):
        return Off(-self.x, self.e)

    def __sub__(self, o):
        return self + -o

    def __mul__(self, f):                              # by what is known to float32's last bits
        if isinstance(f, Off):
            return Off(self.x * f.x, np.hypot(self.e * f.x, self.x * f.e))
        return Off(self.x * f, self.e * np.abs(f))

    def sum(self, axis):
        return Off(self.x.sum(axis), np.sqrt((self.e ** 2).sum(axis)))


class Rule:
    """The rounding of factors: shares only, or (rng) made as well."""

    def __init__(self, rng=None):
        self.rng = rng

    def rounded(self, a, u, least=0.0):
        a = a if isinstance(a, Off) else Off(a)
        off = np.maximum(u * np.abs(a.x), least)
        x = a.x if self.rng is None or u == 0 else a.x + off * self.rng.uniform(-1, 1, a.x.shape)
        return Off(x, np.hypot(a.e, off))

    def product(self, a, b, ua, ub, least_a=0.0, least_b=0.0):
        a, b = self.rounded(a, ua, least_a), self.rounded(b, ub, least_b)
        own = FINE ** 2 * (a.x ** 2 @ b.x ** 2)        # float32 sums
        return Off(a.x @ b.x, np.sqrt(a.e ** 2 @ b.x ** 2 + a.x ** 2 @ b.e ** 2 + own))


def least(y, rows, apart=False):
    """What a block's scale leaves of its smallest values: 2^-39 of the largest of `rows` rows (of each column, if apart)."""
    y = np.abs(y.x if isinstance(y, Off) else y)
    out = np.empty_like(y)
    for r in range(0, len(y), rows):
        out[r:r + rows] = y[r:r + rows].max(0, keepdims=True) if apart else y[r:r + rows].max()
    return 2.0 ** -39 * out


def heads(x, H):
    return np.repeat(x, H // x.shape[2], axis=2)


def chunk_form(x, dtype, scale, back=False, rng=None, drop=(), u_state=FINE):
    """Results of the float64 arrays x (q, k, v, g, beta, state; back: dout, dstate_out) as Off.  drop: terms left out, as a
    mistake would; u_state: the share on the way to the state."""
    q, k, v, g, beta = (x[n] for n in ("q", "k", "v", "g", "beta"))
    B, N, H, d = v.shape
    q, k, C, rule = heads(q, H), heads(k, H), CHUNK[dtype], Rule(rng)
    uc = COARSE[dtype]
    exact = 0.0 if dtype == "bf16" else FINE           # a bf16 input is one fp16 or one bf16 term
    out, last = Off(np.zeros_like(v)), Off(np.zeros((B, H, d, d)))
    names = ("dq", "dk", "dv", "dg", "dbeta")
    grads = {n: Off(np.zeros((B, N, H) + ((d,) if n in ("dq", "dk", "dv") else ()))) for n in names}
    first = Off(np.zeros((B, H, d, d)))
    for b in range(B):
        for h in range(H):
            S = Off(np.zeros((d, d)) if x["state"] is None else x["state"][b, h])
            kept = []
            for t0 in range(0, N, C):
                at = slice(t0, min(t0 + C, N))
                Q, K, V = q[b, at, h], k[b, at, h], v[b, at, h]
                be = beta[b, at, h][:, None]
                run = np.cumsum(np.maximum(g[b, at, h], LOWEST_GATE))
                n = len(run)
                low = np.tril(np.ones((n, n)))
                decay = np.where(low > 0, np.exp(np.minimum(run[:, None] - run[None], 0)), 0)
                inside, after, total = np.exp(run)[:, None], np.exp(run[-1] - run)[:, None], np.exp(run[-1])
                G = np.tril(K @ K.T * decay, -1)
                T = rule.rounded(np.linalg.inv(np.eye(n) + be * G), FINE)
                P = rule.product(Q, K.T, exact, exact) * (scale * decay)
                Kh = rule.product(T, be * inside * K, 0, FINE)
                W = rule.product(T, be * V, 0, FINE)
                if "recall" not in drop:
                    W = W - rule.product(Kh, S, u_state, u_state, least(Kh, 16), least(S, 16, True))
                o = rule.product(Q, S, exact, uc, 0.0, least(S, 16, True)) * (scale * inside)
                if "scores" not in drop:
                    o = o + rule.product(P, W, uc, uc, least(P, 1), least(W, 16, True))
                out.x[b, at, h], out.e[b, at, h] = o.x, o.e
                kept.append((at, Q, K, V, be, decay, inside, after, total, G, T, P, Kh, W, S))
                faded = rule.rounded(S * total, FINE)
                Z = W * after
                S = faded + rule.product(Z.T, K, u_state, exact, least(Z, 16, True).T, least(K, C)).T if "write" not in drop else faded
            last.x[b, h], last.e[b, h] = S.x, S.e
            if not back:
                continue
            D = Off(np.zeros((d, d)) if x["dstate_out"] is None else x["dstate_out"][b, h])
            for at, Q, K, V, be, decay, inside, after, total, G, T, P, Kh, W, S in reversed(kept):
                do = x["dout"][b, at, h]
                dW = rule.product(P.T, do, FINE, exact)
                dW = dW + rule.product(K, D, exact, FINE, least(K, C), least(D, 16, True)) * after
                dR = rule.product(T.T, dW, uc, uc, least(T, C).T, least(dW, C, True))
                strict = np.tril(decay, -1)
                of_w, of_r, of_s, of_d = least(W, C), least(dR, C), least(S, d), least(D, d)   # planes of a chunk
                dRW = rule.product(dR, W.T, uc, uc, of_r, of_w.T)
                A = rule.product(do, W.T, exact, uc, 0.0, of_w.T) * (scale * decay)
                L = dRW * (-be * strict)
                reads = rule.product(do, S.T, exact, uc, 0.0, of_s.T) * (scale * inside)
                recalls = rule.product(dR, S.T, uc, uc, of_r, of_s.T)
                writes = rule.product(W, D.T, uc, uc, of_w, of_d.T) * after
                of_a, of_l = least(A, C), least(L, C)
                none = lambda name, y: y * (0.0 if name in drop else 1.0)
                dq = none("reads", reads) + none("A K", rule.product(A, K, uc, exact, least(A, 1), least(K, C)))
                dk = none("A^T Q", rule.product(A.T, Q, uc, exact, of_a, least(Q, C))) + none("L K", rule.product(L, K, uc, exact, of_l))
                dk = dk + none("L^T K", rule.product(L.T, K, uc, exact, of_l, least(K, C))) - none("recalls", recalls * (be * inside))
                dk = dk + none("writes", writes)
                dv = dR * be
                dbeta = (dR * V).sum(1) - none("e^b K S", (recalls * (inside * K)).sum(1)) - none("rows", (dRW * G).sum(1))
                pairs = A * rule.product(Q, K.T, exact, exact) + L * rule.product(K, K.T, exact, exact)
                pairs = pairs * np.tril(np.ones_like(decay), -1)
                if "pairs" in drop:
                    pairs = pairs * 0.0
                enters = none("enters", (reads * Q).sum(1) - (recalls * (be * inside * K)).sum(1))
                leaves = none("leaves", (writes * K).sum(1))
                through = none("through", (S * D).sum((0, 1)) * total)
                dg = []
                for j in range(len(decay)):
                    parts = (Off(pairs.x[j:, :j], pairs.e[j:, :j]).sum((0, 1)), Off(enters.x[j:], enters.e[j:]).sum(0),
                             Off(leaves.x[:j], leaves.e[:j]).sum(0), through)
                    dg.append((sum(p.x for p in parts), np.sqrt(sum(p.e ** 2 for p in parts))))
                dg = Off([p[0] for p in dg], [p[1] for p in dg])
                for name, y in zip(names, (dq, dk, dv, dg, dbeta)):
                    grads[name].x[b, at, h], grads[name].e[b, at, h] = y.x, y.e
                faded = rule.rounded(D * total, FINE)
                D = faded + rule.product((scale * inside * Q).T, do, FINE, exact) - rule.product(Kh.T, dW, u_state, u_state, least(Kh, 16).T, least(dW, 16, True))
            first.x[b, h], first.e[b, h] = D.x, D.e
    if not back:
        return out, last
    for name in ("dq", "dk"):                          # of the heads that share them
        y = grads[name]
        share = lambda z, f: f(z.reshape(B, N, -1, H // x["q"].shape[2], d))
        grads[name] = Off(share(y.x, lambda z: z.sum(3)), share(y.e, lambda z: np.sqrt((z ** 2).sum(3))))
    return tuple(grads[n] for n in names) + (first,)


def over_axes(z, axes):
    return np.sqrt((z ** 2).sum(axes))


def state_bound(last):
    """Of the norm of each (b, h)'s state."""
    return MARGIN * over_axes(last.e, (-2, -1)) + 2.0 ** -24 * over_axes(last.x, (-2, -1))


def out_bound(out, dtype):
    """Of each token's row of a head: its own error alone, no other token's."""
    return MARGIN * over_axes(out.e, -1) + HALF[dtype] * over_axes(out.x, -1) + 1e-30


def grad_bound(name, y, dtype):
    """Of the norm of each head's gradient; dq and dk of shared heads are summed from float32, dstate stays in it."""
    axes = (-2, -1) if name == "dstate" else (1, 3) if y.x.ndim == 4 else (1,)
    own = 2.0 ** -24 if name == "dstate" else HALF[dtype]
    return MARGIN * over_axes(y.e, axes) + own * over_axes(y.x, axes) + 1e-30, axes


def token_bound(y, dtype):
    """Of each token's own gradient, a row or a value."""
    size = lambda z: over_axes(z, -1) if z.ndim == 4 else np.abs(z)
    return MARGIN * size(y.e) + HALF[dtype] * size(y.x) + 1e-30, size
