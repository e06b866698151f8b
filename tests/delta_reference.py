"""The gated delta rule and its gradients in float64, token by token, for one
sequence and one value head; and bounds on the error of an evaluation in blocks
of 64 tokens.

A bound has two parts.  Within a block, every product and every elementwise step of
the block form is followed with the bound on its operands (class Val).  W = 2**-22 stands
for one such step: an operand of two fp16 numbers is within 2**-22 of a value, or
within 2**-28 of its tile's largest; a sum of n terms adds n 2**-24.  From block to
block only the state goes on, and there an error is carried by the recurrence itself,
I - beta k k^T times a decay: for decays <= 1 and 0 <= beta |k|^2 <= 2 it makes no column of
the state (nor, backwards, of its gradient) longer, so a column's error is at most the sum of the
blocks' own, in the 2-norm.
"""
import numpy as np

W = 2.0 ** -22
BLOCK = 64


class Val:
    """Values and a bound on the error of each."""

    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.v.shape)

    @property
    def T(self):
        return Val(self.v.T, self.e.T)

    def __neg__(self):
        return Val(-self.v, self.e)

    def __add__(self, o):
        v = self.v + o.v
        return Val(v, self.e + o.e + W * np.abs(v))

    def __sub__(self, o):
        return self + (-o)

    def __mul__(self, o):
        v = self.v * o.v
        return Val(v, np.abs(self.v) * o.e + self.e * np.abs(o.v) + self.e * o.e + W * np.abs(v))

    def __matmul__(self, o):
        a, b, n = np.abs(self.v), np.abs(o.v), self.v.shape[-1]
        top = lambda x: x.max() if x.size else 0.0
        floor = 2.0 ** -27 * (top(a) * b.sum(0)[None, :] + a.sum(1)[:, None] * top(b))
        return Val(self.v @ o.v, a @ o.e + self.e @ b + self.e @ o.e + (6 + n / 4) * W * (a @ b) + floor)

    def rounded(self, rel):
        """As an operand of fewer bits."""
        return Val(self.v, self.e + rel * np.abs(self.v))


def unit(x, on, eps):
    """Rows at unit length, and each row's factor."""
    if not on:
        return x, np.ones((len(x), 1))
    s = (x * x).sum(1, keepdims=True) + eps
    with np.errstate(divide="ignore"):
        f = np.where(s > 0, 1 / np.sqrt(s), 0.0)
    return x * f, f


def forward(q, k, v, g, beta, S, scale):
    """y, and S before every token and after the last, (L + 1, dk, dv); q and k as used."""
    L = len(q)
    y, hist = np.zeros_like(v), np.zeros((L + 1,) + S.shape)
    hist[0] = S
    for t in range(L):
        D = np.exp(g[t]) * hist[t] if np.isfinite(g[t]) else np.zeros_like(S)
        hist[t + 1] = D + np.outer(k[t], beta[t] * (v[t] - k[t] @ D))
        y[t] = scale * (q[t] @ hist[t + 1])
    return y, hist


def backward(q, k, v, g, beta, hist, scale, dy, dS):
    """dq, dk (of q and k as used), dv, dg, dbeta, ds0, and dS behind every token."""
    L = len(q)
    dq, dk, dv, dg, db = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros(L), np.zeros(L)
    behind = np.zeros((L,) + dS.shape)
    for t in range(L - 1, -1, -1):
        behind[t] = dS
        a = np.exp(g[t])
        D = a * hist[t]
        e = v[t] - k[t] @ D
        d = dS + scale * np.outer(q[t], dy[t])
        dq[t] = scale * (hist[t + 1] @ dy[t])
        z = k[t] @ d
        db[t] = z @ e
        dv[t] = beta[t] * z
        dk[t] = d @ (beta[t] * e) - D @ dv[t]
        d = d - np.outer(k[t], dv[t])
        dg[t] = (d * D).sum()
        dS = a * d
    return (dq, dk, dv, dg, db, dS), behind


def through_unit(dx, x, f, on):
    """Gradient of rows from that of the rows at unit length, x."""
    return f * (dx - x * (x * dx).sum(1, keepdims=True)) if on else dx


class Pieces:
    """What a block makes of its inputs, with bounds."""

    def __init__(self, q, k, v, g, beta, scale, ku):
        n = len(q)
        self.q, self.k, self.v = Val(q, ku * np.abs(q)), Val(k, ku * np.abs(k)), Val(v)
        self.beta, self.scale = Val(beta[:, None]), Val(np.float64(scale))
        G = np.cumsum(np.maximum(g, -1e4))
        diff = np.where(np.tril(np.ones((n, n))) > 0, G[:, None] - G[None, :], 0.0)
        low = np.tril(np.ones((n, n)))
        D = np.exp(diff) * low
        self.D = Val(D, (np.abs(diff) + 4) * W * D)
        self.E, self.F = (Val(x[:, None], 2 * W * x[:, None]) for x in (np.exp(G), np.exp(G[-1] - G)))
        self.last = Val(np.exp(G[-1]), 2 * W * np.exp(G[-1]))
        strict = Val(self.D.v * np.tril(low, -1), self.D.e * np.tril(low, -1))
        self.strict = strict
        A = self.beta * strict * (self.k @ self.k.T)
        T = np.linalg.inv(np.eye(n) + A.v)
        # of a triangular inverse by substitution and products of blocks: at most n steps behind each element
        t = np.abs(T)
        self.T = Val(T, t @ A.e @ t + (n + 8) * W * (t @ np.abs(A.v) @ t) + W * t)
        self.P = self.scale * self.D * (self.q @ self.k.T)


def _cols(e):
    """The 2-norm of each column."""
    return np.sqrt((e * e).sum(0))


def forward_bounds(q, k, v, g, beta, hist, scale, ku, half, grow=1.0):
    """Bounds of y (L, dv), and of S in front of every block and after the last token (blocks + 1, dv): the 2-norm of the
    error of a column.  q and k as used, ku their relative error; half: products for y take one fp16 number."""
    L = len(q)
    ey, es = np.zeros_like(v), [np.zeros(v.shape[1])]
    for t0 in range(0, L, BLOCK):
        r = slice(t0, min(L, t0 + BLOCK))
        p = Pieces(q[r], k[r], v[r], g[r], beta[r], scale, ku)
        S = Val(hist[t0])
        U = p.T @ (p.beta * (p.v - p.E * (p.k @ S)))
        if half:
            y = p.scale * p.E * (p.q @ S.rounded(2.0 ** -11)) + p.P.rounded(2.0 ** -11) @ U.rounded(2.0 ** -11)
        else:
            y = p.scale * p.E * (p.q @ S) + p.P @ U
        end = p.last * S + (p.F * p.k).T @ U
        # y takes S after each token, whose columns are off by no more than those in front of the block
        ey[r] = y.e + abs(scale) * np.sqrt((q[r] ** 2).sum(1))[:, None] * es[-1]
        es.append(es[-1] + grow * _cols(end.e))
    return ey, np.array(es)


def backward_bounds(q, k, v, g, beta, hist, behind, scale, dy, dsT, ku, f, on, grow=1.0):
    """Bounds of (dq, dk, dv, dg, dbeta) and of the columns of ds0 (2-norm); dq and dk as through_unit leaves them."""
    L, dk_, dv_ = len(q), q.shape[1], v.shape[1]
    eq, ek, ev, eg, eb = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros(L), np.zeros(L)
    ec = np.zeros(dv_)
    for t0 in range((L - 1) // BLOCK * BLOCK, -1, -BLOCK):
        r = slice(t0, min(L, t0 + BLOCK))
        p = Pieces(q[r], k[r], v[r], g[r], beta[r], scale, ku)
        S, dS, o = Val(hist[t0]), Val(behind[r][-1]), Val(dy[r])
        n = len(q[r])
        U = p.T @ (p.beta * (p.v - p.E * (p.k @ S)))
        Z = p.T.T @ (p.P.T @ o + p.F * (p.k @ dS))
        Bm = p.scale * p.D * (o @ U.T)
        M = -(p.strict * (Z @ U.T))
        dq = p.scale * p.E * (o @ S.T) + Bm @ p.k
        read = M @ p.k - p.E * (Z @ S.T)
        wstate = p.F * (U @ dS.T)
        write = Bm.T @ p.q + (p.beta * M).T @ p.k + wstate
        dk = p.beta * read + write
        ones = Val(np.ones((dk_, 1)))
        at = (p.k * read) @ ones
        db = (Z * p.v) @ Val(np.ones((dv_, 1))) + at
        dG = (p.q * dq) @ ones + p.beta * at - (p.k * write) @ ones
        upper = Val(np.triu(np.ones((n, n))))
        kept = p.last * (Val(np.ones((1, dk_))) @ (S * dS) @ Val(np.ones((dv_, 1)))) + Val(np.ones((1, n))) @ (p.k * wstate) @ ones
        dg = upper @ dG + kept
        d0 = p.last * dS + (p.scale * p.E * p.q).T @ o - (p.beta * p.E * p.k).T @ Z
        # dS behind the block is off by ec in each column, and so at most is dS behind each of its tokens
        kn = np.sqrt((k[r] ** 2).sum(1))
        before = np.exp(np.maximum(g[r], -1e4))[:, None, None] * hist[t0:t0 + n]
        e = v[r] - np.einsum("td,tdc->tc", k[r], before)
        u = beta[r][:, None] * e
        eq[r] = dq.e
        ek[r] = dk.e + (np.abs(u) @ ec)[:, None] + (np.abs(beta[r]) * kn)[:, None] * (np.abs(before) @ ec)
        ev[r] = (p.beta * Z).e + np.abs(beta[r])[:, None] * kn[:, None] * ec
        eb[r] = db.e[:, 0] + kn * (np.abs(e) @ ec)
        eg[r] = dg.e[:, 0] + np.sqrt((before ** 2).sum(1)) @ ec
        ec = ec + grow * _cols(d0.e)

    def back(e, x, d, f):
        if not on:
            return e
        a = np.abs(x)
        dot = (a * np.abs(d)).sum(1, keepdims=True)
        return f * (e + a * (a * e).sum(1, keepdims=True) + (2 * ku + (dk_ / 4 + 8) * W) * (np.abs(d) + a * dot))

    return eq, ek, ev, eg, eb, ec, back
