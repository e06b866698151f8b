"""Definitions, in float64 and token by token, of the operators over sequences of
tokens, with bounds on the error of a float32 evaluation beside each value.

u = 2**-23 stands for the error of one float32 operation (two units of rounding,
so that one-ulp hardware functions are covered).  A bound counts the operations
that lead to a value, in any order of the recurrence's sums; 4x covers the
second-order terms.  bf16 results are then rounded once: at most 2**-8 of the value.
"""
import numpy as np

U = 2.0 ** -23
BF16 = 2.0 ** -8


def sig(v):
    return 1.0 / (1.0 + np.exp(-v))


def tol(ref, err, bf16):
    """The bound for an output: the float32 error, then the output's own rounding."""
    return 4 * err + (BF16 * (np.abs(ref) + 4 * err) if bf16 else U * np.abs(ref)) + 1e-37


# ---- causal convolution: x (L, C) of one sequence, state (K-1, C) ---------------

def conv(x, w, bias, state, silu):
    """y, its error bound, the state after it, and what the backward pass needs."""
    L, C = x.shape
    K = w.shape[1]
    full = np.concatenate([state, x])
    p, S = np.zeros((L, C)) + bias, np.zeros((L, C)) + np.abs(bias)
    for t in range(L):
        for j in range(K):
            p[t] += w[:, j] * full[t + j]
            S[t] += np.abs(w[:, j] * full[t + j])
    ep = (K + 1) * U * S
    if not silu:
        return p, ep, full[L:], (full, p, ep)
    with np.errstate(over="ignore"):
        y = p * sig(p)
    # |d silu/dp| <= 1.1; sigmoid: |p| u from its argument, 4 u of its own
    return y, 1.1 * ep + (np.abs(p) + 6) * U * np.abs(y), full[L:], (full, p, ep)


def conv_grad(x, w, bias, state, silu, dy):
    """dx, dw, db, dstate and their error bounds for one sequence."""
    L, C = x.shape
    K = w.shape[1]
    full, p, ep = conv(x, w, bias, state, silu)[3]
    f, ef = np.ones((L, C)), np.zeros((L, C))
    if silu:
        s = sig(p)
        f = s * (1 + p * (1 - s))
        # |d2 silu/dp2| <= 0.5, and the factor's own operations
        ef = 0.5 * ep + (np.abs(p) + 8) * U * s * (1 + np.abs(p))
    dp, edp = dy * f, np.abs(dy) * (ef + U * np.abs(f))
    g, eg = np.zeros((L + K - 1, C)), np.zeros((L + K - 1, C))
    dw, edw = np.zeros((C, K)), np.zeros((C, K))
    for j in range(K):
        g[j:j + L] += w[:, j] * dp
        eg[j:j + L] += np.abs(w[:, j]) * (edp + (K + 1) * U * np.abs(dp))
        dw[:, j] = (dp * full[j:j + L]).sum(0)
        edw[:, j] = (np.abs(full[j:j + L]) * (edp + (L + 8) * U * np.abs(dp))).sum(0)
    db, edb = dp.sum(0), (edp + (L + 8) * U * np.abs(dp)).sum(0)
    return (g[K - 1:], dw, db, g[:K - 1]), (eg[K - 1:], edw, edb, eg[:K - 1])


# ---- gated recurrence: x, g, u (L, C) of one sequence ----------------------------

def gates(g, u, decay, scale):
    """k, r, s, a, m and the relative errors of z = k r, a, s and m."""
    k = scale * np.logaddexp(0.0, decay)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        r, s = (np.where(v < 2.0 ** -126, 0.0, v) for v in (sig(g), sig(u)))      # part of the definition
        z = k * r
        a, v = np.exp(-z), -np.expm1(-2 * z)
        m = np.sqrt(v)
        dz = (np.minimum(np.abs(g), 90) + 12) * U
        da = z * (dz + 2 * U) + 2 * U
        ds = (np.minimum(np.abs(u), 90) + 4) * U
        # the series keeps z's relative error; the difference 1 - a^2 (from w = 2z = 1/4 on) has an absolute one
        dv = np.where(2 * z < 0.25, dz + 4 * U, (2 * a * a * da + 2 * U) / np.maximum(v, 0.2))
    return k, r, s, a, m, dz, da, ds, dv / 2 + 2 * U


def scan(x, g, u, decay, scale, h0):
    """h of every token (L, C), its error bound, and h before every token."""
    k, r, s, a, m, dz, da, ds, dm = gates(g, u, decay, scale)
    b = m * s * x
    db = (dm + ds + 3 * U) * np.abs(b)
    h, e = h0.astype(np.float64).copy(), np.zeros_like(h0, dtype=np.float64)
    hs, es, before, ebefore = (np.zeros_like(b) for _ in range(4))
    for t in range(len(b)):
        before[t], ebefore[t] = h, e
        e = a[t] * e + (da[t] + U) * a[t] * np.abs(h) + db[t]
        h = a[t] * h + b[t]
        e = e + U * np.abs(h)
        hs[t], es[t] = h, e
    return hs, es, before, ebefore


def scan_grad(x, g, u, decay, scale, h0, dy, dhT):
    """(dx, dgate, dinp, ddecay, dh0) and their error bounds for one sequence."""
    k, r, s, a, m, dz, da, ds, dm = gates(g, u, decay, scale)
    before, eb = scan(x, g, u, decay, scale, h0)[2:]
    L = len(x)
    dh, edh = np.zeros_like(x), np.zeros_like(x)
    e, ee = dhT.astype(np.float64).copy(), np.zeros_like(dhT, dtype=np.float64)
    for t in range(L - 1, -1, -1):
        dh[t] = dy[t] + e
        edh[t] = ee + U * (np.abs(dy[t]) + np.abs(e))
        e = a[t] * dh[t]
        ee = a[t] * edh[t] + (da[t] + U) * np.abs(e)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(m > 0, s * x * a * a / np.where(m > 0, m, 1), 0.0)
    dla = dh * (a * before - q)
    edla = edh * (np.abs(a * before) + np.abs(q)) + np.abs(dh) * (
        a * eb + np.abs(a * before) * (da + 3 * U) + np.abs(q) * (2 * da + dm + ds + 5 * U))
    dx = dh * m * s
    edx = edh * m * s + np.abs(dx) * (dm + ds + 3 * U)
    di = dx * x * (1 - s)
    # 1 - s is off by 2 u in itself, whatever it is
    edi = np.abs(x) * (edx * (1 - s) + np.abs(dx) * 4 * U) + np.abs(di) * (np.minimum(np.abs(u), 90) + 4) * U
    dg = -k * dla * r * (1 - r)
    edg = k * r * (edla * (1 - r) + np.abs(dla) * 4 * U) + np.abs(dg) * (2 * dz + 6 * U)
    dk = (r * dla).sum(0)
    edk = (r * (edla + np.abs(dla) * (dz + (L + 8) * U))).sum(0)
    f = -scale * sig(decay)
    dd = f * dk
    edd = np.abs(f) * edk + np.abs(dd) * (np.abs(decay) + 6) * U
    return (dx, dg, di, dd, e), (edx, edg, edi, edd, ee)
