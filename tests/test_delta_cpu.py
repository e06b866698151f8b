"""The gated delta rule without a GPU: the reference's gradients against central
differences, the block form against it, and every refusal of the entry points and
helpers (all pointers here are fake)."""
import ctypes

import numpy as np
import pytest
import torch

import delta_reference as R
from cnn_convolution_forward_amd import binding as B

Q, K, V, G, BE, S0, Y, ST, SS, WS = (0x10000000 * i for i in range(1, 11))


def _data(rng, L, dk, dv):
    q, k, v = rng.standard_normal((L, dk)), rng.standard_normal((L, dk)), rng.standard_normal((L, dv))
    return q, k, v, -rng.uniform(0, 1, L), rng.uniform(0, 1, L), rng.standard_normal((dk, dv))


@pytest.mark.parametrize("on", [True, False])
@pytest.mark.parametrize("L", [1, 2, 9])
def test_reference_gradient(L, on):
    """Central differences along random directions; third derivatives of O(1) data leave less than 1e-6 of the terms."""
    rng = np.random.default_rng(L)
    args = list(_data(rng, L, 3, 2))
    if not on:
        args[1] /= 2
    dy, dS = rng.standard_normal((L, 2)), rng.standard_normal((3, 2))

    def f(q, k, v, g, b, S):
        y, hist = R.forward(R.unit(q, on, 1e-2)[0], R.unit(k, on, 1e-2)[0], v, g, b, S, 0.7)
        return (y * dy).sum() + (hist[-1] * dS).sum()

    (q, fq), (k, fk) = R.unit(args[0], on, 1e-2), R.unit(args[1], on, 1e-2)
    _, hist = R.forward(q, k, *args[2:], 0.7)
    (dq, dk, dv, dg, db, ds), _ = R.backward(q, k, *args[2:5], hist, 0.7, dy, dS)
    grads = (R.through_unit(dq, q, fq, on), R.through_unit(dk, k, fk, on), dv, dg, db, ds)
    for i, g in enumerate(grads):
        d = rng.standard_normal(g.shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
        num = (f(*up) - f(*dn)) / 2e-5
        assert abs(num - (g * d).sum()) <= 1e-6 * (np.abs(g * d).sum() + 1), i


def test_bounds_hold_for_the_block_form_in_float32():
    """The bounds are made for more roundings than plain float32 has; they must hold for it, and must not be empty."""
    rng = np.random.default_rng(3)
    q, k, v, g, b, S = _data(rng, 130, 16, 8)
    q, k = R.unit(q, True, 0)[0], R.unit(k, True, 0)[0]
    y, hist = R.forward(q, k, v, g, b, S, 0.25)
    ey, es = R.forward_bounds(q, k, v, g, b, hist, 0.25, 8 * R.W, False)
    assert np.all(ey > 0) and np.median(ey / np.abs(y).mean()) < 2e-3 and np.all(es[-1] < 1e-2)
    s, out = S.astype(np.float32), []
    for t in range(130):
        s = s * np.float32(np.exp(g[t]))
        s = s + np.outer(k[t], b[t] * (v[t] - k[t].astype(np.float32) @ s)).astype(np.float32)
        out.append(0.25 * (q[t].astype(np.float32) @ s))
    assert np.all(np.abs(np.array(out) - y) <= ey)


# ---- refusals ------------------------------------------------------------------

def _seq(**kw):
    return B.SeqParams(**{**dict(dtype=1, B=2, T=70, C=4 * 24, offsets=None, tokens=0), **kw})


def _par(**kw):
    return B.DeltaParams(**{**dict(heads=2, heads_v=4, dim_k=16, dim_v=24, unit=1, scale=0.25, eps=1e-6), **kw})


def _f(seq=None, par=None, q=Q, ldq=32, k=K, ldk=32, v=V, ldv=96, g=G, ldg=4, b=BE, ldb=4, s0=S0, y=Y, ldy=96, sT=ST, ss=SS, ws=WS, n=1 << 30):
    return B.conv_delta_fwd(_seq() if seq is None else seq, _par() if par is None else par, q, ldq, k, ldk, v, ldv, g, ldg, b, ldb, s0, y,
                            ldy, sT, ss, ws, n)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(g=None), 1), (dict(b=None), 1), (dict(y=None), 1),
    (dict(ldq=31), 2), (dict(ldk=0), 2), (dict(ldv=95), 2), (dict(ldg=3), 2), (dict(ldb=1), 2), (dict(ldy=95), 2), (dict(q=Q + 1), 2),
    (dict(g=G + 2), 2), (dict(s0=S0 + 2), 2), (dict(ldv=1 << 22), 4), (dict(ldg=1 << 22), 4),
    (dict(ws=None), 6), (dict(n=100), 6), (dict(ws=WS + 8), 6),
    (dict(y=V), 5), (dict(y=Q + 4), 5), (dict(sT=S0), 5), (dict(ss=S0 + 4), 5), (dict(ws=Q), 5), (dict(sT=Y), 5), (dict(y=G), 5)])
def test_forward_refusals(kw, status):
    assert _f(**kw) == status


def test_heads_and_batches_are_checked():
    L = B.lib()
    assert L.conv_delta_fwd(None, ctypes.byref(_par()), *[None, 0] * 5, None, None, 0, None, None, None, 0, None) == 1
    assert L.conv_delta_fwd(ctypes.byref(_seq()), None, *[None, 0] * 5, None, None, 0, None, None, None, 0, None) == 1
    nan, inf = float("nan"), float("inf")
    for bad in (dict(heads=0), dict(heads=3), dict(heads_v=0), dict(heads_v=5), dict(dim_k=0), dict(dim_k=129), dict(dim_v=23), dict(dim_v=0),
                dict(unit=2), dict(unit=-1), dict(scale=nan), dict(scale=inf), dict(eps=-1.0), dict(eps=nan), dict(eps=inf)):
        assert _f(par=_par(**bad)) == 2, bad
        assert B.conv_delta_fwd_workspace_bytes(_seq(), _par(**bad)) == 0
    assert _f(_seq(C=129), _par(heads=1, heads_v=1, dim_v=129)) == 2
    for bad in (dict(dtype=3), dict(B=0), dict(T=-1), dict(C=95), dict(offsets=WS, tokens=-1), dict(offsets=WS + 2)):
        assert _f(_seq(**bad)) == 2, bad
    for big in (dict(B=1 << 19, T=1), dict(B=1 << 15, T=1 << 15), dict(offsets=WS, tokens=1 << 30), dict(B=500000, T=1)):
        assert _f(_seq(**big), _par(dim_k=128)) == 4, big
    assert B.conv_delta_fwd_workspace_bytes(_seq(), _par()) > 0
    assert B.conv_delta_fwd_workspace_bytes(_seq(T=0), _par()) == 0


def test_backward_refusals():
    dy, dq, dk, dv, dg, db, d0, dT = (Q + 0x01000000 * i for i in range(1, 9))
    need = B.conv_delta_bwd_workspace_bytes(_seq(), _par())
    assert need > B.conv_delta_fwd_workspace_bytes(_seq(), _par())

    def f(seq=None, par=None, q=Q, ss=SS, dy=dy, lddy=96, dT=dT, dq=dq, lddq=32, dk=dk, dv=dv, lddv=96, dg=dg, lddg=4, db=db, d0=d0, ws=WS, n=need):
        return B.conv_delta_bwd(_seq() if seq is None else seq, _par() if par is None else par, q, 32, K, 32, V, 96, G, 4, BE, 4, ss, dy, lddy,
                                dT, dq, lddq, dk, 32, dv, lddv, dg, lddg, db, 4, d0, ws, n)

    for name in ("q", "ss", "dy", "dq", "dk", "dv", "dg", "db"):
        assert f(**{name: None}) == 1, name
    assert f(lddq=31) == 2 and f(lddv=95) == 2 and f(lddy=2) == 2 and f(lddg=3) == 2 and f(dT=dT + 1) == 2 and f(par=_par(heads=3)) == 2
    assert f(lddq=1 << 22) == 4
    assert f(n=need - 1) == 6 and f(ws=None) == 6 and f(ws=WS + 4) == 6
    assert f(dq=Q) == 5 and f(dk=dq + 8) == 5 and f(dv=dy) == 5 and f(dg=G) == 5 and f(db=dg) == 5 and f(d0=dT) == 5 and f(d0=SS) == 5 and f(ws=V) == 5
    # no tokens need no states; refused for its workspace here, not for them
    seq = _seq(T=0, offsets=0x100, tokens=50)
    assert f(seq, ss=None, ws=None, n=0) == 6


def test_step_refusals():
    def f(seq=None, par=None, q=Q, k=K, v=V, g=G, b=BE, s=S0, y=Y, ldy=96, ldk=32):
        return B.conv_delta_step(_seq() if seq is None else seq, _par() if par is None else par, q, 32, k, ldk, v, 96, g, 4, b, 4, s, y, ldy)

    for name in ("q", "k", "v", "g", "b", "s", "y"):
        assert f(**{name: None}) == 1, name
    assert f(ldy=95) == 2 and f(s=S0 + 1) == 2 and f(par=_par(dim_k=200)) == 2 and f(seq=_seq(C=97)) == 2 and f(ldk=1 << 22) == 4
    assert f(y=Q) == 5 and f(s=V) == 5 and f(y=S0) == 5 and f(s=G) == 5


def test_helpers_refuse():
    q, v, g = torch.zeros(2, 5, 2, 8), torch.zeros(2, 5, 4, 6), torch.zeros(2, 5, 4)
    with pytest.raises(ValueError):
        B.delta_rule(q, q, v, g, g)                               # not on a GPU
    with pytest.raises(ValueError):
        B.delta_rule(q[0], q[0], v[0], g[0], g[0])                # packed rows need offsets
    with pytest.raises(ValueError):
        B.delta_rule_step(q, q, v, g, g, torch.zeros(2, 4, 8, 6))
    with pytest.raises(TypeError):
        B.make_delta(q.double(), v.double())
