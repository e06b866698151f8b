"""Operators over sequences and the optimiser step, without a GPU: the
references' gradients against central differences, and every refusal of the
entry points, which comes before any HIP call (all pointers here are fake)."""
import ctypes

import numpy as np
import pytest

import seq_reference as R
from cnn_convolution_forward_amd import binding as B

X, G, I, Y, W, D, S, H, WS = (0x10000000 * i for i in range(1, 10))


# ---- the references' gradients -----------------------------------------------

def _difference(f, args, grads, rng, eps=1e-5):
    """Central differences of f along random directions of each argument, against the gradients: the
    third derivatives of these functions on O(1) data leave less than 1e-7 of the sum of magnitudes,
    rounding 1e-16 / eps of f's terms."""
    for i, (a, g) in enumerate(zip(args, grads)):
        d = rng.standard_normal(a.shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = a + eps * d, a - eps * d
        num, ana = (f(*up) - f(*dn)) / (2 * eps), (g * d).sum()
        assert abs(num - ana) <= 1e-6 * (np.abs(g * d).sum() + 1), (i, num, ana)


@pytest.mark.parametrize("K,silu,L", [(1, True, 5), (2, False, 1), (4, True, 7), (4, True, 2), (3, False, 9)])
def test_conv_reference_gradient(K, silu, L):
    rng = np.random.default_rng(K * 10 + L)
    x, w, b, st = rng.standard_normal((L, 3)), rng.standard_normal((3, K)), rng.standard_normal(3), rng.standard_normal((K - 1, 3))
    dy = rng.standard_normal((L, 3))
    f = lambda x, w, b, st: (R.conv(x, w, b, st, silu)[0] * dy).sum()
    _difference(f, (x, w, b, st), R.conv_grad(x, w, b, st, silu, dy)[0], rng)


@pytest.mark.parametrize("L", [1, 2, 17])
def test_scan_reference_gradient(L):
    rng = np.random.default_rng(L)
    x, g, u = (rng.standard_normal((L, 3)) for _ in range(3))
    decay, h0, dy, dh = rng.uniform(-4, 0, 3), rng.standard_normal(3), rng.standard_normal((L, 3)), rng.standard_normal(3)

    def f(x, g, u, decay, h0):
        h = R.scan(x, g, u, decay, 8.0, h0)[0]
        return (h * dy).sum() + (h[-1] * dh).sum()

    _difference(f, (x, g, u, decay, h0), R.scan_grad(x, g, u, decay, 8.0, h0, dy, dh)[0], rng)


# ---- refusals ------------------------------------------------------------------

def _seq(**kw):
    return B.SeqParams(**{**dict(dtype=1, B=2, T=70, C=24, offsets=None, tokens=0), **kw})


def _cf(seq=None, K=4, silu=1, x=X, ldx=24, w=W, b=D, st=S, y=Y, ldy=24, so=None):
    return B.conv_causal_fwd(_seq() if seq is None else seq, K, silu, x, ldx, w, b, st, y, ldy, so)


def test_sequence_batches_are_checked():
    assert B.lib().conv_causal_fwd(None, 4, 1, X, 24, W, D, S, Y, 24, None, None) == 1
    for bad in (dict(dtype=2), dict(dtype=-1), dict(B=0), dict(T=-1), dict(C=0), dict(offsets=WS, tokens=-1),
                dict(offsets=WS + 2)):
        assert _cf(_seq(**bad)) == 2, bad
    for big in (dict(B=1 << 15, T=1 << 15), dict(C=(1 << 20) + 1), dict(B=1 << 12, C=1 << 19),
                dict(B=1 << 22, T=65, C=1), dict(B=1, T=1 << 30), dict(offsets=WS, tokens=1 << 30)):
        assert _cf(_seq(**big), ldx=1 << 21, ldy=1 << 21) == 4, big


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(K=0), 2), (dict(K=9), 2), (dict(silu=2), 2),
    (dict(ldx=23), 2), (dict(ldy=0), 2), (dict(x=X + 1), 2), (dict(b=D + 2), 2), (dict(y=X), 5), (dict(y=X + 48 * 139), 5),
    (dict(y=W), 5), (dict(y=D - 4), 5), (dict(so=S + 2), 5), (dict(so=Y), 5), (dict(so=X + 100), 5)])
def test_causal_fwd_refusals(kw, status):
    assert _cf(**kw) == status


def test_column_slices_of_one_buffer_do_not_overlap():
    """y beside x in rows of 72 elements: refused only where the columns meet (the call itself, with a
    seq of 0 rows, would launch: so only the refusing side runs here)."""
    assert _cf(ldx=72, ldy=72, y=X + 2 * 23) == 5
    assert _cf(ldx=72, ldy=72, y=X + 2 * 60) == 5          # wraps into the next row's x
    assert _cf(ldx=72, ldy=48, y=X + 2 * 24) == 5          # other strides: columns cross


def test_causal_bwd_refusals():
    need = B.conv_causal_bwd_workspace_bytes(_seq(), 4)
    assert need > 0 and need % (5 * 24 * 4) == 0
    assert B.conv_causal_bwd_workspace_bytes(None, 4) == 0 and B.conv_causal_bwd_workspace_bytes(_seq(), 9) == 0
    dy, dx, dw, db, ds = (0x01000000 * i + X for i in range(1, 6))

    def f(seq=None, K=4, silu=0, x=X, ldx=24, dy=dy, dx=dx, dw=dw, db=db, ds=ds, ws=WS, n=need):
        return B.conv_causal_bwd(_seq() if seq is None else seq, K, silu, x, ldx, W, D, S, dy, 24, dx, 24, dw, db, ds, ws, n)

    assert f(x=None) == 1 and f(dy=None) == 1 and f(dx=None) == 1 and f(dw=None) == 1
    assert f(K=0) == 2 and f(silu=-1) == 2 and f(ldx=20) == 2
    assert f(ws=None) == 6 and f(n=need - 1) == 6 and f(ws=WS + 8) == 6
    assert f(dx=dy + 16) == 5 and f(dw=W) == 5 and f(db=dw + 4) == 5 and f(ds=S) == 5 and f(ws=X) == 5


def test_scan_refusals():
    def f(seq=None, scale=8.0, x=X, ldx=24, g=G, i=I, d=D, h0=H, y=Y, hT=S, st=None, ws=WS, n=1 << 30):
        return B.conv_scan_fwd(_seq() if seq is None else seq, scale, x, ldx, g, 24, i, 24, d, h0, y, 24, hT, st, ws, n)

    assert f(x=None) == 1 and f(g=None) == 1 and f(i=None) == 1 and f(d=None) == 1 and f(y=None) == 1
    for bad in (-1.0, float("nan"), float("inf")):
        assert f(scale=bad) == 2
    assert f(ldx=1) == 2 and f(x=X + 1) == 2 and f(hT=S + 2) == 2 and f(_seq(B=0)) == 2
    assert f(y=X) == 5 and f(y=G + 24) == 5 and f(hT=H) == 5 and f(st=S) == 5 and f(st=Y) == 5
    assert B.conv_scan_fwd_workspace_bytes(None) == 0 and B.conv_scan_bwd_workspace_bytes(_seq(C=0)) == 0
    dy, dx, dg, di, dd, d0 = (0x01000000 * i + X for i in range(1, 7))
    need = B.conv_scan_bwd_workspace_bytes(_seq())
    assert need > 0

    def b(seq=None, scale=8.0, states=S, dy=dy, dx=dx, dg=dg, di=di, dd=dd, d0=d0, ws=WS, n=need, lddx=24):
        return B.conv_scan_bwd(_seq() if seq is None else seq, scale, X, 24, G, 24, I, 24, D, states, dy, 24, H, dx, lddx,
                               dg, 24, di, 24, dd, d0, ws, n)

    assert b(states=None) == 1 and b(dy=None) == 1 and b(dx=None) == 1 and b(dg=None) == 1 and b(di=None) == 1 and b(dd=None) == 1
    assert b(scale=-0.5) == 2 and b(lddx=7) == 2
    assert b(n=need - 1) == 6 and b(ws=None) == 6 and b(ws=WS + 4) == 6
    assert b(dx=X) == 5 and b(dg=dx + 4) == 5 and b(dd=D) == 5 and b(d0=H) == 5 and b(ws=S) == 5


def test_step_refusals():
    c = lambda x=X, w=W, st=S, y=Y, K=4, seq=None: B.conv_causal_step(_seq() if seq is None else seq, K, 1, x, 24, w, D, st, y, 24)
    assert c(x=None) == 1 and c(w=None) == 1 and c(st=None) == 1 and c(y=None) == 1
    assert c(K=9) == 2 and c(seq=_seq(C=0)) == 2 and c(y=X) == 5 and c(st=X) == 5 and c(y=S) == 5
    g = lambda h=H, y=Y, scale=8.0: B.conv_scan_step(_seq(), scale, X, 24, G, 24, I, 24, D, h, y, 24)
    assert g(h=None) == 1 and g(y=None) == 1 and g(scale=float("nan")) == 2 and g(y=X) == 5 and g(h=D) == 5


def test_adamw_refusals():
    ok = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, bits=32, grad_dtype=0, seed=0, grad_scale=None)
    ten = dict(n=100, p=X, g=G, m=I, v=Y, m_scale=None, v_scale=None, copy=W, weight_decay=0.01)

    def f(o=None, **t):
        arr = (B.AdamwTensor * 1)(B.AdamwTensor(**{**ten, **t}))
        return B.conv_adamw_step(B.AdamwOptions(**{**ok, **(o or {})}), arr, 1)

    assert B.lib().conv_adamw_step(None, None, 0, None) == 1
    assert B.conv_adamw_step(B.AdamwOptions(**ok), None, 1) == 1
    assert B.conv_adamw_step(B.AdamwOptions(**ok), None, -1) == 2
    for k in ("p", "g", "m", "v"):
        assert f(**{k: None}) == 1
    assert f(dict(bits=8)) == 1                                  # no scales
    nan, inf = float("nan"), float("inf")
    for o in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(beta2=nan), dict(lr=-1.0), dict(lr=nan), dict(eps=inf),
              dict(bits=16), dict(grad_dtype=2), dict(grad_scale=W + 1)):
        assert f(o) == 2, o
    assert f(n=-1) == 2 and f(weight_decay=-1.0) == 2 and f(p=X + 2) == 2 and f(copy=W + 1) == 2
    assert f(n=1 << 31) == 4
    assert f(m=X) == 5 and f(v=I + 396) == 5 and f(copy=G) == 5 and f(dict(grad_scale=X + 8)) == 5
    assert f(dict(bits=8), m_scale=S, v_scale=S) == 5
    # nothing to do: no launch
    assert B.conv_adamw_step(B.AdamwOptions(**ok), None, 0) == 0
    assert f(n=0, p=None) == 0


def test_state_values_refusals():
    ten = dict(n=100, p=None, g=None, m=I, v=Y, m_scale=S, v_scale=H, copy=None, weight_decay=0)

    def f(mo=X, vo=G, **t):
        arr = (B.AdamwTensor * 1)(B.AdamwTensor(**{**ten, **t}))
        return B.conv_adamw_state_values(arr, 1, (ctypes.c_void_p * 1)(mo), (ctypes.c_void_p * 1)(vo))

    assert B.conv_adamw_state_values(None, 1, None, None) == 1 and B.conv_adamw_state_values(None, -1, None, None) == 2
    assert f(mo=None) == 1 and f(m=None) == 1 and f(v_scale=None) == 1
    assert f(n=-3) == 2 and f(mo=X + 2) == 2 and f(n=1 << 31) == 4 and f(mo=I) == 5 and f(vo=X) == 5
    assert f(n=0) == 0


def test_helpers_refuse_cpu_tensors_and_wrong_shapes():
    import torch
    x = torch.zeros(2, 5, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError):
        B.causal_conv(x, w)
    with pytest.raises(ValueError):
        B.causal_conv(torch.zeros(5, 8), w)                       # packed rows need offsets
    with pytest.raises(TypeError):
        B.causal_conv(x.double(), w)
    with pytest.raises(ValueError):
        B.make_seq(torch.zeros(5, 8), offsets=torch.zeros(3, dtype=torch.int32), max_len=5)
    with pytest.raises(ValueError):
        B.gated_scan(x, x, x, torch.zeros(8))
    with pytest.raises(ValueError):
        B.AdamW([x], [x])
    with pytest.raises(ValueError):
        B.AdamW([x], [x], bits=4)


def test_scan_backward_of_no_tokens_needs_no_states():
    """Packed rows with T = 0: the (B, 0, C) states have no address.  Refused for its workspace here, not for them."""
    seq = _seq(T=0, offsets=0x100, tokens=50)
    call = lambda seq: B.conv_scan_bwd(seq, 8.0, X, 24, G, 24, I, 24, D, None, Y, 24, None, S, 24, H, 24, WS, 24, W, None, None, 0)
    assert call(seq) == 6 and call(_seq(offsets=0x100, tokens=50)) == 1
