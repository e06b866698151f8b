"""Infinities in sequences go where the definition, taken token by token, sends
them: an infinite value or gradient passes every factor above 0, however small
the product of many is, and terms that a sum does not have are not there."""
import numpy as np
import pytest
import torch

import seq_reference as R
from cnn_convolution_forward_amd import binding as B

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _cuda(a, dt=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dt).to("cuda")


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _same(got, ref, err, half, label):
    """NaN and infinities in the same places, and within the bound elsewhere."""
    got = _np(got)
    for f in (np.isnan, np.isposinf, np.isneginf):
        bad = np.argwhere(f(got) != f(ref))
        assert not len(bad), "%s: %s at %s: gpu %r, definition %r" % (label, f.__name__, tuple(bad[0]), got[tuple(bad[0])], ref[tuple(bad[0])])
    on = np.isfinite(ref)
    bound = R.tol(ref[on], err[on], half)
    assert np.all(np.abs(got[on] - ref[on]) <= bound), label


# lengths about a wave's run, a chunk and several; factors exp(-24) to exp(-2) a token: 16 of them leave no float32
LENGTHS = [20, 100, 130, 700]


def _inputs(L, C, dt, seed):
    rng = np.random.default_rng(seed)
    x, g, u, dy = (_cuda(rng.standard_normal((1, L, C)), dt) for _ in range(4))
    return rng, x, g, u, dy, _cuda(np.full(C, 3.0)), _cuda(rng.standard_normal((1, C))), _cuda(rng.standard_normal((1, C)))


@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_states_and_inputs_pass_strong_decay(dtype, L):
    dt, C, inf = DT[dtype], 9, float("inf")
    _, x, g, u, _, decay, h0, _ = _inputs(L, C, dt, L)
    h0[0, 0], h0[0, 1] = inf, -inf
    x[0, 3, 2], x[0, L // 2, 3], x[0, L - 1, 4] = inf, -inf, inf
    h0[0, 5] = inf                                  # meets its opposite: NaN from there on
    x[0, L // 2, 5] = -inf
    h0[0, 6], x[0, 5, 6] = inf, inf                 # and its like
    y, hT, st = B.gated_scan(x, g, u, decay, h0=h0, with_states=True)
    with np.errstate(invalid="ignore"):
        h, e, before, eb = R.scan(_np(x)[0], _np(g)[0], _np(u)[0], _np(decay), 8.0, _np(h0)[0])
    _same(y[0], h, e, dtype == "bf16", "y")
    _same(hT[0], h[-1], e[-1], False, "hT")
    _same(st[0], before[::64], eb[::64], False, "states")
    one = h0.clone()                                # and token by token
    ys = torch.stack([B.gated_scan_step(x[:, t], g[:, t], u[:, t], decay, one) for t in range(L)], 1)
    assert torch.equal(torch.isnan(ys), torch.isnan(y)) and torch.equal(torch.isinf(ys), torch.isinf(y))


@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_gradients_pass_strong_decay(dtype, L):
    dt, C, inf = DT[dtype], 8, float("inf")
    _, x, g, u, dy, decay, h0, dh = _inputs(L, C, dt, L + 1)
    _, _, st = B.gated_scan(x, g, u, decay, h0=h0, with_states=True)
    dh[0, 0], dh[0, 1] = inf, -inf
    dy[0, L - 2, 2], dy[0, L // 2, 3], dy[0, 0, 4] = inf, -inf, inf
    dh[0, 5], dy[0, L // 2, 5] = inf, -inf
    got = B.gated_scan_backward(x, g, u, decay, dy, st, dh=dh)
    with np.errstate(invalid="ignore"):
        ref, err = R.scan_grad(_np(x)[0], _np(g)[0], _np(u)[0], _np(decay), 8.0, _np(h0)[0], _np(dy)[0], _np(dh)[0])
    for i, name in enumerate(("dx", "dgate", "dinp")):
        _same(got[i][0], ref[i], err[i], dtype == "bf16", name)
    _same(got[4][0], ref[4], err[4], False, "dh0")
    _same(got[3], ref[3], err[3] * (2 + L / 512), False, "ddecay")


def test_zero_factor_stops_infinities_as_nan():
    """A factor that is 0 makes 0 * inf of an infinite state, and 0 of a finite one, in every form."""
    L, C = 300, 3
    x, u = torch.ones(1, L, C, device="cuda"), torch.zeros(1, L, C, device="cuda")
    g = torch.zeros(1, L, C, device="cuda")
    g[0, 150] = float("inf")
    decay = torch.full((C,), 40.0, device="cuda")           # a = exp(-320 r): 0 where the gate is open, exp(-160) = 0 half way
    decay[1] = 2.0
    h0 = torch.full((1, C), float("inf"), device="cuda")
    h0[0, 2] = 1.0
    y, _ = B.gated_scan(x, g, u, decay, h0=h0)
    assert bool(torch.isnan(y[0, :, 0]).all()) and bool((y[0, :, 1] == float("inf")).all()) and bool(torch.isfinite(y[0, :, 2]).all())


# ---- causal convolution: a term that the sum does not have ------------------------

@pytest.mark.parametrize("dtype,C", [("f32", 3), ("f32", 8), ("bf16", 24)])
@pytest.mark.parametrize("weight", [float("inf"), float("nan")])
def test_weights_touch_only_the_terms_there_are(dtype, C, weight):
    """dX[t] sums w[j] dp[t+K-1-j] over the tokens there are: near a sequence's end, and in front of its start
    for the carried rows, a weight whose token is missing does not enter."""
    dt, K = DT[dtype], 4
    for lens in ([1], [2], [7], [64], [65], [130]):
        L = lens[0]
        rng = np.random.default_rng(L)
        x, dy = (_cuda(rng.standard_normal((1, L, C)), dt) for _ in range(2))
        for j in range(K):
            w = _cuda(rng.standard_normal((C, K)), dt)
            w[:, j] = weight
            dx, dw, db, ds = B.causal_conv_backward(x, w, dy, state=_cuda(rng.standard_normal((1, K - 1, C)), dt))
            whole = np.zeros((L + K - 1, C))                   # rows -3 .. L-1 of dX
            wv, dp, err = _np(w), _np(dy)[0], np.zeros((L + K - 1, C))
            with np.errstate(invalid="ignore"):
                for i in range(K):
                    whole[i:i + L] += wv[:, i] * dp
                    err[i:i + L] += (K + 1) * R.U * np.abs(wv[:, i] * dp)
            _same(dx[0], whole[K - 1:], err[K - 1:], dtype == "bf16", "dx, %d tokens, tap %d" % (L, j))
            _same(ds[0], whole[:K - 1], err[:K - 1], dtype == "bf16", "dstate, %d tokens, tap %d" % (L, j))
