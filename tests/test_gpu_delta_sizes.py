"""Values far apart in size, and ones that are not finite, in the gated delta rule: what a token's results do not depend on
costs them no bits.  Powers of two are exact, so most tests ask for equal bits; the rest go against the definition in
float64, token by token, with the infinities and NaN that it has."""
import numpy as np
import pytest
import torch

import delta_reference as R
from cnn_convolution_forward_amd import binding as B
from test_gpu_delta import NAN, Case, _np

pytestmark = pytest.mark.gpu

INF = float("inf")


def _forward(c, **other):
    d = dict(zip("qkvgb", c.data()))
    return B.delta_rule(*{**d, **other}.values(), s0=c.s0, with_states=True, **c.opts())


def _backward(c, states, dy=None, **other):
    d = dict(zip("qkvgb", c.data()))
    return B.delta_rule_backward(*{**d, **other}.values(), c.dy if dy is None else dy, states, ds=c.ds, **c.opts())


# ---- columns of values and of upstream gradients -----------------------------------------

@pytest.mark.parametrize("dt,unit", [("bf16", True), ("f32", True), ("f32", False)])
@pytest.mark.parametrize("token,clean", [(40, 32), (63, 32), (70, 64), (100, 96), (127, 96)])
def test_large_values_leave_earlier_tokens_alone(dt, unit, token, clean):
    """A value 2**60 times the others', which no token before it depends on: up to the 32 tokens of its own, the same bits."""
    c = Case(dt, [130], 2, 4, 40, 48, unit=unit, seed=30)
    y0, _, st0 = _forward(c)
    v = c.v.clone()
    v[:, token] *= 2.0 ** 60
    y, _, st = _forward(c, v=v)
    assert torch.equal(y[:, :clean], y0[:, :clean]) and torch.equal(st[:, :token // 64 + 1], st0[:, :token // 64 + 1])
    assert not torch.equal(y[:, clean:], y0[:, clean:])


@pytest.mark.parametrize("dt,unit", [("bf16", True), ("f32", True), ("f32", False)])
@pytest.mark.parametrize("token,clean", [(0, 32), (10, 32), (31, 32), (50, 64), (64, 96), (90, 96)])
def test_large_upstream_gradients_leave_later_tokens_alone(dt, unit, token, clean):
    c = Case(dt, [130], 2, 4, 40, 48, unit=unit, seed=31)
    st = _forward(c)[2]
    want = _backward(c, st)
    dy = c.dy.clone()
    dy[:, token] *= 2.0 ** 60
    got = _backward(c, st, dy)
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        assert torch.equal(a[:, clean:], b[:, clean:]), name
        assert not torch.equal(a[:, :clean], b[:, :clean]), name


@pytest.mark.parametrize("dt,unit", [("bf16", True), ("f32", True), ("f32", False)])
def test_upstream_gradients_of_any_size(dt, unit):
    """A query's gradient is linear in the upstream gradient of its token, and depends on no other's."""
    c = Case(dt, [130], 2, 4, 40, 48, unit=unit, seed=37)
    st = _forward(c)[2]
    f = torch.from_numpy(np.ldexp(1.0, np.random.default_rng(2).integers(-40, 40, (1, 130, 1, 1)))).float().cuda()
    same = torch.equal(_backward(c, st, (c.dy * f).to(c.dt))[0], (_backward(c, st)[0] * f).to(c.dt))
    assert same


def _definition(q, k, v, g, b, S, scale):
    """The recurrence with the infinities and NaN that it makes."""
    y = np.zeros_like(v)
    with np.errstate(all="ignore"):
        for t in range(len(q)):
            S = np.exp(g[t]) * S
            S = S + np.outer(k[t], b[t] * (v[t] - k[t] @ S))
            y[t] = scale * (q[t] @ S)
    return y, S


def _held(c, clean, name, token, head, bad, first):
    """One bad value in an input: outputs that are finite have to be the definition's, those of tokens from `first` on may be NaN."""
    data = dict(zip("qkvgb", (t.clone() for t in c.data())))
    x = data[name]
    x[(0, token, head) + ((3,) if x.dim() == 4 else ())] = bad
    y, sT, _ = _forward(c, **data)
    c2 = Case.__new__(Case)
    c2.__dict__.update(c.__dict__)
    c2.q, c2.k, c2.v, c2.g, c2.beta = data.values()
    y, sT, yc = _np(y).reshape(-1, c.Hv, c.dv), _np(sT), _np(clean[0]).reshape(-1, c.Hv, c.dv)
    with np.errstate(all="ignore"):
        todo = list(c2.sequences())
    for (i, h, hk, r, q, k, v, g, b, _, _), (*_, q0, k0, v0, g0, b0, _, _) in zip(todo, c.sequences()):
        at = "%s token %d head %d unit %d" % (name, token, h, c.unit)
        mine = head == (hk if name in "qk" else h)
        ref, S = _definition(q, k, v, g, b, _np(c.s0)[i, h], c.scale)
        fin, got = np.isfinite(ref), np.isfinite(y[r, h])
        assert mine or fin.all()
        assert not (got & ~fin).any(), at                            # nothing finite where the definition is not
        assert got[:first].all() if mine else got.all(), at
        _, hist = R.forward(q0, k0, v0, g0, b0, _np(c.s0)[i, h], c.scale)
        grow = 2 * c.dk ** 0.5 if max(c.lens) > 448 else 1.0          # as in test_gpu_delta
        ey, es = R.forward_bounds(q0, k0, v0, g0, b0, hist, c.scale, c.ku(), False, grow)
        tol = ey + (2.0 ** -8 * (np.abs(ref) + ey) if c.half else 2.0 ** -23 * np.abs(ref))
        with np.errstate(invalid="ignore"):
            assert not (got & ~(np.abs(y[r, h] - ref) <= tol)).any(), at
            sg, sf = np.isfinite(sT[i, h]), np.isfinite(S)
            assert not (sg & ~sf).any() and not (sg & ~(np.abs(sT[i, h] - S) <= es[-1] + 2.0 ** -23 * np.abs(S))).any(), at


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dt,unit", [("bf16", True), ("bf16", False), ("f32", True), ("f32", False)])
def test_values_that_are_not_finite(dt, unit, bad):
    """In every quarter of a block.  Earlier tokens may be lost, back to the 32 that a tile holds; what stays finite is right."""
    c = Case(dt, [130], 1, 2, 32, 40, unit=unit, seed=32)
    clean = _forward(c)
    for token in (0, 20, 31, 32, 50, 63, 64, 97, 129):
        _held(c, clean, "v", token, 1, bad, token // 32 * 32)


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("dt,unit", [("bf16", True), ("f32", False)])
def test_upstream_gradients_that_are_not_finite(dt, unit, bad):
    """A column of one token: later tokens, other heads, and dv's and ds0's other columns keep their bits."""
    c = Case(dt, [130], 1, 2, 32, 40, unit=unit, seed=33)
    st = _forward(c)[2]
    want = _backward(c, st)
    for token in (0, 20, 31, 32, 50, 63, 64, 97, 129):
        dy = c.dy.clone()
        dy[0, token, 1, 3] = bad
        got = _backward(c, st, dy)
        later = (token // 32 + 1) * 32
        for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
            assert torch.equal(a[:, later:], b[:, later:]), (name, token)
            if name not in ("dq", "dk"):
                assert torch.equal(a[:, :, 0], b[:, :, 0]), (name, token)
        other = torch.arange(40, device="cuda") != 3
        assert torch.equal(got[2][:, :, 1][..., other], want[2][:, :, 1][..., other]), token
        assert torch.equal(got[5][:, :, :, other], want[5][:, :, :, other]), token
        assert not bool(torch.isfinite(got[2][0, :token + 1, 1, 3]).any()), token


# ---- rows of queries and keys, gates ------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_queries_of_any_size(dt):
    """y is linear in a token's query: with rows many powers of two apart, each has the bits that it has alone."""
    c = Case(dt, [130], 2, 4, 40, 48, unit=False, seed=34)
    y0, s0, _ = _forward(c)
    f = torch.from_numpy(np.ldexp(1.0, np.random.default_rng(1).integers(-40, 40, (1, 130, 2, 1)))).float().cuda()
    y, s, _ = _forward(c, q=(c.q * f).to(c.dt))
    assert torch.equal(y, (y0 * f.repeat_interleave(2, 2)).to(c.dt)) and torch.equal(s, s0)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dt,unit", [("bf16", True), ("bf16", False), ("f32", True), ("f32", False)])
def test_one_token_that_is_not_finite(dt, unit, bad):
    """A query spoils its own output only; a key or a gate the tokens from its 32 on."""
    c = Case(dt, [130], 1, 2, 32, 40, unit=unit, seed=35)
    clean = _forward(c)
    for token in (0, 20, 31, 32, 50, 63, 64, 97, 129):
        for name, head in (("q", 0), ("k", 0), ("g", 1), ("b", 1)):
            if name == "g" and bad == -INF:
                continue                                             # a decay to nothing
            _held(c, clean, name, token, head, bad, token // 32 * 32)
        data = c.q.clone()
        data[0, token, 0, 3] = bad
        y = _forward(c, q=data)[0]
        other = torch.arange(130, device="cuda") != token
        assert torch.equal(y[:, other], clean[0][:, other]) and not bool(torch.isfinite(y[:, token]).any()), token


@pytest.mark.parametrize("e", [-80, 95])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_tiny_and_huge_values(dt, e):
    """Results follow the size of values and states, and, for themselves, of upstream gradients: the same bits but for the power of two."""
    c = Case(dt, [130], 2, 4, 40, 48, seed=40, g=lambda r, s: -r.uniform(0, 0.05, s))
    f = 2.0 ** e
    y, s, st = _forward(c)
    want = _backward(c, st)
    s0, ds = c.s0, c.ds
    c.s0 = s0 * f
    y2, s2, st2 = _forward(c, v=c.v * f)
    same = torch.equal(y2, y * f), torch.equal(s2, s * f), torch.equal(st2, st * f)
    assert all(same), same
    for got, power in ((_backward(c, st2, v=c.v * f), (1, 1, 0, 1, 1, 0)), (None, (1, 1, 1, 1, 1, 1))):
        if got is None:
            c.ds = ds * f
            got = _backward(c, st, c.dy * f)
        for what, a, w, n in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), got, want, power):
            same = torch.equal(a, w * f ** n)
            assert same, (what, power)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_huge_queries_beside_tiny_keys(dt):
    """With unit = 0: a factor of 2**120 in the queries and of 2**-80 in the keys, whose products are of an ordinary size."""
    c = Case(dt, [130], 2, 4, 40, 48, unit=False, seed=41, g=lambda r, s: -r.uniform(0, 0.05, s))
    c.s0.zero_()
    (y, s, _), (y2, s2, _) = (_forward(c, q=c.q * 2.0 ** a, k=c.k * 2.0 ** b) for a, b in ((0, -60), (120, -80)))
    same = torch.equal(y2, y * 2.0 ** 100), torch.equal(s2, s * 2.0 ** -20)
    assert all(same), same


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["q", "k"])
def test_tiny_queries_and_keys(dt, name):
    """With unit = 0: 2**-90 times the queries, and 2**-90 beside 2**-60 times the keys, whose products with each other
    are nothing beside 1 either way.  Outputs and gradients follow by powers of two, up to roundings.

    Powers of two end at 2**113.  A row of q or k and what is made of it with values of size 1 stays below that.  In the backward pass
    one operand (products of dy and corrections, times what makes a row of q from numbers of size 2**13) is near 2**-103
    and ends up with an error of 2**-25 2**-113 = 2**-138, less than 2**-30 of its row's largest, where it had 22 bits.  Other fp32 values
    then round the other way, by 2**-24 of a partial sum; no sum has more than 192 terms, 192 2**-24 < 2**-16."""
    c = Case(dt, [130], 2, 4, 40, 48, unit=False, seed=38, g=lambda r, s: -r.uniform(0, 0.05, s))
    c.ds.zero_()
    if name == "k":
        c.s0.zero_()
    got = []
    for e in (0, -90) if name == "q" else (-60, -90):
        x = {name: getattr(c, name) * 2.0 ** e}
        y, s, st = _forward(c, **x)
        got.append((y, s) + _backward(c, st, **x))
    f = 2.0 ** -90 if name == "q" else 2.0 ** -30
    power = (1, 0, 0, 1, 1, 1, 1, 1) if name == "q" else (1, 1, 1, 0, 1, 1, 1, 0)
    for what, a, b, n in zip(("y", "sT", "dq", "dk", "dv", "dg", "dbeta", "ds0"), *got, power):
        w = a.double() * f ** n
        assert float((b.double() - w).abs().max()) <= (2.0 ** -8 if a.dtype == torch.bfloat16 else 2.0 ** -16) * float(w.abs().max()), what
        assert bool((a != 0).any()), what


def _gradients(c, q, k, v, g, b, fq, fk, S, dy, ds):
    """The definition's, with the infinities and NaN that they have."""
    hist = np.zeros((len(q) + 1,) + S.shape)
    hist[0] = S
    with np.errstate(all="ignore"):
        for t in range(len(q)):
            D = np.exp(g[t]) * hist[t]
            hist[t + 1] = D + np.outer(k[t], b[t] * (v[t] - k[t] @ D))
        (dq, dk, dv, dg, db, d0), _ = R.backward(q, k, v, g, b, hist, c.scale, dy, ds)
        return R.through_unit(dq, q, fq, c.unit), R.through_unit(dk, k, fk, c.unit), dv, dg, db, d0


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("dt,unit", [("bf16", True), ("bf16", False), ("f32", True), ("f32", False)])
def test_gradients_beside_one_that_is_not_finite(dt, unit, bad):
    """What stays finite is what the definition leaves finite, and keeps its bits; outside the value's block all of that does."""
    c = Case(dt, [130], 1, 1, 32, 40, unit=unit, seed=36)
    st = _forward(c)[2]
    want = _backward(c, st)
    for token in (0, 20, 31, 32, 50, 63, 64, 97, 129):
        for name in "qkvgb":
            data = dict(zip("qkvgb", (t.clone() for t in c.data())))
            x = data[name]
            x[(0, token, 0) + ((3,) if x.dim() == 4 else ())] = bad
            st2 = _forward(c, **data)[2]
            got = _backward(c, st2, **data)
            c2 = Case.__new__(Case)
            c2.__dict__.update(c.__dict__)
            c2.q, c2.k, c2.v, c2.g, c2.beta = data.values()
            with np.errstate(all="ignore"):
                (_, _, _, _, q, k, v, g, b, fq, fk), = c2.sequences()
            ref = _gradients(c, q, k, v, g, b, fq, fk, _np(c.s0)[0, 0], _np(c.dy)[0, :, 0], _np(c.ds)[0, 0])
            outside = np.arange(130) // 64 != token // 64
            for what, a, w, r in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), got, want, ref):
                at = (name, token, what)
                a, w = _np(a).reshape(r.shape), _np(w).reshape(r.shape)
                fin, held = np.isfinite(r), np.isfinite(a)
                assert not (held & ~fin).any(), at
                assert np.array_equal(a[held], w[held]), at
                if what != "ds0":
                    assert np.array_equal(held[outside], fin[outside]), at
