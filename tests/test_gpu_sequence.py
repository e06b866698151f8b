"""Operators over sequences of tokens on the GPU against seq_reference (float64,
token by token), element by element within the bounds derived there: sizes
around every block edge, odd and narrow channel counts, packed sequences with
empty and single-token ones, column slices, extreme gates, streams, graphs and
rows beyond 2^31 elements.  Buffers are poisoned with NaN first, and what lies
between slices must stay untouched."""
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


def _check(got, ref, err, bf16, label):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    bound = R.tol(ref, err, bf16)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d beyond the bound; first at %s: gpu %r ref %r bound %r"
                             % (label, bad.sum(), bad.size, i, got[i], ref[i], bound[i]))


class Rows:
    """Random rows on the GPU, and as float64: equal sequences, packed ones, or (slices) columns of a
    wider buffer whose other columns hold a marker."""

    def __init__(self, rng, lens, C, dt, packed, slices, rand=None):
        self.n, self.C = sum(lens), C
        a = rng.standard_normal((self.n, C)) if rand is None else rand((self.n, C))
        self.shape = (self.n, C) if packed else (len(lens), lens[0], C)
        self.wide = None
        if slices:
            pad = {True: 8, False: 3}[slices == "aligned"]
            self.wide = torch.full(self.shape[:-1] + (C + 2 * pad,), 77.0, dtype=dt, device="cuda")
            self.t = self.wide[..., pad:pad + C]
            self.t.copy_(_cuda(a, dt).reshape(self.shape))
        else:
            self.t = _cuda(a, dt).reshape(self.shape)
        self.v = _np(self.t).reshape(self.n, C)

    def untouched(self):
        if self.wide is not None:
            w = self.wide.float()
            out = (w != 77.0).sum() - (self.t.float() != 77.0).sum()
            assert int(out) == 0, "wrote outside its columns"


def _out(rng, lens, C, dt, packed, slices):
    o = Rows(rng, lens, C, dt, packed, slices, rand=np.zeros)
    o.t.fill_(float("nan"))
    return o


def _batch(lens, packed):
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    kw = {}
    if packed:
        kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_len=max(lens))
    return off, kw


CASES = [
    # dtype, lengths, C, K, silu, packed, slices
    ("bf16", [1], 1, 1, True, False, None),
    ("bf16", [1, 1, 1], 8, 4, True, False, None),
    ("bf16", [2] * 3, 24, 8, False, False, None),
    ("bf16", [33] * 2, 64, 4, True, False, "aligned"),
    ("bf16", [130], 72, 3, True, False, None),
    ("bf16", [65, 0, 1, 3, 200, 0], 136, 4, True, True, None),
    ("bf16", [0, 0], 16, 4, True, True, None),
    ("bf16", [5, 300, 2], 37, 5, False, True, "odd"),
    ("bf16", [257] * 2, 520, 4, False, False, None),
    ("bf16", [70] * 2, 640, 6, True, False, "odd"),
    ("f32", [1], 1, 2, False, False, None),
    ("f32", [63, 64, 65, 0, 1], 33, 3, True, True, None),
    ("f32", [129] * 3, 260, 4, True, False, "aligned"),
    ("f32", [40, 2, 7], 12, 7, False, True, "odd"),
    ("f32", [300], 100, 4, True, False, None),
]


@pytest.mark.parametrize("carried", [True, False])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_causal_conv(case, carried):
    dtype, lens, C, K, silu, packed, slices = case
    dt, half = DT[dtype], dtype == "bf16"
    rng = np.random.default_rng(C * 7 + K)
    off, kw = _batch(lens, packed)
    x, dy = (Rows(rng, lens, C, dt, packed, slices) for _ in range(2))
    w, bias = _cuda(rng.standard_normal((C, K)), dt), _cuda(rng.uniform(-1, 1, C))
    state = _cuda(rng.standard_normal((len(lens), K - 1, C)), dt) if carried else None
    wv, bv = _np(w), _np(bias)
    sv = _np(state) if carried else np.zeros((len(lens), K - 1, C))
    y, dx = (_out(rng, lens, C, dt, packed, slices) for _ in range(2))
    got, end = B.causal_conv(x.t, w, bias, silu=silu, state=state, with_state=True, out=y.t, **kw)
    gdx, gdw, gdb, gds = B.causal_conv_backward(x.t, w, dy.t, bias, silu=silu, state=state, out=dx.t, **kw)
    torch.cuda.synchronize()
    y.untouched(), dx.untouched()
    yv, dxv = _np(got).reshape(-1, C), _np(gdx).reshape(-1, C)
    dw, edw, db, edb = np.zeros((C, K)), np.zeros((C, K)), np.zeros(C), np.zeros(C)
    for b, n in enumerate(lens):
        rows = slice(off[b], off[b] + n)
        ref, err, after, _ = R.conv(x.v[rows], wv, bv, sv[b], silu)
        _check(yv[rows], ref, err, half, "y of sequence %d" % b)
        assert np.array_equal(_np(end)[b], after)
        g, e = R.conv_grad(x.v[rows], wv, bv, sv[b], silu, dy.v[rows])
        _check(dxv[rows], g[0], e[0], half, "dx of sequence %d" % b)
        if carried:
            _check(_np(gds)[b], g[3], e[3], half, "dstate of sequence %d" % b)
        dw, edw, db, edb = dw + g[1], edw + e[1], db + g[2], edb + e[2]
    assert carried or gds is None
    # adding the sequences and the ranges of tokens: a rounding for each
    more = (sum(lens) // 32 + len(lens) + 8) * R.U
    _check(gdw, dw, edw + more * edw / R.U / 8, False, "dw")
    _check(gdb, db, edb + more * edb / R.U / 8, False, "db")


def test_causal_conv_without_bias_and_continued():
    """No bias is a zero bias; a sequence in two calls with the state between them is the sequence in one."""
    rng = np.random.default_rng(3)
    x, w = _cuda(rng.standard_normal((2, 50, 48)), torch.bfloat16), _cuda(rng.standard_normal((48, 4)), torch.bfloat16)
    whole, end = B.causal_conv(x, w, silu=True, with_state=True)
    zero = B.causal_conv(x, w, torch.zeros(48, device="cuda"), silu=True)
    assert torch.equal(whole, zero)
    a, mid = B.causal_conv(x[:, :2].contiguous(), w, silu=True, with_state=True)
    b, last = B.causal_conv(x[:, 2:].contiguous(), w, silu=True, state=mid, with_state=True)
    assert torch.equal(torch.cat([a, b], 1), whole) and torch.equal(last, end)
    # and token by token
    st = torch.zeros(2, 3, 48, dtype=torch.bfloat16, device="cuda")
    ys = [B.causal_conv_step(x[:, t], w, st, silu=True) for t in range(50)]
    assert torch.equal(torch.stack(ys, 1), whole) and torch.equal(st, end)


@pytest.mark.parametrize("dtype,n,C,K", [("bf16", 1, 1, 1), ("bf16", 3, 37, 4), ("bf16", 64, 256, 4), ("f32", 5, 130, 8), ("f32", 2, 64, 2)])
def test_causal_conv_step(dtype, n, C, K):
    dt, rng = DT[dtype], np.random.default_rng(C)
    x, w, bias = _cuda(rng.standard_normal((n, C)), dt), _cuda(rng.standard_normal((C, K)), dt), _cuda(rng.uniform(-1, 1, C))
    st = _cuda(rng.standard_normal((n, K - 1, C)), dt)
    refs = [R.conv(_np(x)[b:b + 1], _np(w), _np(bias), _np(st)[b], True) for b in range(n)]
    wide = torch.full((n, C + 5), 77.0, dtype=dt, device="cuda")
    y = B.causal_conv_step(x, w, st, bias, silu=True, out=wide[:, 2:2 + C])
    for b, (ref, err, after, _) in enumerate(refs):
        _check(_np(y)[b:b + 1], ref, err, dtype == "bf16", "y")
        assert np.array_equal(_np(st)[b], after)
    assert bool((wide[:, :2] == 77).all()) and bool((wide[:, 2 + C:] == 77).all())


# ---- the recurrence ---------------------------------------------------------------

SCANS = [
    # dtype, lengths, C, packed, slices
    ("bf16", [1], 1, False, None),
    ("bf16", [1] * 3, 8, False, None),
    ("bf16", [63] * 2, 64, False, None),
    ("bf16", [64] * 2, 130, False, None),
    ("bf16", [65], 128, False, "aligned"),
    ("bf16", [200] * 2, 129, False, "odd"),
    ("bf16", [300, 0, 1, 64, 127, 0, 129], 96, True, None),
    ("bf16", [0], 16, True, None),
    ("bf16", [700], 33, False, None),
    ("bf16", [1100] * 2, 256, False, None),
    ("f32", [1], 1, False, None),
    ("f32", [128] * 2, 63, False, None),
    ("f32", [129, 1, 0, 400, 63], 65, True, "odd"),
    ("f32", [520] * 2, 192, False, "aligned"),
]


def _scan_inputs(rng, lens, C, dt, packed, slices):
    x, g, u, dy = (Rows(rng, lens, C, dt, packed, slices) for _ in range(4))
    decay = _cuda(rng.uniform(-7, -1, C))
    h0, dh = (_cuda(rng.standard_normal((len(lens), C))) for _ in range(2))
    return x, g, u, dy, decay, h0, dh


@pytest.mark.parametrize("carried", [True, False])
@pytest.mark.parametrize("case", SCANS, ids=[str(i) for i in range(len(SCANS))])
def test_gated_scan(case, carried):
    dtype, lens, C, packed, slices = case
    dt, half = DT[dtype], dtype == "bf16"
    rng = np.random.default_rng(C * 11 + len(lens))
    off, kw = _batch(lens, packed)
    x, g, u, dy, decay, h0, dh = _scan_inputs(rng, lens, C, dt, packed, slices)
    y, dx, dg, di = (_out(rng, lens, C, dt, packed, slices) for _ in range(4))
    got, hT, states = B.gated_scan(x.t, g.t, u.t, decay, h0=h0 if carried else None, with_states=True, out=y.t, **kw)
    plain, hT2 = B.gated_scan(x.t, g.t, u.t, decay, h0=h0 if carried else None, **kw)
    grads = B.gated_scan_backward(x.t, g.t, u.t, decay, dy.t, states, dh=dh if carried else None,
                                  out=(dx.t, dg.t, di.t), **kw)
    torch.cuda.synchronize()
    for o in (y, dx, dg, di):
        o.untouched()
    assert torch.equal(plain, got) and torch.equal(hT, hT2), "saving the states changed the result"
    yv, gv = _np(got).reshape(-1, C), [_np(t).reshape(-1, C) for t in grads[:3]]
    dd, edd = np.zeros(C), np.zeros(C)
    dv = _np(decay)
    for b, n in enumerate(lens):
        rows = slice(off[b], off[b] + n)
        args = (x.v[rows], g.v[rows], u.v[rows], dv, 8.0, _np(h0)[b] if carried else np.zeros(C))
        h, e, before, eb = R.scan(*args)
        _check(yv[rows], h, e, half, "y of sequence %d" % b)
        _check(_np(hT)[b], h[-1] if n else args[-1], e[-1] if n else np.zeros(C), False, "hT")
        for k in range(-(-n // 64)):
            _check(_np(states)[b, k], before[64 * k], eb[64 * k], False, "states")
        ref, err = R.scan_grad(*args, dy.v[rows], _np(dh)[b] if carried else np.zeros(C))
        for name, a, r, q in zip(("dx", "dgate", "dinp"), gv, ref, err):
            _check(a[rows], r, q, half, "%s of sequence %d" % (name, b))
        _check(_np(grads[4])[b], ref[4], err[4], False, "dh0")
        dd, edd = dd + ref[3], edd + err[3]
    _check(grads[3], dd, edd * (2 + (sum(lens) // 64 + len(lens)) / 8), False, "ddecay")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_scan_extremes(dtype):
    """Gates of +-inf and +-100, decays from -40 (a = 1 to the last bit) to 40 (a = 0): the reference's
    values, and no NaN anywhere."""
    dt, rng = DT[dtype], np.random.default_rng(5)
    L, C = 150, 80
    g = rng.standard_normal((1, L, C)) * 30
    u = rng.standard_normal((1, L, C)) * 30
    g[0, ::7], g[0, 3::11] = np.inf, -np.inf
    u[0, ::5], u[0, 4::13] = -np.inf, np.inf
    x, dy = rng.standard_normal((1, L, C)), rng.standard_normal((1, L, C))
    decay = np.linspace(-40, 40, C)
    X, G, I, DY, D = _cuda(x, dt), _cuda(g, dt), _cuda(u, dt), _cuda(dy, dt), _cuda(decay)
    h0 = rng.standard_normal((1, C))
    y, hT, st = B.gated_scan(X, G, I, D, h0=_cuda(h0), with_states=True)
    grads = B.gated_scan_backward(X, G, I, D, DY, st)
    args = (_np(X)[0], _np(G)[0], _np(I)[0], _np(D), 8.0, _np(_cuda(h0))[0])
    h, e, _, _ = R.scan(*args)
    _check(_np(y)[0], h, e, dtype == "bf16", "y")
    for t in grads:
        assert bool(torch.isfinite(t).all())
    # dx and dinp have no 1/m: they hold to the bound as well
    ref, err = R.scan_grad(*args, _np(DY)[0], np.zeros(C))
    tiny = 1e-18 * (1 + np.abs(_np(DY)[0]).max()) * L      # m is clamped at 2^-63 where a = 1
    _check(_np(grads[0])[0], ref[0], err[0] + tiny, dtype == "bf16", "dx")
    _check(_np(grads[2])[0], ref[2], err[2] + tiny * np.abs(x).max(), dtype == "bf16", "dinp")


def test_gated_scan_nan_stays_in_its_sequence_and_channel():
    rng = np.random.default_rng(9)
    lens, C = [100, 70, 130], 40
    off, kw = _batch(lens, True)
    x, g, u, dy, decay, h0, dh = _scan_inputs(rng, lens, C, torch.bfloat16, True, None)
    clean, _ = B.gated_scan(x.t, g.t, u.t, decay, h0=h0, **kw)
    x.t[off[1] + 10, 7] = float("nan")
    y, hT, st = B.gated_scan(x.t, g.t, u.t, decay, h0=h0, with_states=True, **kw)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[off[1] + 10:off[2], 7] = True
    assert torch.equal(torch.isnan(y), hit) and torch.equal(y[~hit], clean[~hit])
    dx = B.gated_scan_backward(x.t, g.t, u.t, decay, dy.t, st, dh=dh, **kw)[0]
    assert not bool(torch.isnan(dx[:off[1]]).any()) and not bool(torch.isnan(dx[off[2]:]).any())


@pytest.mark.parametrize("L", [1, 65, 300])
def test_gated_scan_gradient_against_differences(L):
    """float32 gradients against central differences of the float64 definition along random directions.
    The gradients' own bound (scan_grad) times the direction, and 1e-6 of the terms for the difference."""
    rng = np.random.default_rng(L)
    C = 20
    x, g, u, dy = (rng.standard_normal((L, C)) for _ in range(4))
    decay, h0, dh = rng.uniform(-5, -1, C), rng.standard_normal(C), rng.standard_normal(C)
    x, g, u, dy, decay, h0, dh = (np.float32(v).astype(np.float64) for v in (x, g, u, dy, decay, h0, dh))
    one = lambda v: _cuda(v)[None].contiguous()
    _, _, st = B.gated_scan(one(x), one(g), one(u), _cuda(decay), h0=one(h0), with_states=True)
    got = B.gated_scan_backward(one(x), one(g), one(u), _cuda(decay), one(dy), st, dh=one(dh))
    got = [_np(t).reshape(v.shape) for t, v in zip(got, (x, g, u, decay, h0))]
    err = R.scan_grad(x, g, u, decay, 8.0, h0, dy, dh)[1]

    def f(*a):
        h = R.scan(a[0], a[1], a[2], a[3], 8.0, a[4])[0]
        return (h * dy).sum() + (h[-1] * dh).sum()

    args, eps = [x, g, u, decay, h0], 1e-5
    for i in range(5):
        d = rng.standard_normal(args[i].shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + eps * d, args[i] - eps * d
        num, ana = (f(*up) - f(*dn)) / (2 * eps), (got[i] * d).sum()
        bound = (R.tol(got[i], err[i], False) * np.abs(d)).sum() + 1e-6 * (np.abs(got[i] * d).sum() + 1)
        assert abs(num - ana) <= bound, (i, num, ana, bound)


@pytest.mark.parametrize("K,silu", [(4, True), (3, False)])
def test_causal_conv_gradient_against_differences(K, silu):
    rng = np.random.default_rng(K)
    L, C = 70, 12
    x, w, b, st, dy = (np.float32(v).astype(np.float64) for v in (
        rng.standard_normal((L, C)), rng.standard_normal((C, K)), rng.standard_normal(C), rng.standard_normal((K - 1, C)),
        rng.standard_normal((L, C))))
    got = B.causal_conv_backward(_cuda(x)[None], _cuda(w), _cuda(dy)[None], _cuda(b), silu=silu, state=_cuda(st)[None])
    got = [_np(t).reshape(v.shape) for t, v in zip(got, (x, w, b, st))]
    err = R.conv_grad(x, w, b, st, silu, dy)[1]
    args, eps = [x, w, b, st], 1e-5
    for i in range(4):
        d = rng.standard_normal(args[i].shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + eps * d, args[i] - eps * d
        num = ((R.conv(*up, silu)[0] - R.conv(*dn, silu)[0]) * dy).sum() / (2 * eps)
        ana = (got[i] * d).sum()
        bound = (R.tol(got[i], err[i], False) * np.abs(d)).sum() + 1e-6 * (np.abs(got[i] * d).sum() + 1)
        assert abs(num - ana) <= bound, (i, num, ana, bound)


@pytest.mark.parametrize("dtype,n,C", [("bf16", 1, 1), ("bf16", 3, 37), ("bf16", 64, 256), ("f32", 5, 130)])
def test_gated_scan_step(dtype, n, C):
    """One token at a time gives what the definition gives, from a state or on from a prompt."""
    dt, rng = DT[dtype], np.random.default_rng(C + n)
    x, g, u = (_cuda(rng.standard_normal((n, 9, C)), dt) for _ in range(3))
    decay, h = _cuda(rng.uniform(-7, -1, C)), _cuda(rng.standard_normal((n, C)))
    h0 = _np(h)
    ys = []
    for t in range(9):
        wide = torch.full((n, C + 5), 77.0, dtype=dt, device="cuda")
        ys.append(B.gated_scan_step(x[:, t], g[:, t], u[:, t], decay, h, out=wide[:, 3:3 + C]))
        assert bool((wide[:, :3] == 77).all()) and bool((wide[:, 3 + C:] == 77).all())
    for b in range(n):
        ref, err, _, _ = R.scan(_np(x)[b], _np(g)[b], _np(u)[b], _np(decay), 8.0, h0[b])
        _check(np.stack([_np(y)[b] for y in ys]), ref, err, dtype == "bf16", "y")
        _check(_np(h)[b], ref[-1], err[-1], False, "h")


def test_packed_equals_separate_and_is_reproducible():
    """A packed sequence gives the bits that it gives alone, however often it is run."""
    rng = np.random.default_rng(21)
    lens, C = [513, 0, 64, 1, 300], 200
    off, kw = _batch(lens, True)
    x, g, u, dy, decay, h0, dh = _scan_inputs(rng, lens, C, torch.bfloat16, True, None)
    first = None
    for _ in range(5):
        y, hT, st = B.gated_scan(x.t, g.t, u.t, decay, h0=h0, with_states=True, **kw)
        out = (y, hT) + tuple(B.gated_scan_backward(x.t, g.t, u.t, decay, dy.t, st, dh=dh, **kw))
        first = out if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(out, first))
    for b, n in enumerate(lens):
        if n:
            cut = lambda r: r.t[off[b]:off[b] + n][None].contiguous()
            y1, h1, s1 = B.gated_scan(cut(x), cut(g), cut(u), decay, h0=h0[b:b + 1].contiguous(), with_states=True)
            assert torch.equal(y1[0], first[0][off[b]:off[b] + n]) and torch.equal(h1[0], first[1][b])
            g1 = B.gated_scan_backward(cut(x), cut(g), cut(u), decay, cut(dy), s1, dh=dh[b:b + 1].contiguous())
            for a, q in zip(g1[:3], first[2:5]):
                assert torch.equal(a[0], q[off[b]:off[b] + n])


def test_bad_offsets_are_clamped():
    """Offsets past the tensor or decreasing, and sequences longer than max_len: rows outside are neither
    read nor written, and the rest is computed."""
    rng = np.random.default_rng(2)
    C, n = 32, 100
    x, g, u = (_cuda(rng.standard_normal((n, C)), torch.bfloat16) for _ in range(3))
    w, decay = _cuda(rng.standard_normal((C, 4)), torch.bfloat16), _cuda(rng.uniform(-5, -1, C))
    off = torch.tensor([-5, 40, 30, 5000], dtype=torch.int32, device="cuda")
    y = torch.full((n, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.causal_conv(x, w, offsets=off, max_len=50, out=y)
    want = B.causal_conv(x[:40][None].contiguous(), w)[0]
    tail = B.causal_conv(x[30:80][None].contiguous(), w)[0]
    assert torch.equal(y[:30], want[:30]) and torch.equal(y[40:80], tail[10:]) and bool(torch.isnan(y[80:]).all())
    y.fill_(float("nan"))
    B.gated_scan(x, g, u, decay, offsets=off, max_len=50, out=y)
    assert bool(torch.isfinite(y[:80]).all()) and bool(torch.isnan(y[80:]).all())


def test_other_stream_and_graph():
    """On a stream of its own, and captured in a graph: every replay equals the eager result."""
    rng = np.random.default_rng(8)
    lens, C = [700] * 2, 256
    x, g, u, dy, decay, h0, dh = _scan_inputs(rng, lens, C, torch.bfloat16, False, None)
    w = _cuda(rng.standard_normal((C, 4)), torch.bfloat16)

    def work():
        c = B.causal_conv(x.t, w, silu=True)
        y, hT, st = B.gated_scan(c, g.t, u.t, decay, h0=h0, with_states=True)
        dx, dg, di, dd, d0 = B.gated_scan_backward(c, g.t, u.t, decay, dy.t, st, dh=dh)
        dx2, dw, db, _ = B.causal_conv_backward(x.t, w, dx, silu=True)
        return [y, hT, dg, di, dd, d0, dx2, dw, db]

    want = [t.clone() for t in work()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = work()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), "replay %d" % i
        assert all(torch.equal(a, b) for a, b in zip(work(), want)), "eager after replay %d" % i


def test_rows_beyond_32_bit_offsets():
    """70000 rows of a 32768-wide buffer hold more than 2^31 elements: slices at its end are exact there."""
    T, ld, C = 70000, 32768, 16
    buf = torch.empty((1, T, ld), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(4)
    cols = [buf[..., i * C:(i + 1) * C] for i in range(4)] + [buf[..., ld - (i + 1) * C:ld - i * C] for i in range(4)]
    vals = [rng.standard_normal((1, T, C)) for _ in range(4)]
    for c, v in zip(cols, vals):
        c.copy_(_cuda(v, torch.bfloat16))
    x, g, u, dy = cols[:4]
    decay = _cuda(rng.uniform(-5, -1, C))
    dense = [c.contiguous() for c in (x, g, u, dy)]
    w = _cuda(rng.standard_normal((C, 4)), torch.bfloat16)
    y, hT, st = B.gated_scan(x, g, u, decay, with_states=True, out=cols[4])
    y2, hT2, st2 = B.gated_scan(dense[0], dense[1], dense[2], decay, with_states=True)
    assert torch.equal(y, y2) and torch.equal(hT, hT2) and torch.equal(st, st2)
    a = B.gated_scan_backward(x, g, u, decay, dy, st, out=tuple(cols[5:8]))
    b = B.gated_scan_backward(*dense[:3], decay, dense[3], st2)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    c = B.causal_conv(x, w, out=cols[4])
    assert torch.equal(c, B.causal_conv(dense[0], w))
    ref, err, _, _ = R.scan(_np(dense[0])[0, -2000:], _np(dense[1])[0, -2000:], _np(dense[2])[0, -2000:], _np(decay), 8.0, np.zeros(C))
    _check(_np(y2)[0, -100:], ref[-100:], err[-100:] + 1e-3 * np.abs(ref[-100:]), True, "y far from the start")


def test_helpers_refuse_wrong_tensors_and_overlap():
    x = torch.zeros(2, 70, 24, dtype=torch.bfloat16, device="cuda")
    w, d = torch.zeros(24, 4, dtype=torch.bfloat16, device="cuda"), torch.zeros(24, device="cuda")
    with pytest.raises(B.ConvError):
        B.causal_conv(x, w, out=x)
    with pytest.raises(ValueError):
        B.causal_conv(x.transpose(1, 2), w)
    with pytest.raises(TypeError):
        B.causal_conv(x, w.float())
    with pytest.raises(ValueError):
        B.causal_conv(x, w, state=torch.zeros(2, 4, 24, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        B.gated_scan(x, x.float(), x, d)
    with pytest.raises(ValueError):
        B.gated_scan(x, x[:1], x, d)
    with pytest.raises(TypeError):
        B.gated_scan_step(x[:, 0], x[:, 0], x[:, 0], d, torch.zeros(2, 24, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(B.ConvError):
        B.gated_scan(x, x, x, d, scale=float("nan"))
    with pytest.raises(B.ConvError):
        B.causal_conv(x, torch.zeros(24, 9, dtype=torch.bfloat16, device="cuda"))
    assert B.causal_conv(x[:, :0], w).shape == (2, 0, 24)
    y, hT = B.gated_scan(x[:, :0], x[:, :0], x[:, :0], d, h0=torch.ones(2, 24, device="cuda"))
    assert y.shape == (2, 0, 24) and bool((hT == 1).all())


def test_many_packed_sequences():
    """150 packed sequences of 0 to 300 tokens that do not start at row 0 nor end at the last: rows outside
    stay untouched, each sequence gives the bits that it gives alone."""
    rng = np.random.default_rng(31)
    lens = [int(v) for v in rng.integers(0, 300, 150)]
    lens[3] = lens[70] = lens[149] = 0
    C, lead, tail = 24, 77, 300
    off = lead + np.concatenate([[0], np.cumsum(lens)])
    n = int(off[-1]) + tail
    x, g, u, dy = (_cuda(rng.standard_normal((n, C)), torch.bfloat16) for _ in range(4))
    w, decay, h0 = _cuda(rng.standard_normal((C, 4)), torch.bfloat16), _cuda(rng.uniform(-5, -1, C)), _cuda(rng.standard_normal((150, C)))
    kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_len=max(lens))
    out = [torch.full((n, C), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    B.causal_conv(x, w, silu=True, out=out[0], **kw)
    _, dw, db, _ = B.causal_conv_backward(x, w, dy, silu=True, out=out[1], **kw)
    _, hT, st = B.gated_scan(x, g, u, decay, h0=h0, with_states=True, out=out[2], **kw)
    _, _, _, dd, dh0 = B.gated_scan_backward(x, g, u, decay, dy, st, out=tuple(out[3:]), **kw)
    for o in out:
        assert bool(torch.isnan(o[:lead]).all()) and bool(torch.isnan(o[int(off[-1]):]).all())
    sums = [torch.zeros_like(t, dtype=torch.float64) for t in (dw, db, dd)]
    for b in range(150):
        if not lens[b]:
            assert torch.equal(hT[b], h0[b]) and not bool(dh0[b].any())
            continue
        r = slice(int(off[b]), int(off[b + 1]))
        one = [t[r][None].contiguous() for t in (x, g, u, dy)]
        cdx, cdw, cdb, _ = B.causal_conv_backward(one[0], w, one[3], silu=True)
        y1, h1, s1 = B.gated_scan(*one[:3], decay, h0=h0[b:b + 1].contiguous(), with_states=True)
        g1 = B.gated_scan_backward(*one[:3], decay, one[3], s1)
        want = [B.causal_conv(one[0], w, silu=True), cdx, y1, *g1[:3]]
        assert all(torch.equal(o[r], q[0]) for o, q in zip(out, want)), b
        assert torch.equal(hT[b], h1[0]) and torch.equal(dh0[b], g1[4][0])
        for t, q in zip(sums, (cdw, cdb, g1[3])):
            t += q.double()
    for t, q in zip((dw, db, dd), sums):
        assert float((t.double() - q).abs().max()) <= 1e-5 * float(q.abs().max())


@pytest.mark.parametrize("off", [[0, 700, 300, 1500], [900, 100, 1400, 20], [1500, 0, 0, 0], [-3, 2000, 5, 1 << 30]])
def test_descending_offsets_end_within_the_rows(off):
    """Which rows are computed is unspecified; that the calls end, and write no row outside, is not."""
    rng = np.random.default_rng(2)
    C, n = 32, 1500
    buf = torch.full((n + 200, C), 5.0, dtype=torch.bfloat16, device="cuda")
    x, g, u, dy = (_cuda(rng.standard_normal((n, C)), torch.bfloat16) for _ in range(4))
    decay, w = _cuda(rng.uniform(-5, -1, C)), _cuda(rng.standard_normal((C, 4)), torch.bfloat16)
    kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_len=1500)
    y = buf[100:100 + n]
    B.causal_conv(x, w, out=y, **kw)
    B.causal_conv_backward(x, w, dy, out=y, **kw)
    _, _, st = B.gated_scan(x, g, u, decay, with_states=True, out=y, **kw)
    B.gated_scan_backward(x, g, u, decay, dy, torch.zeros_like(st), **kw)
    torch.cuda.synchronize()
    assert bool((buf[:100] == 5).all()) and bool((buf[100 + n:] == 5).all())


def test_nan_of_all_ones():
    """A float32 NaN whose bits are all ones passes from chunk to chunk like any other."""
    T, C = 700, 3
    x = torch.zeros(1, T, C, device="cuda")
    x.view(torch.int32)[0, 130, 1] = -1
    g = torch.zeros(1, T, C, device="cuda")
    y, hT, st = B.gated_scan(x, g, g, torch.zeros(C, device="cuda"), with_states=True)
    hit = torch.zeros(1, T, C, dtype=torch.bool, device="cuda")
    hit[0, 130:, 1] = True
    assert torch.equal(torch.isnan(y), hit)
    x.view(torch.int32)[0, 130, 1] = 0
    y, hT, st = B.gated_scan(x, g, g, torch.zeros(C, device="cuda"), with_states=True)
    dy = torch.zeros(1, T, C, device="cuda")
    dy.view(torch.int32)[0, 600, 2] = -1
    dx = B.gated_scan_backward(x, g, g, torch.zeros(C, device="cuda"), dy, st)[0]
    hit = torch.zeros(1, T, C, dtype=torch.bool, device="cuda")
    hit[0, :601, 2] = True
    assert torch.equal(torch.isnan(dx), hit)


@pytest.mark.parametrize("B_", [65, 4097, 5000])
def test_thousands_of_packed_sequences(B_):
    """Packed sequences, many of them empty, give the rows of the same sequences in an equal batch with
    arbitrary rows behind their ends: bit for bit, forward and backward."""
    rng = np.random.default_rng(B_)
    lens = rng.integers(0, 200, B_) * (rng.random(B_) < 0.7)
    lens[-1] = 199
    T, C = int(lens.max()), 8
    x, g, u, dy = (_cuda(rng.standard_normal((B_, T, C)), torch.bfloat16) for _ in range(4))
    w, decay = _cuda(rng.standard_normal((C, 4)), torch.bfloat16), _cuda(rng.uniform(-5, -1, C))
    live = torch.arange(T, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None]
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    kw = dict(offsets=off, max_len=T)
    px, pg, pu, pd = (t[live] for t in (x, g, u, dy))
    assert torch.equal(B.causal_conv(px, w, silu=True, **kw), B.causal_conv(x, w, silu=True)[live])
    y, hT, st = B.gated_scan(px, pg, pu, decay, with_states=True, **kw)
    want, _, st2 = B.gated_scan(x, g, u, decay, with_states=True)
    assert torch.equal(y, want[live])
    # a gradient of zero behind the ends is no gradient
    grads = B.gated_scan_backward(px, pg, pu, decay, pd, st, **kw)
    ref = B.gated_scan_backward(x, g, u, decay, dy * live[..., None], st2)
    for a, b in zip(grads[:3], ref[:3]):
        assert torch.equal(a, b[live])
    dx = B.causal_conv_backward(px, w, pd, silu=True, **kw)[0]
    assert torch.equal(dx, B.causal_conv_backward(x, w, dy * live[..., None], silu=True)[0][live])


def test_workspaces_of_other_memory_are_refused():
    """A workspace has to be the GPU's, dense and large enough; one that is gives the same bits as none."""
    rng = np.random.default_rng(1)
    x, g, u, dy = (_cuda(rng.standard_normal((2, 300, 32)), torch.bfloat16) for _ in range(4))
    decay = _cuda(rng.uniform(-5, -1, 32))
    y, hT, st = B.gated_scan(x, g, u, decay, with_states=True)
    want = B.gated_scan_backward(x, g, u, decay, dy, st)
    seq = B.make_seq(x)
    for n, call in ((B.conv_scan_fwd_workspace_bytes(seq), lambda w: B.gated_scan(x, g, u, decay, with_states=True, workspace=w)),
                    (B.conv_scan_bwd_workspace_bytes(seq), lambda w: B.gated_scan_backward(x, g, u, decay, dy, st, workspace=w))):
        for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)):
            with pytest.raises(ValueError):
                call(bad)
        with pytest.raises(B.ConvError):
            call(torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
        got = call(torch.empty(n, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(got, (y, hT, st) if len(got) == 3 else want))
    # checked on the host only: no call is made with it
    with pytest.raises(ValueError):
        B.gated_scan(x, g, u, decay.cpu())
    with pytest.raises(ValueError):
        B.gated_scan(x, g.cpu(), u, decay)


def test_long_sequences_of_one_channel():
    """65 sequences of 2^22 tokens: 65 x 65536 chunks, near what a launch can hold.  Each gives the bits
    that it gives alone."""
    n, T = 65, 1 << 22
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, g, u, dy = (torch.empty(n, T, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(4))
    decay = torch.tensor([-4.0], device="cuda")
    y, hT, st = B.gated_scan(x, g, u, decay, with_states=True)
    grads = B.gated_scan_backward(x, g, u, decay, dy, st)
    for b in (0, 31, 64):
        one = [t[b:b + 1] for t in (x, g, u, dy)]
        y1, h1, s1 = B.gated_scan(*one[:3], decay, with_states=True)
        assert torch.equal(y1[0], y[b]) and torch.equal(h1[0], hT[b]) and torch.equal(s1[0], st[b])
        alone = B.gated_scan_backward(*one[:3], decay, one[3], s1)
        for p, q in zip(alone[:3], grads[:3]):
            assert torch.equal(p[0], q[b])


def test_packed_rows_of_no_tokens():
    """max_len = 0: every sequence is empty, whatever rows there are; all gradients are there."""
    x = torch.ones(50, 8, dtype=torch.bfloat16, device="cuda")
    kw = dict(offsets=torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda"), max_len=0)
    decay, h0 = torch.zeros(8, device="cuda"), torch.full((2, 8), 3.0, device="cuda")
    _, hT, st = B.gated_scan(x, x, x, decay, h0=h0, with_states=True, **kw)
    assert torch.equal(hT, h0) and st.shape == (2, 0, 8)
    grads = B.gated_scan_backward(x, x, x, decay, x, st, dh=h0, **kw)
    assert not bool(grads[3].any()) and torch.equal(grads[4], h0)


# ---- rows that no sequence holds ---------------------------------------------------

GAPS = [
    # offsets, rows, max_len
    ([0, 40, 40, 100], 100, 60),                    # none
    ([7, 40, 40, 100], 131, 60),                    # in front and behind
    ([0, 300, 300, 1000], 2300, 200),               # and past max_len
    ([0, 0, 0], 70, 1),                             # all rows
    ([0, 0], 500, 0),
    ([64, 64 + 900], 64 * 40, 900),
    ([3] + [3 + 5 * i for i in range(1, 200)], 1500, 5),
    ([3] + [3 + 5 * i for i in range(1, 200)], 1500, 2),
]


def _held(off, rows, max_len):
    on = np.zeros(rows, dtype=bool)
    for a, b in zip(off, off[1:]):
        on[a:min(b, a + max_len)] = True
    return torch.from_numpy(on).cuda()


def _dirty(n):
    """Memory that the next allocations may get: all NaN."""
    t = [torch.full((n,), float("nan"), device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("dtype,C", [("bf16", 1), ("bf16", 13), ("bf16", 600), ("f32", 3), ("f32", 132)])
@pytest.mark.parametrize("case", range(len(GAPS)))
def test_rows_of_no_sequence_are_zero(case, dtype, C):
    """Without an out, rows that no sequence holds are zeros, in results and in gradients; in a given out
    they stay as they are, and rows that a sequence holds are the same either way."""
    off, rows, max_len = GAPS[case]
    dt, rng = DT[dtype], np.random.default_rng(case)
    on = _held(off, rows, max_len)
    kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_len=max_len)
    x, g, u, dy = (_cuda(rng.standard_normal((rows, C)), dt) for _ in range(4))
    for t in (x, g, u, dy):
        t[~on] = float("nan")
    w, decay = _cuda(rng.standard_normal((C, 4)), dt), _cuda(rng.uniform(-5, -1, C))

    def both(call, n):
        given = [torch.full((rows, 3 * C + 2), 5.0, dtype=dt, device="cuda")[:, 1 + C:1 + 2 * C] for _ in range(n)]
        _dirty(rows * C)
        new = call(None)
        call(tuple(given) if n > 1 else given[0])
        for a, b in zip(new if n > 1 else [new], given):
            assert bool((a[~on] == 0).all()) and bool((b[~on] == 5).all())
            assert torch.equal(a[on], b[on]) and not bool(torch.isnan(a).any())

    both(lambda o: B.causal_conv(x, w, silu=True, out=o, **kw), 1)
    both(lambda o: B.causal_conv_backward(x, w, dy, silu=True, out=o, **kw)[0], 1)
    both(lambda o: B.gated_scan(x, g, u, decay, out=o, **kw)[0], 1)
    _, _, st = B.gated_scan(x, g, u, decay, with_states=True, **kw)
    both(lambda o: B.gated_scan_backward(x, g, u, decay, dy, st, out=o, **kw)[:3], 3)
    one = torch.full((rows, C), 5.0, dtype=dt, device="cuda")
    _dirty(rows * C)
    mixed = B.gated_scan_backward(x, g, u, decay, dy, st, out=(None, one, None), **kw)
    assert bool((mixed[0][~on] == 0).all()) and bool((one[~on] == 5).all()) and bool((mixed[2][~on] == 0).all())


def test_rows_of_no_sequence_in_a_graph():
    """A captured call fills them at every replay."""
    rng = np.random.default_rng(1)
    off, rows = [5, 300, 420], 700
    on = _held(off, rows, 250)
    kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_len=250)
    x, g, u = (_cuda(rng.standard_normal((rows, 72)), torch.bfloat16) for _ in range(3))
    w, decay = _cuda(rng.standard_normal((72, 4)), torch.bfloat16), _cuda(rng.uniform(-5, -1, 72))
    run = lambda: (B.causal_conv(x, w, **kw), B.gated_scan(x, g, u, decay, **kw)[0])
    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b) and bool((a[~on] == 0).all())
        run()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_scan_extreme_gradients(dtype):
    """All gradients at gates of +-inf and +-100 and decays from -40 to 40, within the bounds of scan_grad.  Where
    v = 1 - a^2 is below 2^-126, 1/m is clamped to 2^63: what it stands beside there, k r (or scale sigmoid(decay) r,
    which is no more), is at most v/2 of the exact m = sqrt(v) and at most 2^-127 of the clamped one, so that both
    terms are below 2^-63 |dh s x|.  dh0 has none."""
    dt, half, rng = DT[dtype], dtype == "bf16", np.random.default_rng(15)
    L, C = 150, 80
    g, u = (rng.standard_normal((1, L, C)) * 30 for _ in range(2))
    g[0, ::7], g[0, 3::11] = np.inf, -np.inf
    u[0, ::5], u[0, 4::13] = -np.inf, np.inf
    x, dy = rng.standard_normal((1, L, C)), rng.standard_normal((1, L, C))
    X, G, I, DY, D = _cuda(x, dt), _cuda(g, dt), _cuda(u, dt), _cuda(dy, dt), _cuda(np.linspace(-40, 40, C))
    h0, dh = _cuda(rng.standard_normal((1, C))), _cuda(rng.standard_normal((1, C)))
    _, _, st = B.gated_scan(X, G, I, D, h0=h0, with_states=True)
    got = B.gated_scan_backward(X, G, I, D, DY, st, dh=dh)
    args = (_np(X)[0], _np(G)[0], _np(I)[0], _np(D), 8.0, _np(h0)[0])
    ref, err = R.scan_grad(*args, _np(DY)[0], _np(dh)[0])
    # |dh| <= |dhT| + the sum of |dy| behind, as a <= 1; s <= 1
    most = np.abs(_np(dh)[0]) + np.abs(_np(DY)[0])[::-1].cumsum(0)[::-1]
    clamp = 2.0 ** -63 * most * np.abs(_np(X)[0])
    _check(got[1][0], ref[1], err[1] + clamp, half, "dgate")
    _check(got[3], ref[3], (err[3] + clamp.sum(0)) * (2 + L / 512), False, "ddecay")
    _check(got[4][0], ref[4], err[4], False, "dh0")
    # dx and dinp: m itself is below 2^-63 there
    _check(got[0][0], ref[0], err[0] + 2.0 ** -63 * most, half, "dx")
    _check(got[2][0], ref[2], err[2] + clamp, half, "dinp")
