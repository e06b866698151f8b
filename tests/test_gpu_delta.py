"""The gated delta rule on the GPU against delta_reference (float64, token by
token), element by element within the bounds derived there: lengths around every
block edge, odd head sizes, shared heads, packed sequences with empty and
single-token ones, slices of fused projections, strong and absent decays, streams,
graphs.  Outputs are poisoned with NaN first, and what lies between slices must
stay untouched."""
import numpy as np
import pytest
import torch

import delta_reference as R
from cnn_convolution_forward_amd import binding as B

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAN = float("nan")


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check(got, ref, err, half, label):
    bound = err + (2.0 ** -8 * (np.abs(ref) + err) if half else 2.0 ** -23 * np.abs(ref)) + 1e-37
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d beyond the bound; first at %s: gpu %r ref %r bound %r" % (label, bad.sum(), bad.size, i, got[i], ref[i], bound[i]))


class Case:
    """Random inputs on the GPU, equal or packed sequences, dense or (slices) in wider rows whose other columns hold a marker."""

    def __init__(self, dt, lens, H, Hv, dk, dv, packed=False, unit=True, slices=0, seed=0, g=None, beta=None, eps=1e-6, gaps=None):
        rng = self.rng = np.random.default_rng(seed + 97 * len(lens) + dk)
        self.dt, self.half, self.lens, self.H, self.Hv, self.dk, self.dv, self.unit, self.eps = DT[dt], dt == "bf16", lens, H, Hv, dk, dv, unit, eps
        self.scale = dk ** -0.5
        self.off = np.concatenate([[0], np.cumsum(lens)]).astype(int)
        n = self.off[-1]
        self.rows = (n,) if packed else (len(lens), lens[0])
        self.kw = dict(offsets=torch.tensor(self.off, dtype=torch.int32, device="cuda"), max_len=max(lens)) if packed else {}
        self.wide, self.slices = [], slices
        std = 1.0 if unit else dk ** -0.5 / 1.5
        self.q, self.k = (self.tensor(rng.standard_normal((n, H, dk)) * std) for _ in range(2))
        self.v, self.dy = (self.tensor(rng.standard_normal((n, Hv, dv))) for _ in range(2))
        g = -np.exp(rng.uniform(-5, 1, (n, Hv))) if g is None else g(rng, (n, Hv))
        beta = rng.uniform(0, 1, (n, Hv)) if beta is None else beta(rng, (n, Hv))
        self.g, self.beta = self.tensor(g[..., None], torch.float32)[..., 0], self.tensor(beta[..., None], torch.float32)[..., 0]
        ends = (len(lens), Hv, dk, dv)
        self.s0, self.ds = (torch.from_numpy(rng.standard_normal(ends) * 0.3).float().cuda() for _ in range(2))

    def tensor(self, a, dt=None):
        """A tensor of heads in rows of its own, or (slices) of `slices` more elements in front and behind."""
        dt = dt or self.dt
        a = torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()
        h, d = a.shape[1:]
        if not self.slices:
            return a.reshape(*self.rows, h, d)
        w = torch.full(self.rows + (h * d + 2 * self.slices,), 77.0, dtype=dt, device="cuda")
        t = w[..., self.slices:self.slices + h * d].unflatten(-1, (h, d))
        t.copy_(a.reshape(*self.rows, h, d))
        self.wide.append(w)
        return t

    def like(self, t):
        """An output like t, poisoned."""
        o = self.tensor(np.zeros((self.off[-1],) + tuple(t.shape[len(self.rows):]) + ((1,) if t.dim() == len(self.rows) + 1 else ())), t.dtype)
        o = o[..., 0] if t.dim() == len(self.rows) + 1 else o
        o.fill_(NAN)
        return o

    def opts(self):
        return dict(scale=self.scale, unit=self.unit, eps=self.eps, **self.kw)

    def data(self):
        return self.q, self.k, self.v, self.g, self.beta

    def untouched(self):
        for w in self.wide:
            assert bool((w[..., :self.slices] == 77).all()) and bool((w[..., w.shape[-1] - self.slices:] == 77).all())

    def sequences(self):
        """Of each sequence and value head: its number and head, rows, q, k, v, g, beta as float64, q and k as used with their factors."""
        flat = lambda t, *d: _np(t).reshape(self.off[-1], *d)
        q, k, v = flat(self.q, self.H, self.dk), flat(self.k, self.H, self.dk), flat(self.v, self.Hv, self.dv)
        g, b = flat(self.g, self.Hv), flat(self.beta, self.Hv)
        for i, n in enumerate(self.lens):
            r = slice(self.off[i], self.off[i] + n)
            for h in range(self.Hv):
                hk = h // (self.Hv // self.H)
                (qu, fq), (ku, fk) = (R.unit(x[r, hk], self.unit, np.float64(np.float32(self.eps))) for x in (q, k))
                yield i, h, hk, r, qu, ku, v[r, h], g[r, h], b[r, h], fq, fk

    def ku(self):
        return (self.dk / 16 + 6) * R.W if self.unit else R.W


def _whole(c, s0=True):
    """Forward and backward against the reference; returns what the calls returned."""
    n = c.off[-1]
    grow = 2 * c.dk ** 0.5 if max(c.lens) > 1000 else 1.0        # sequences that may be run in segments
    s0 = c.s0 if s0 else None
    y = c.like(c.v)
    out = tuple(c.like(t) for t in c.data())
    got, sT, states = B.delta_rule(*c.data(), s0=s0, with_states=True, out=y, **c.opts())
    grads = B.delta_rule_backward(*c.data(), c.dy, states, ds=c.ds, out=out, **c.opts())
    torch.cuda.synchronize()
    c.untouched()
    yv, sv, stv, s0v = _np(got).reshape(n, c.Hv, c.dv), _np(sT), _np(states), _np(c.s0) * (s0 is not None)
    dyv, dsv = _np(c.dy).reshape(n, c.Hv, c.dv), _np(c.ds)
    gv = [_np(t).reshape((n,) + s) for t, s in zip(grads, ((c.H, c.dk), (c.H, c.dk), (c.Hv, c.dv), (c.Hv,), (c.Hv,)))]
    sums = [np.zeros((n, c.H, c.dk)) for _ in range(4)]          # dq, dk and their bounds
    for i, h, hk, r, q, k, v, g, b, fq, fk in c.sequences():
        at = "sequence %d head %d" % (i, h)
        ref, hist = R.forward(q, k, v, g, b, s0v[i, h], c.scale)
        ey, es = R.forward_bounds(q, k, v, g, b, hist, c.scale, c.ku(), c.half, grow)
        _check(yv[r, h], ref, ey, c.half, "y of " + at)
        for t in range(0, len(q), 64):
            assert np.all(np.abs(stv[i, t // 64, h] - hist[t]) <= es[t // 64] + 2.0 ** -23 * np.abs(hist[t])), "state %d of %s" % (t, at)
        assert np.all(np.abs(sv[i, h] - hist[-1]) <= es[-1] + 2.0 ** -23 * np.abs(hist[-1])), "last state of " + at
        # the gradients start from the states as they were saved
        _, hist = R.forward(q, k, v, g, b, stv[i, 0, h] if len(q) else s0v[i, h], c.scale)
        (dq, dk, dv, dg, db, d0), behind = R.backward(q, k, v, g, b, hist, c.scale, dyv[r, h], dsv[i, h])
        if len(q):
            eq, ek, ev, eg, eb, ec, back = R.backward_bounds(q, k, v, g, b, hist, behind, c.scale, dyv[r, h], dsv[i, h], c.ku(), None, c.unit, grow)
            # a saved state is off by its own bound, and what is made of it in its block by as much as a gradient of it says
            more = np.repeat(es[:-1], 64, 0)[:len(q)]
            kn, on = np.sqrt((k * k).sum(1)), np.sqrt((q * q).sum(1))
            z = dv / np.where(b == 0, 1, b)[:, None]
            bh = np.concatenate([behind, dsv[i, h][None]])[:len(q)] + c.scale * q[:, :, None] * dyv[r, h][:, None]
            eq = eq + abs(c.scale) * (np.abs(dyv[r, h]) * more).sum(1, keepdims=True)
            eb = eb + kn * (np.abs(z) * more).sum(1)
            ek = ek + b[:, None] * (kn * 1.0)[:, None] * (np.sqrt((bh ** 2).sum(1)) * more).sum(1, keepdims=True) + b[:, None] * (np.abs(z) * more).sum(1, keepdims=True)
            eg = eg + (np.sqrt((bh ** 2).sum(1)) * more).sum(1) * 2
            _check(gv[2][r, h], dv, ev, c.half, "dv of " + at)
            _check(gv[3][r, h], dg, eg, False, "dg of " + at)
            _check(gv[4][r, h], db, eb, False, "dbeta of " + at)
            assert np.all(np.abs(_np(grads[5])[i, h] - d0) <= ec + 2.0 ** -23 * np.abs(d0)), "ds0 of " + at
            sums[0][r, hk] += R.through_unit(dq, q, fq, c.unit)
            sums[1][r, hk] += R.through_unit(dk, k, fk, c.unit)
            sums[2][r, hk] += back(eq, q, dq, fq) + 2 * R.W * fq * np.abs(dq)
            sums[3][r, hk] += back(ek, k, dk, fk) + 2 * R.W * fk * np.abs(dk)
        else:
            assert np.array_equal(_np(grads[5])[i, h], dsv[i, h]) and np.array_equal(sv[i, h], s0v[i, h])
    _check(gv[0], sums[0], sums[2], c.half, "dq")
    _check(gv[1], sums[1], sums[3], c.half, "dk")
    return got, sT, states, grads


CASES = [
    # dtype, lengths, heads, value heads, dk, dv, packed, unit, slices
    ("bf16", [1], 1, 1, 1, 1, False, False, 0),
    ("bf16", [1, 1, 1], 2, 2, 32, 32, False, True, 0),
    ("bf16", [63], 1, 2, 64, 64, False, True, 0),
    ("bf16", [64] * 2, 1, 1, 128, 128, False, True, 0),
    ("bf16", [65], 2, 4, 128, 128, False, True, 8),
    ("bf16", [200], 1, 1, 128, 96, False, True, 3),
    ("bf16", [130, 0, 1, 3, 66, 0], 1, 3, 40, 72, True, True, 0),
    ("bf16", [0, 0], 1, 1, 16, 16, True, True, 0),
    ("bf16", [5, 150, 2], 2, 2, 33, 31, True, False, 1),
    ("bf16", [129], 3, 3, 96, 128, False, False, 0),
    ("f32", [1], 1, 1, 3, 2, False, True, 0),
    ("f32", [63, 64, 65, 0, 1], 1, 2, 33, 20, True, True, 0),
    ("f32", [129] * 2, 1, 1, 128, 128, False, True, 4),
    ("f32", [40, 2, 7], 2, 4, 12, 99, True, False, 3),
    ("f32", [70], 1, 1, 72, 64, False, False, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_delta_rule(case):
    _whole(Case(*case))


@pytest.mark.parametrize("case", [("bf16", [1100], 1, 1, 32, 32, False, True, 0), ("bf16", [64 * 40, 0, 700, 1, 64 * 16, 1300], 1, 2, 33, 40, True, True, 3),
                                  ("f32", [64 * 16] * 2, 1, 2, 24, 72, False, True, 0), ("f32", [1500, 64 * 5, 64 * 6 + 1], 2, 2, 96, 20, True, False, 0)],
                         ids=["0", "1", "2", "3"])
def test_sequences_in_segments(case):
    """Long sequences of few heads are cut into segments that run at once."""
    c = Case(*case, g=lambda r, s: -np.exp(r.uniform(-9, -2, s)))
    got = _whole(c)
    again = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dt,max_len", [("bf16", 900), ("f32", 5000)])
def test_segments_among_many_short_sequences(dt, max_len):
    """One long sequence among short and empty ones, with the longest given exactly and far too long."""
    c = Case(dt, [3] * 20 + [900, 0, 0, 640] + [70] * 6, 1, 2, 32, 40, packed=True, g=lambda r, s: -np.exp(r.uniform(-9, -2, s)))
    c.kw["max_len"] = max_len
    _whole(c)


def test_no_first_state():
    _whole(Case("bf16", [100], 1, 2, 48, 40), s0=False)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("g", ["none", "strong", "mixed", "shut"])
def test_decays(g, dt):
    """No decay at all; decays that forget within a token; both in turn (differences of large sums); and decays of exp(-inf)."""
    f = {"none": lambda r, s: np.zeros(s), "strong": lambda r, s: -r.uniform(20, 200, s),
         "mixed": lambda r, s: np.where(r.uniform(0, 1, s) < 0.1, -r.uniform(50, 3000, s), -r.uniform(0, 0.01, s)),
         "shut": lambda r, s: np.where(r.uniform(0, 1, s) < 0.1, -1e4, -r.uniform(0, 1, s))}[g]
    c = Case(dt, [150], 1, 2, 32, 24, g=f, seed=5)
    got = _whole(c)
    if g == "shut":
        c.g[c.g == -1e4] = -np.inf
        y, sT = B.delta_rule(*c.data(), s0=c.s0, **c.opts())
        assert torch.equal(y, got[0]) and torch.equal(sT, got[1])
        c.g[c.g == -np.inf] = -3e38
        assert torch.equal(B.delta_rule(*c.data(), s0=c.s0, **c.opts())[0], got[0])


@pytest.mark.parametrize("b", [0.0, 1.0])
def test_strengths_at_their_ends(b):
    """beta = 0 writes nothing, and its gradient is there; beta = 1 replaces what stood at the key."""
    _whole(Case("f32", [80], 1, 1, 32, 32, beta=lambda r, s: np.full(s, b)))


@pytest.mark.parametrize("size", [1e-12, 1e15])
def test_sizes_of_values(size):
    """Powers of two bring every tile into the range of fp16: results scale with the values."""
    a, b = (Case("f32", [100], 1, 1, 32, 48, seed=2) for _ in range(2))
    f = 2.0 ** round(np.log2(size))
    for t in (b.v, b.s0, b.dy, b.ds):
        t.mul_(f)
    ya, sa, sta = B.delta_rule(*a.data(), s0=a.s0, with_states=True, **a.opts())
    yb, sb, stb = B.delta_rule(*b.data(), s0=b.s0, with_states=True, **b.opts())
    assert torch.equal(ya * f, yb) and torch.equal(sa * f, sb) and torch.equal(sta * f, stb)
    ga, gb = B.delta_rule_backward(*a.data(), a.dy, sta, ds=a.ds, **a.opts()), B.delta_rule_backward(*b.data(), b.dy, stb, ds=b.ds, **b.opts())
    for i, p in ((0, 2), (1, 2), (2, 1), (5, 1)):
        assert torch.equal(ga[i] * f ** p, gb[i]), i


def test_columns_and_keys_of_different_sizes():
    """Columns of v, and with unit = 1 rows of q and k, many powers of two apart: each keeps its own precision."""
    for unit in (True, False):
        c = Case("bf16", [130], 1, 1, 64, 64, unit=unit, seed=8)
        c.v.mul_(2.0 ** torch.randint(-30, 30, (64,), device="cuda"))
        c.s0.mul_(2.0 ** torch.randint(-3, 3, (64,), device="cuda"))
        if unit:
            c.k.mul_(2.0 ** torch.randint(-8, 30, (130, 1), device="cuda").reshape(1, 130, 1, 1))
            c.q.mul_(2.0 ** torch.randint(-8, 30, (130, 1), device="cuda").reshape(1, 130, 1, 1))
        n = 130
        y, sT = B.delta_rule(*c.data(), s0=c.s0, **c.opts())
        for i, h, hk, r, q, k, v, g, b, _, _ in c.sequences():
            for j in range(c.dv):                                # one column after another: none is looked at beside another
                ref, hist = R.forward(q, k, v[:, j:j + 1], g, b, _np(c.s0)[0, 0][:, j:j + 1], c.scale)
                ey, es = R.forward_bounds(q, k, v[:, j:j + 1], g, b, hist, c.scale, c.ku(), True)
                _check(_np(y)[0, :, 0, j:j + 1], ref, ey, True, "column %d" % j)
                assert np.all(np.abs(_np(sT)[0, 0][:, j:j + 1] - hist[-1]) <= es[-1] + 2.0 ** -23 * np.abs(hist[-1]))


def test_rows_of_zeros():
    """Keys and queries of zeros have no direction: with eps they stay zeros, and without it too."""
    for eps in (1e-6, 0.0):
        c = Case("bf16", [70], 1, 1, 32, 32, eps=eps)
        c.k[:, ::3], c.q[:, 1::4] = 0, 0
        y, sT, st = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
        grads = B.delta_rule_backward(*c.data(), c.dy, st, ds=c.ds, **c.opts())
        assert bool((y[:, 1::4] == 0).all()) and all(bool(torch.isfinite(t).all()) for t in (y, sT) + grads)


@pytest.mark.parametrize("dt,eps,packed", [("bf16", 1e-6, False), ("f32", 1e-2, True), ("f32", 1e4, False)])
def test_gradients_of_rows_of_zeros(dt, eps, packed):
    """x / sqrt(sum x^2 + eps) has the slope 1 / sqrt(eps) at zero (a padded batch's keys and queries)."""
    c = Case(dt, [40, 70] if packed else [70] * 2, 2, 4, 32, 48, packed=packed, eps=eps)
    c.k[..., ::3, :, :] = 0
    c.q[..., 1::4, :, :] = 0
    got = _whole(c)
    assert bool((got[3][1][..., ::3, :, :] != 0).any())


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -60, 2.0 ** 60, 2.0 ** 100])
def test_unit_length_of_tiny_and_huge_rows(size):
    """Without eps the unit length does not depend on the size, down to squares far below fp32 and up to those beyond it: the same bits,
    whole and by steps; and a step leaves rows of zeros, as whole sequences do."""
    c = Case("f32", [70], 1, 2, 40, 32, eps=0.0)
    y, sT, st = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
    q, k, *rest = c.data()
    y2, sT2 = B.delta_rule(q * size, k * size, *rest, s0=c.s0, **c.opts())
    assert torch.equal(y, y2) and torch.equal(sT, sT2)
    grads = [B.delta_rule_backward(q * f, k * f, *rest, c.dy, st, ds=c.ds, **c.opts()) for f in (1.0, size)]
    assert torch.equal(grads[0][2], grads[1][2]) and torch.equal(grads[0][5], grads[1][5])
    assert torch.equal(grads[0][0], grads[1][0] * size) and torch.equal(grads[0][1], grads[1][1] * size)
    o = dict(scale=c.scale, unit=True, eps=0.0)
    out = []
    for f in (1.0, size, 0.0):
        s = c.s0.clone()
        out.append((B.delta_rule_step(q[:, 0] * f, k[:, 0] * f, *(t[:, 0] for t in rest), s, **o), s))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert bool((out[2][0] == 0).all()) and float((out[2][1] - c.s0 * torch.exp(c.g[:, 0])[..., None, None]).abs().max()) <= 1e-6


# ---- token by token, and in parts --------------------------------------------------

@pytest.mark.parametrize("dt,H,Hv,dk,dv,unit", [("bf16", 2, 4, 128, 128, True), ("f32", 1, 3, 37, 99, False), ("bf16", 1, 1, 1, 1, False),
                                                ("f32", 2, 2, 128, 33, True)])
def test_step_by_step(dt, H, Hv, dk, dv, unit):
    """Every token alone, from and to the same state: the reference's recurrence, each step within the errors of its own sums."""
    c = Case(dt, [9] * 3, H, Hv, dk, dv, unit=unit, slices=5)
    s = c.s0.clone()
    flat = lambda t: t.reshape(3, 9, *t.shape[2:])
    for t in range(9):
        before = _np(s)
        y = torch.full((3, Hv, dv), NAN, dtype=c.dt, device="cuda")
        assert B.delta_rule_step(c.q[:, t], c.k[:, t], c.v[:, t], c.g[:, t], c.beta[:, t], s, scale=c.scale, unit=unit, eps=c.eps, out=y) is y
        for i, h, hk, r, q, k, v, g, b, _, _ in c.sequences():
            q, k, v, g, b = (x[t:t + 1] for x in (q, k, v, g, b))
            ref, hist = R.forward(q, k, v, g, b, before[i, h], c.scale)
            S, a = np.abs(before[i, h]) * np.exp(g[0]), np.abs
            ku = (dk / 16 + 6) * R.W
            ee = (dk / 4 + 4) * R.W * (a(v[0]) + a(k[0]) @ S) + ku * (a(k[0]) @ S)
            es = 2 * R.W * S + np.outer(a(k[0]), b[0] * ee) + (ku + 4 * R.W) * np.outer(a(k[0]), b[0] * (a(v[0]) + a(k[0]) @ S))
            ey = c.scale * (a(q[0]) @ es + ((dk / 4 + 6) * R.W + ku) * (a(q[0]) @ (S + np.outer(a(k[0]), b[0] * (a(v[0]) + a(k[0]) @ S)))))
            _check(_np(s)[i, h], hist[-1], es, False, "state")
            _check(_np(y)[i, h], ref[0], ey, c.half, "y")
    c.untouched()


def test_in_two_parts_with_the_state_between():
    """Cut at a block's edge the same bits; cut elsewhere within the bounds; and a step goes on where a whole sequence ended."""
    c = Case("bf16", [200], 2, 2, 64, 64)
    y, sT = B.delta_rule(*c.data(), s0=c.s0, **c.opts())
    for cut in (64, 128, 37):
        a, b = [t[:, :cut].contiguous() for t in c.data()], [t[:, cut:].contiguous() for t in c.data()]
        y1, s1 = B.delta_rule(*a, s0=c.s0, **c.opts())
        y2, s2 = B.delta_rule(*b, s0=s1, **c.opts())
        if cut % 64 == 0:
            assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(s2, sT)
        else:
            assert float((s2 - sT).norm()) <= 1e-5 * float(sT.norm())
            # two roundings to bf16 of nearly the same value
            assert float((torch.cat([y1, y2], 1).float() - y.float()).abs().amax()) <= 2.0 ** -7 * float(y.float().abs().amax())


def test_same_bits_in_any_batch_and_at_any_time():
    """A sequence alone, packed among others and in equal ones; twice the same call."""
    lens = [70, 1, 0, 130, 64]
    c = Case("bf16", lens, 2, 4, 64, 64, packed=True)
    y, sT, st = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
    grads = B.delta_rule_backward(*c.data(), c.dy, st, ds=c.ds, **c.opts())
    again = B.delta_rule_backward(*c.data(), c.dy, st, ds=c.ds, **c.opts())
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    o = dict(scale=c.scale, unit=True, eps=c.eps)
    for i, n in enumerate(lens):
        if not n:
            continue
        r = slice(c.off[i], c.off[i] + n)
        one = [t[r][None] for t in c.data()]
        y1, s1, st1 = B.delta_rule(*one, s0=c.s0[i:i + 1], with_states=True, **o)
        assert torch.equal(y1[0], y[r]) and torch.equal(s1[0], sT[i]) and torch.equal(st1[0], st[i, :st1.shape[1]])
        g1 = B.delta_rule_backward(*one, c.dy[r][None], st1, ds=c.ds[i:i + 1], **o)
        for a, b in zip(g1[:5], grads[:5]):
            assert torch.equal(a[0], b[r])
        assert torch.equal(g1[5][0], grads[5][i])


@pytest.mark.parametrize("dt,lens,dk,dv", [("bf16", [64 * 200], 64, 96), ("f32", [64 * 120], 64, 96), ("bf16", [1000] * 8, 128, 128), ("bf16", [70] * 64, 32, 32)],
                         ids=["segments", "segments-f32", "equal", "short"])
def test_shared_heads_are_the_same_as_repeated_ones(dt, lens, dk, dv):
    """Queries and keys of a group of value heads, once for all of them and once for each: the same bits, however many workgroups run at once."""
    c = Case(dt, lens, 4, 16, dk, dv, g=lambda r, s: -np.exp(r.uniform(-9, -2, s)))
    q, k, *rest = c.data()
    o = dict(scale=c.scale, unit=True, eps=c.eps)
    want = B.delta_rule(q.repeat_interleave(4, -2), k.repeat_interleave(4, -2), *rest, s0=c.s0, with_states=True, **o)
    back = B.delta_rule_backward(q.repeat_interleave(4, -2), k.repeat_interleave(4, -2), *rest, c.dy, want[2], ds=c.ds, **o)
    for _ in range(4):
        got = [B.delta_rule(q, k, *rest, s0=c.s0, with_states=True, **o) for _ in range(2)]
        grads = [B.delta_rule_backward(q, k, *rest, c.dy, want[2], ds=c.ds, **o) for _ in range(2)]
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
        assert all(torch.equal(a, b) for g in grads for a, b in zip(g[2:], back[2:]))
        assert all(torch.equal(a, b) for a, b in zip(grads[0][:2], grads[1][:2]))


# ---- what does not belong to a sequence ------------------------------------------------

@pytest.mark.parametrize("off,rows,max_len", [([7, 40, 40, 140], 171, 100), ([0, 300, 300, 400], 500, 130), ([0, 0, 0], 70, 1), ([0, 0], 90, 0),
                                              ([3] + [3 + 5 * i for i in range(1, 40)], 300, 2)])
def test_rows_of_no_sequence(off, rows, max_len):
    """Zeros where the helpers allocate, as they were in a given out; NaN in them reach nothing."""
    c = Case("bf16", [rows], 1, 2, 32, 40)
    on = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for a, b in zip(off, off[1:]):
        on[a:min(b, a + max_len)] = True
    data = [t[0].clone() for t in c.data()]
    dy = c.dy[0].clone()
    for t in data + [dy]:
        t[~on] = NAN
    kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_len=max_len, scale=c.scale, unit=True)
    given = [torch.full_like(t, 5.0) for t in [data[2]] + data]
    y, sT, st = B.delta_rule(*data, with_states=True, **kw)
    B.delta_rule(*data, out=given[0], **kw)
    grads = B.delta_rule_backward(*data, dy, st, **kw)
    B.delta_rule_backward(*data, dy, st, out=tuple(given[1:]), **kw)
    assert bool(torch.isfinite(sT).all()) and bool(torch.isfinite(grads[5]).all())
    for new, old in zip((y,) + grads[:5], given):
        assert bool((new[~on] == 0).all()) and bool((old[~on] == 5).all()) and torch.equal(new[on], old[on]) and bool(torch.isfinite(new).all())
    mixed = B.delta_rule_backward(*data, dy, st, out=(None, given[2], None, None, None), **kw)
    assert bool((mixed[0][~on] == 0).all()) and bool((given[2][~on] == 5).all()) and bool((mixed[3][~on] == 0).all())


@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_sequence_head_and_later_blocks(bad):
    c = Case("bf16", [200, 130, 64], 2, 4, 32, 32, packed=True)
    y0, s0, st0 = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
    g0 = B.delta_rule_backward(*c.data(), c.dy, st0, ds=c.ds, **c.opts())
    for name, h in (("q", 1), ("k", 0), ("v", 3), ("g", 2), ("beta", 1)):
        if name == "g" and bad == -float("inf"):
            continue                                             # a decay to nothing
        data = dict(zip(("q", "k", "v", "g", "beta"), (t.clone() for t in c.data())))
        data[name][c.off[1] + 70, h] = bad                       # sequence 1, its second block
        y, sT, st = B.delta_rule(*data.values(), s0=c.s0, with_states=True, **c.opts())
        heads = [h] if name in ("v", "g", "beta") else [2 * h, 2 * h + 1]
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[c.off[1] + 64:c.off[2], heads] = True
        assert torch.equal(y[~hit], y0[~hit]) and not bool(torch.isfinite(y[c.off[1] + 70, heads]).all()), name
        keep = torch.ones_like(sT, dtype=torch.bool)
        keep[1, heads] = False
        assert torch.equal(sT[keep], s0[keep]), name
        grads = B.delta_rule_backward(*data.values(), c.dy, st0, ds=c.ds, **c.opts())
        for i, (a, b) in enumerate(zip(grads[:5], g0[:5])):
            other = torch.ones(a.shape[:2], dtype=torch.bool, device="cuda")
            per = 2 if i < 2 else 1
            other[c.off[1]:c.off[2], [x // per for x in heads]] = False
            assert torch.equal(a[other], b[other]), (name, i)
        assert torch.equal(grads[5][keep], g0[5][keep]), name


# ---- streams, graphs, workspaces ---------------------------------------------------------

def test_two_streams_at_once():
    """Two calls under way at once, each with a workspace of its own."""
    cs = [Case(dt, [300] * 4, 2, 2, 64, 64, seed=i) for i, dt in enumerate(("bf16", "f32"))]
    want = []
    for c in cs:
        y, sT, st = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
        want.append((y, sT, st) + B.delta_rule_backward(*c.data(), c.dy, st, ds=c.ds, **c.opts()))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cs], [None, None]
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                y, sT, st = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
                got[i] = (y, sT, st) + B.delta_rule_backward(*c.data(), c.dy, st, ds=c.ds, **c.opts())
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_graph():
    """Forward, backward and a step in one graph, replayed with other inputs and eager work between."""
    c = Case("bf16", [150] * 2, 1, 2, 64, 32)
    s = c.s0.clone()
    first = [t[:, 0].contiguous() for t in c.data()]

    def run():
        y, sT, st = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
        g = B.delta_rule_backward(*c.data(), c.dy, st, ds=c.ds, **c.opts())
        return (y, sT, st) + g + (B.delta_rule_step(*first, s, scale=c.scale, unit=True),)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        c.v.copy_(torch.randn_like(c.v.float()))
        s.copy_(c.s0)
        graph.replay()
        torch.cuda.synchronize()
        after = s.clone()
        s.copy_(c.s0)
        want = run()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(after, s), i


def test_segments_on_two_streams_and_in_a_graph():
    """Sequences that are cut: calls on two streams at once and a replayed graph give the bits of a call alone."""
    long = lambda r, s: -np.exp(r.uniform(-9, -2, s))
    cs = [Case("bf16", [900, 0, 3, 1400], 1, 2, 64, 96, packed=True, g=long), Case("f32", [1100] * 2, 2, 2, 40, 33, g=long, seed=3)]

    def run(c):
        y, sT, st = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
        return (y, sT) + B.delta_rule_backward(*c.data(), c.dy, st, ds=c.ds, **c.opts())

    want = [run(c) for c in cs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cs], [None, None]
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                got[i] = run(c)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for a, b in zip(want, got) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [run(c) for c in cs]
    for i in range(3):
        for c in cs:
            c.v.copy_(torch.randn_like(c.v.float()))
        graph.replay()
        torch.cuda.synchronize()
        want = [run(c) for c in cs]
        assert all(torch.equal(p, q) for a, b in zip(want, out) for p, q in zip(a, b)), i


def test_descending_offsets_of_long_sequences_stay_inside():
    """As below, with sequences that are cut into segments, and a workspace between guards."""
    c = Case("bf16", [1500], 1, 2, 32, 32)
    data, dy = [t[0].contiguous() for t in c.data()], c.dy[0].contiguous()
    for off in ([0, 1500, 0, 1500], [1500, 700, 0, 1 << 30], [0, 1500, 700, 1500]):
        kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_len=1500, unit=True)
        seq, par = B.make_delta(data[0], data[2], fill=True, **kw)
        held = torch.full((B.conv_delta_bwd_workspace_bytes(seq, par) + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
        n = B.conv_delta_fwd_workspace_bytes(seq, par)
        y, sT, st = B.delta_rule(*data, with_states=True, workspace=held[4096:4096 + n], **kw)
        assert bool((held[:4096] == 0x5a).all()) and bool((held[4096 + n:] == 0x5a).all())
        B.delta_rule_backward(*data, dy, torch.zeros_like(st), workspace=held[4096:-4096], **kw)
        assert bool((held[:4096] == 0x5a).all()) and bool((held[-4096:] == 0x5a).all())


def test_given_workspaces():
    c = Case("bf16", [100], 1, 2, 48, 40)
    par = B.make_delta(c.q, c.v, scale=c.scale, unit=True)
    ws = [torch.full((f(*par),), 0xff, dtype=torch.uint8, device="cuda") for f in (B.conv_delta_fwd_workspace_bytes, B.conv_delta_bwd_workspace_bytes)]
    y, sT, st = B.delta_rule(*c.data(), s0=c.s0, with_states=True, workspace=ws[0], **c.opts())
    want = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
    assert all(torch.equal(a, b) for a, b in zip((y, sT, st), want))
    got = B.delta_rule_backward(*c.data(), c.dy, st, ds=c.ds, workspace=ws[1], **c.opts())
    want = B.delta_rule_backward(*c.data(), c.dy, st, ds=c.ds, **c.opts())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(B.ConvError):
        B.delta_rule(*c.data(), workspace=ws[0][:-16], **c.opts())
    with pytest.raises(B.ConvError):
        B.delta_rule_backward(*c.data(), c.dy, st, workspace=ws[1][:-16], **c.opts())


def test_descending_offsets_stay_inside():
    """Which rows are computed is unspecified; what lies outside the tensors stays as it was, and the call ends."""
    c = Case("bf16", [300], 1, 2, 32, 32)
    data, dy = [t[0].contiguous() for t in c.data()], c.dy[0].contiguous()
    for off in ([0, 200, 100, 300], [250, -5, 1 << 30, 7], [300, 0, 300, 0], [-9, -9, -9, -9]):
        kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_len=200, unit=True)
        y, sT, st = B.delta_rule(*data, with_states=True, **kw)
        st = torch.zeros_like(st)
        grads = B.delta_rule_backward(*data, dy, st, **kw)
        torch.cuda.synchronize()
        assert y.shape == data[2].shape and grads[0].shape == data[0].shape


def test_refusals_leave_outputs():
    c = Case("bf16", [10] * 2, 2, 4, 16, 16)
    q, k, v, g, b = c.data()
    y = torch.full_like(v, 3.0)
    for bad in (lambda: B.delta_rule(q, k[..., :15], v, g, b, out=y), lambda: B.delta_rule(q, k, v, g[..., :3], b, out=y),
                lambda: B.delta_rule(q, k, v, g.bfloat16(), b, out=y), lambda: B.delta_rule(q.float(), k, v, g, b, out=y),
                lambda: B.delta_rule(q, k, v, g, b, s0=c.s0[:1], out=y), lambda: B.delta_rule(q.transpose(2, 3), k, v, g, b, out=y),
                lambda: B.delta_rule(q, k, v.cpu(), g, b, out=y), lambda: B.delta_rule(q, k, v, g, b, out=y[:, :5])):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: B.delta_rule(q[:, :, [0, 1, 1]], k[:, :, [0, 1, 1]], v, g, b, out=y), lambda: B.delta_rule(q, k, v, g, b, out=v),
                lambda: B.delta_rule(q, k, v, g, b, scale=NAN, out=y)):
        with pytest.raises(B.ConvError):
            bad()
    assert bool((y == 3).all())
