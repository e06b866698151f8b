"""The AdamW step on the GPU.  32-bit moments against float64 within a bound of
a few roundings; 8-bit moments against a numpy float32 evaluation of the same
operations, whose codes and scales must be equal; the random rounding is right
on average and follows the 32-bit moments over many steps."""
import numpy as np
import pytest
import torch

from cnn_convolution_forward_amd import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
f32 = np.float32
HYPER = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8)


def _cuda(a, dt=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dt)


def _shift(t, by):
    """The same values at an address `by` elements past an aligned one."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    buf[by:].copy_(t)
    return buf[by:]


SIZES = [1, 3, 255, 256, 257, 0, 4095, 4096, 4097, 20001]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_step_32(grad, shift):
    rng = np.random.default_rng(1)
    p, g, m, v = ([rng.standard_normal(n) * s for n in SIZES] for s in (0.1, 0.01, 0.002, 0.0))
    v = [rng.random(n) * 1e-4 for n in SIZES]
    tp, tm, tv = ([_shift(_cuda(f32(t)), shift) for t in a] for a in (p, m, v))
    tg = [_shift(_cuda(f32(t), grad), shift) for t in g]
    copies = [_shift(torch.full((n,), float("nan"), dtype=torch.bfloat16, device="cuda"), shift) if i % 3 else None
              for i, n in enumerate(SIZES)]
    decays = [0.1 * (i % 2) for i in range(len(SIZES))]
    opt = B.AdamW(tp, tg, tm, tv, copies=copies, weight_decay=decays, steps=6, grad_scale=_cuda(f32([0.5])), **HYPER)
    before = [[t.double().cpu().numpy() for t in a] for a in (tp, tg, tm, tv)]
    opt.step()
    assert opt.steps == 7
    c1, c2 = 1 - 0.9 ** 7, 1 - 0.999 ** 7
    for i, (P, G, M, V) in enumerate(zip(*before)):
        G = G * 0.5
        m1, v1 = 0.9 * M + 0.1 * G, 0.999 * V + 0.001 * G * G
        em, ev = 3 * U * (np.abs(0.9 * M) + np.abs(0.1 * G)), 3 * U * v1
        d = HYPER["lr"] / c1 * m1 / (np.sqrt(v1 / c2) + 1e-8)
        ed = HYPER["lr"] / c1 * em / (np.sqrt(v1 / c2) + 1e-8) + 8 * U * np.abs(d)
        p1 = P * (1 - HYPER["lr"] * decays[i]) - d
        for name, got, ref, err in (("m", tm, m1, em), ("v", tv, v1, ev), ("p", tp, p1, ed + 3 * U * (np.abs(P) + np.abs(p1)))):
            got = got[i].double().cpu().numpy()
            assert np.all(np.abs(got - ref) <= err + 1e-40), (name, SIZES[i])
        if copies[i] is not None:
            assert torch.equal(copies[i], tp[i].to(torch.bfloat16))


# ---- 8 bits ------------------------------------------------------------------------

def _bits(seed, step, which, n):
    u = np.uint64
    mask = u(0xffffffff)
    key = (u(seed) * u(0x632be5ab) + u(step) * u(0x2545f491) + u(which) * u(0x7feb352d)) & mask
    z = (key + np.arange(n, dtype=u) * u(0x9e3779b1)) & mask
    z = ((z ^ (z >> u(15))) * u(0x2c1b3c6d)) & mask
    z = ((z ^ (z >> u(12))) * u(0x297a2d39)) & mask
    return z ^ (z >> u(15))


def _decode(q, s, top, power):
    t = f32(q) * f32(1.0 / top)
    t = t * t
    return (t * t if power == 4 else t) * s


def _blocks(a):
    return np.pad(a, (0, -len(a) % 256)).reshape(-1, 256)


def _encode(x, top, power, rnd, keep):
    n, x, rnd = len(x), _blocks(x), _blocks(f32(rnd) * f32(2.0 ** -16))
    s = x.max(1, keepdims=True)
    s = np.where(s < f32(2.0 ** -126), f32(0), s)
    inv = np.where(s > 0, f32(1) / np.where(s > 0, s, f32(1)), f32(0))
    root = np.sqrt(x * inv)
    root = np.sqrt(root) if power == 4 else root
    low = np.minimum(np.floor(root * f32(top)), f32(top - 1))
    v0, v1 = _decode(low, s, top, power), _decode(low + f32(1), s, top, power)
    q = low + (rnd * (v1 - v0) < x - v0)
    if keep:
        q = np.where((q == 0) & (x > 0) & (s > 0), 1, q)
    return q.reshape(-1)[:n], s[:, 0]


def _step8(m, ms, v, vs, g, seed, step, which):
    """numpy float32: every operation rounded by itself."""
    m = np.sign(m) * _decode(np.abs(m), np.repeat(ms, 256)[:len(m)], 127, 2)
    v = _decode(v, np.repeat(vs, 256)[:len(v)], 255, 4)
    m1 = f32(m) * f32(0.9) + g * f32(1 - 0.9)
    v1 = v * f32(0.999) + g * g * f32(1 - 0.999)
    z = _bits(seed, step, which, len(g))
    qm, sm = _encode(np.abs(m1), 127, 2, (z & np.uint64(0xffff)).astype(np.int64), False)
    qv, sv = _encode(v1, 255, 4, (z >> np.uint64(16)).astype(np.int64), True)
    return m1, v1, np.sign(m1) * qm, sm, qv, sv


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_step_8(grad, shift):
    rng = np.random.default_rng(2)
    g = [f32(rng.standard_normal(n) * np.exp(rng.uniform(-6, 0, n))) for n in SIZES]
    for t in g:
        t[::17] = 0
    p = [f32(rng.standard_normal(n)) for n in SIZES]
    tp, tg = [_shift(_cuda(t), shift) for t in p], [_shift(_cuda(t, grad), shift) for t in g]
    q = [_shift(torch.zeros(n, dtype=torch.int8, device="cuda"), shift) for n in SIZES]
    r = [_shift(torch.zeros(n, dtype=torch.uint8, device="cuda"), shift) for n in SIZES]
    copies = [_shift(torch.zeros(n, dtype=torch.bfloat16, device="cuda"), shift) for n in SIZES]
    opt = B.AdamW(tp, tg, q, r, copies=copies, bits=8, seed=5, weight_decay=0.01, **HYPER)
    for step in range(1, 4):
        old = [[t.cpu().numpy().copy() for t in a] for a in (opt.m, opt.m_scale, opt.v, opt.v_scale, tp)]
        opt.step()
        vm, vv = opt.state_values()
        c1, c2 = 1 - 0.9 ** step, 1 - 0.999 ** step
        for i, n in enumerate(SIZES):
            if not n:
                continue
            gi = tg[i].float().cpu().numpy()
            m1, v1, qm, sm, qv, sv = _step8(f32(old[0][i]), old[1][i], f32(old[2][i]), old[3][i], gi, 5, step, i)
            got = [t[i].cpu().numpy() for t in (opt.m, opt.m_scale, opt.v, opt.v_scale)]
            for name, a, b in zip(("m", "m_scale", "v", "v_scale"), got, (qm, sm, qv, sv)):
                assert np.array_equal(a.astype(np.float64), b.astype(np.float64)), (name, step, n)
            assert np.array_equal(vm[i].cpu().numpy(), np.sign(qm) * _decode(np.abs(qm), np.repeat(sm, 256)[:n], 127, 2))
            assert np.array_equal(vv[i].cpu().numpy(), _decode(qv, np.repeat(sv, 256)[:n], 255, 4))
            P = old[4][i].astype(np.float64)
            d = HYPER["lr"] / c1 * m1.astype(np.float64) / (np.sqrt(v1.astype(np.float64) / c2) + 1e-8)
            ref = P * (1 - HYPER["lr"] * 0.01) - d
            now = tp[i].double().cpu().numpy()
            assert np.all(np.abs(now - ref) <= U * (8 * np.abs(d) + 3 * np.abs(P) + 3 * np.abs(ref)) + 1e-40)
            assert torch.equal(copies[i], tp[i].to(torch.bfloat16))


def test_random_rounding_is_right_on_average():
    """4096 elements of equal gradients, 64 seeds: the mean of the decoded moments is the moment.  A
    rounding between two codes varies by at most half their distance (here below 1/60 of the value for m,
    1/30 for v), so the mean of 64 * 4096 draws is off by less than 6/(2*512) of that."""
    n = 4096
    g = torch.full((n,), 0.3, device="cuda")
    g[::256] = 1.0                                   # the block's largest
    tot_m = tot_v = 0.0
    for seed in range(64):
        opt = B.AdamW([torch.zeros(n, device="cuda")], [g], bits=8, seed=seed)
        opt.step()
        m, v = opt.state_values()
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[::256] = False
        tot_m += float(m[0][keep].double().mean()) / 64
        tot_v += float(v[0][keep].double().mean()) / 64
    assert abs(tot_m / 0.03 - 1) < 6 / 1024 / 30
    assert abs(tot_v / 0.9e-4 - 1) < 6 / 1024 / 15


def test_8_bit_moments_follow_32_bit_ones():
    """1500 steps of noisy gradients whose size falls tenfold on the way: the 8-bit v goes down with the
    32-bit one (rounding to the nearest code would leave it), to a tenth on average over the elements."""
    rng = np.random.default_rng(3)
    n = 2048
    size = _cuda(f32(np.exp(rng.uniform(-2, 0, n))))
    a = B.AdamW([torch.zeros(n, device="cuda")], [size], lr=1e-4)
    b = B.AdamW([torch.zeros(n, device="cuda")], [size], lr=1e-4, bits=8)
    gen = torch.Generator(device="cuda").manual_seed(0)
    for i in range(1500):
        g = size * torch.randn(n, generator=gen, device="cuda") * (1.0 if i < 300 else 0.1)
        a.step([g])
        b.step([g])
    ratio = (b.state_values()[1][0] / a.v[0]).double()
    assert abs(float(ratio.mean()) - 1) < 0.1
    assert float((b.params[0] - a.params[0]).norm() / a.params[0].norm()) < 0.1


def test_zero_and_non_finite_gradients():
    n = 600
    g = torch.zeros(n, device="cuda")
    opt = B.AdamW([torch.ones(n, device="cuda")], [g], bits=8)
    opt.step()
    assert bool((opt.params[0] == 1).all()) and not bool(opt.m[0].any()) and not bool(opt.v[0].any())
    assert not bool(opt.m_scale[0].any())
    g[300] = float("nan")
    opt.step()
    assert bool(torch.isnan(opt.m_scale[0]).eq(torch.tensor([False, True, False], device="cuda")).all())
    bad = torch.isnan(opt.params[0])
    assert int(bad.sum()) == 1 and bool(bad[300])
    one = B.AdamW([torch.ones(n, device="cuda")], [g])
    one.step()
    assert int(torch.isnan(one.params[0]).sum()) == 1 and int(torch.isnan(one.m[0]).sum()) == 1


def test_many_tensors_streams_and_graph():
    """170 tensors (more than a launch takes): the same bits on another stream, and from replays of a graph."""
    rng = np.random.default_rng(6)
    sizes = [int(rng.integers(1, 9000)) for _ in range(170)]
    start = [_cuda(f32(rng.standard_normal(n))) for n in sizes]
    grads = [_cuda(f32(rng.standard_normal(n))) for n in sizes]

    def fresh(bits):
        return B.AdamW([t.clone() for t in start], grads, bits=bits, weight_decay=0.01)

    for bits in (32, 8):
        want, other, cap = fresh(bits), fresh(bits), fresh(bits)
        want.step()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            other.step()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want.params, other.params))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cap.step()
        for i in range(3):                       # a captured step keeps its number: replays equal eager calls of it
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(cap.params + cap.m + cap.v, want.params + want.m + want.v)), (bits, i)
            want.steps = 0
            want.step()


def test_helper_refuses():
    p, g = [torch.zeros(10, device="cuda")], [torch.zeros(10, device="cuda")]
    with pytest.raises(ValueError):
        B.AdamW(p, [])
    with pytest.raises(ValueError):
        B.AdamW(p, [torch.zeros(9, device="cuda")])
    with pytest.raises(TypeError):
        B.AdamW([p[0].bfloat16()], g)
    with pytest.raises(TypeError):
        B.AdamW(p, g, copies=[torch.zeros(10, device="cuda")])
    with pytest.raises(ValueError):
        B.AdamW(p, g, bits=8, m_scale=[])
    with pytest.raises(B.ConvError):
        B.AdamW(p, g, m=[p[0]]).step()
    with pytest.raises(B.ConvError):
        B.AdamW(p, g, betas=(1.0, 0.9)).step()
    empty = B.AdamW([], [])
    empty.step()


def test_refused_step_changes_nothing():
    """After a list that is refused, the next step equals that of an optimiser that never saw it."""
    n = 300
    start, grad = torch.linspace(-1, 1, n, device="cuda"), torch.linspace(1, 2, n, device="cuda")
    a, b = (B.AdamW([start.clone(), start.clone()], [grad.clone(), grad.clone()]) for _ in range(2))
    for bad in ([grad.bfloat16(), grad], [grad * 3, grad[1:]], [grad * 3, a.params[1]]):     # a type, a size, an overlap
        with pytest.raises((TypeError, ValueError, B.ConvError)):
            a.step(bad)
        a.step()
        b.step()
        for x, y in zip(a.params + a.m + a.v, b.params + b.m + b.v):
            assert torch.equal(x, y)
