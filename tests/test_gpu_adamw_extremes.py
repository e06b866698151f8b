"""The AdamW step at the ends of float32's range: 8-bit blocks whose scale has no
normal reciprocal, or is at the cut below which a block is stored as zeros, and
an epsilon below the smallest normal number."""
import numpy as np
import pytest
import torch

from cnn_convolution_forward_amd import binding as B

pytestmark = pytest.mark.gpu


def _between_neighbours(x, scale, got, top, power):
    """`got` is the value of one of the two codes around x, or of x's own: codes q = 0 .. top stand for
    scale (q / top)^power.  2^-20 of slack on the place, for the roots that find it."""
    place = top * (x / scale) ** (1 / power)
    q = np.rint(top * (got / scale) ** (1 / power))
    slack = 2.0 ** -20 * top
    return (q >= np.floor(place - slack)) & (q <= np.ceil(place + slack)) & (np.abs(got - scale * (q / top) ** power) <= 2.0 ** -20 * got + 1e-44)


@pytest.mark.parametrize("largest", [2.0 ** 62.4, 2.0 ** -57.9, 2.0 ** -58.0])
def test_scales_from_gradients(largest):
    """v = g^2 / 1000: the largest |g| near the one whose square is still finite, and at the cut at v = 2^-126."""
    n = 1024
    rng = np.random.default_rng(7)
    g = np.float32(largest * np.exp(rng.uniform(-3, 0, n)) * rng.choice([-1, 1], n))
    g[::256] = np.float32(largest)
    opt = B.AdamW([torch.zeros(n, device="cuda")], [torch.from_numpy(g).cuda()], bits=8, seed=3)
    opt.step()
    m, v = (t[0].double().cpu().numpy() for t in opt.state_values())
    m1 = np.float64(np.float32(g * np.float32(1 - 0.9)))
    v1 = np.float64(np.float32(np.float32(g * g) * np.float32(1 - 0.999)))
    sm, sv = (np.repeat(np.abs(a).reshape(-1, 256).max(1), 256) for a in (m1, v1))
    assert np.array_equal(np.repeat(opt.m_scale[0].double().cpu().numpy(), 256), sm)
    kept = sv >= 2.0 ** -126
    assert np.array_equal(np.repeat(opt.v_scale[0].double().cpu().numpy(), 256), np.where(kept, sv, 0))
    assert np.all(np.sign(m[m != 0]) == np.sign(m1[m != 0])) and np.all(_between_neighbours(np.abs(m1), sm, np.abs(m), 127, 2))
    assert np.all(v[~kept] == 0) and np.all(_between_neighbours(v1[kept], sv[kept], v[kept], 255, 4))
    assert np.all(opt.m[0].cpu().numpy()[::256] == 127) and (not kept.all() or np.all(opt.v[0].cpu().numpy()[::256] == 255))


@pytest.mark.parametrize("largest", [2.0 ** 123, 2.0 ** 125.5, 2.0 ** 126.5, 2.0 ** 127.9])
def test_scales_without_a_normal_reciprocal(largest):
    """Moments up to 2^127.9, which a state carries on: 1/scale is below the normal numbers from 2^126 on."""
    n = 512
    rng = np.random.default_rng(8)
    g = torch.zeros(n, device="cuda")
    q = torch.from_numpy(rng.integers(-127, 128, n).astype(np.int8)).cuda()
    r = torch.from_numpy(rng.integers(0, 256, n).astype(np.uint8)).cuda()
    q[::256], r[::256] = 127, 255
    opt = B.AdamW([torch.zeros(n, device="cuda")], [g], [q], [r], bits=8, m_scale=[torch.full((2,), largest, device="cuda")],
                  v_scale=[torch.full((2,), largest, device="cuda")])
    before = opt.state_values()
    opt.step()
    for old, new, factor, top, power in zip(before, opt.state_values(), (0.9, 0.999), (127, 255), (2, 4)):
        now = np.float64(old[0].cpu().numpy() * np.float32(factor))
        scale = np.abs(now).max()
        got = new[0].double().cpu().numpy()
        assert np.all(_between_neighbours(np.abs(now), scale, np.abs(got), top, power)), (top, largest)
        assert np.all(np.abs(got[::256]) == scale) and np.all(np.sign(got[got != 0]) == np.sign(now[got != 0]))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-40, 1e-45, 1e-60])
def test_zero_moments_with_a_tiny_epsilon(bits, eps):
    """0 / eps is 0 for every eps above 0; the update of other elements does not notice it."""
    n = 300
    g = torch.zeros(n, device="cuda")
    g[::3] = 0.5
    opt = B.AdamW([torch.ones(n, device="cuda")], [g], bits=bits, eps=eps, lr=0.25)
    opt.step()
    p = opt.params[0]
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[::3] = False
    assert bool((p[rest] == 1).all())
    assert float((p[::3] - 0.75).abs().max()) <= 16 * 2.0 ** -23
