"""Layer norm on the GPU against norm_reference (float64), element by element
within the bounds derived there: widths around every change of layout, odd ones,
column slices, constant and shifted rows, infinities and NaN, streams, graphs, and rows beyond
2^31 elements.  Outputs are poisoned with NaN first."""
import numpy as np
import pytest
import torch

import norm_reference as R
from cnn_convolution_forward_amd import binding as B
from seq_reference import tol

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAN = float("nan")


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check(got, ref, err, bf16, label):
    got = _np(got).reshape(ref.shape)
    bad = ~(np.abs(got - ref) <= tol(ref, err, bf16))
    assert not bad.any(), (label, int(bad.sum()), got[bad][:3], ref[bad][:3], tol(ref, err, bf16)[bad][:3])


def _make(seed, n, C, dt):
    rng = np.random.default_rng(seed)
    t = lambda a, k=torch.float32: torch.from_numpy(np.asarray(a)).to(k).cuda()
    x = t(rng.standard_normal((n, C)) * rng.uniform(0.1, 3, (n, 1)) + rng.standard_normal((n, 1)), DT[dt])
    return x, t(1 + rng.standard_normal(C) * 0.3), t(rng.standard_normal(C)), t(rng.standard_normal((n, C)), DT[dt])


def _both(x, w, b, dy, eps, dt, label, **out):
    """Forward and backward of rows x against the reference; returns all outputs."""
    C = x.shape[-1]
    got = B.layer_norm(x, w, b, eps=eps, with_stats=True, out=out.get("y"))
    xs = _np(x).reshape(-1, C)
    wn, bn = (np.full(C, d) if p is None else _np(p) for p, d in ((w, 1.0), (b, 0.0)))
    ref, err = R.norm(xs, wn, bn, np.float64(np.float32(eps)))
    for i, name in enumerate(("y", "mean", "rstd")):
        _check(got[i], ref[i], err[i], dt == "bf16" and i == 0, (label, name))
    mean, rstd = got[1:]
    grads = B.layer_norm_backward(x, w, dy, mean, rstd, out=out.get("dx"))
    ref, err = R.norm_grad(xs, wn, _np(dy).reshape(-1, C), _np(mean).reshape(-1), _np(rstd).reshape(-1))
    for i, name in enumerate(("dx", "dweight", "dbias")):
        _check(grads[i], ref[i], err[i], dt == "bf16" and i == 0, (label, name))
    return got, grads


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 2, 7, 16, 63, 64, 65, 127, 128, 129, 250, 256, 257, 511, 513, 999, 1024, 1025, 2047, 2048, 2049, 4095,
                               4096, 4097, 8192, 8193, 20001])
def test_widths(C, dt):
    for n in (1, 3, 37):
        _both(*_make(C * 10 + n, n, C, dt), 1e-5, dt, (C, n))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,C", [(1, 8194), (700, 8200), (530, 12288), (300, 16379), (530, 16384), (300, 16385), (3, 40000)])
def test_wide_rows(n, C, dt):
    """Rows that take a workgroup of 1024 threads, and wider ones; more of them than workgroups too."""
    _both(*_make(n + C, n, C, dt), 1e-5, dt, (n, C))


@pytest.mark.parametrize("dt,n,C", [("bf16", 40000, 128), ("f32", 70001, 33), ("bf16", 9001, 520), ("f32", 2500, 2048), ("bf16", 1300, 9000)])
def test_many_rows(dt, n, C):
    """More rows than the workgroups take in one turn."""
    _both(*_make(n, n, C, dt), 1e-6, dt, (n, C))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C,pad", [(128, 8), (99, 3), (640, 1), (2049, 5), (9001, 2)])
def test_column_slices_and_no_parameters(C, pad, dt):
    """(B, T, C) as columns of wider tensors, outputs too; what lies between stays as it was."""
    x, w, b, dy = _make(C, 15, C, dt)
    wide = [torch.full((3, 5, C + 2 * pad), 77.0, dtype=DT[dt], device="cuda") for _ in range(4)]
    cut = [t[..., pad:pad + C] for t in wide]
    cut[0].copy_(x.reshape(3, 5, C))
    cut[1].copy_(dy.reshape(3, 5, C))
    for t in cut[2:]:
        t.fill_(NAN)
    for p in ((w, b), (None, None), (w, None)):
        _both(cut[0], *p, cut[1], 1e-5, dt, (C, p[0] is None), y=cut[2], dx=cut[3])
    for t in wide:
        assert bool((t[..., :pad] == 77).all()) and bool((t[..., pad + C:] == 77).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_constant_and_shifted_rows(dt):
    """A constant row has no variance: y is the bias up to the mean's rounding over sqrt(eps).  Shifted rows keep what the
    shift left of them."""
    x, w, b, dy = _make(5, 6, 384, dt)
    x[0], x[1] = 0, 3.25
    x[2] += 100
    x[3] *= 1e-20
    x[4] = x[4] * 1e15
    _both(x, w, b, dy, 1e-5, dt, "shifted")
    y = B.layer_norm(torch.zeros_like(x), w, b, eps=0.0)
    assert bool(torch.isnan(y).all())          # 0 / 0: no variance and no eps


@pytest.mark.parametrize("C", [100, 700, 3001, 9000])
def test_non_finite_rows_stay_their_own(C):
    x, w, b, dy = _make(C, 9, C, "f32")
    clean = B.layer_norm(x, w, b)
    for bad, row in ((NAN, 1), (float("inf"), 4), (-float("inf"), 8)):
        x[row, C // 2] = bad
    y, mean, rstd = B.layer_norm(x, w, b, with_stats=True)
    keep = [0, 2, 3, 5, 6, 7]
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[[1, 4, 8]]).all())
    dx, dw, db = B.layer_norm_backward(x, w, dy, mean, rstd)
    assert bool(torch.isfinite(dx[keep]).all()) and bool(torch.isnan(dx[[1, 4, 8]]).all())
    assert bool(torch.isnan(dw).all()) and bool(torch.isfinite(db).all())


def test_same_bits_in_any_batch():
    for C in (128, 777, 5000):
        x, w, b, dy = _make(C, 700, C, "bf16")
        y, mean, rstd = B.layer_norm(x, w, b, with_stats=True)
        dx = B.layer_norm_backward(x, w, dy, mean, rstd)[0]
        for i in (0, 399, 699):
            yi, mi, ri = B.layer_norm(x[i:i + 1], w, b, with_stats=True)
            assert torch.equal(yi, y[i:i + 1]) and torch.equal(mi, mean[i:i + 1])
            assert torch.equal(B.layer_norm_backward(x[i:i + 1], w, dy[i:i + 1], mi, ri)[0], dx[i:i + 1])


def test_no_rows():
    x, w = torch.empty(0, 50, device="cuda"), torch.ones(50, device="cuda")
    y, mean, rstd = B.layer_norm(x, w, with_stats=True)
    assert y.shape == (0, 50) and mean.shape == (0,)
    dx, dw, db = B.layer_norm_backward(x, w, x, mean, rstd)
    assert dx.shape == (0, 50) and bool((dw == 0).all()) and bool((db == 0).all())


def test_refusals_leave_outputs():
    x, w, b, dy = _make(1, 4, 64, "f32")
    for bad in (lambda: B.layer_norm(x, w[:63], b), lambda: B.layer_norm(x, w.bfloat16(), b), lambda: B.layer_norm(x, w.cpu(), b),
                lambda: B.layer_norm_backward(x, w, dy[:3], x[:, 0].contiguous(), x[:, 0].contiguous()),
                lambda: B.layer_norm_backward(x, w, dy, x[:, 0], x[:, 0].contiguous())):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(B.ConvError):
        B.layer_norm(x, w, b, eps=-1.0)
    with pytest.raises(B.ConvError):
        B.layer_norm(x, w, b, out=x)
    with pytest.raises(B.ConvError):
        B.layer_norm_backward(x, w, dy, x[:, 0].contiguous(), x[:, 1].contiguous(), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_other_stream_and_captured_graph():
    """A captured forward and backward, replayed with other inputs and eager work between."""
    x, w, b, dy = _make(2, 300, 640, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            y, m, k = B.layer_norm(x, w, b, with_stats=True)
            g = B.layer_norm_backward(x, w, dy, m, k)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, m, k = B.layer_norm(x, w, b, with_stats=True)
        g = B.layer_norm_backward(x, w, dy, m, k)
    for i in range(4):
        x.copy_(_make(20 + i, 300, 640, "bf16")[0])
        graph.replay()
        torch.cuda.synchronize()
        y2, m2, k2 = B.layer_norm(x, w, b, with_stats=True)
        want = (y2, m2, k2) + B.layer_norm_backward(x, w, dy, m2, k2)
        for a, c in zip((y, m, k) + tuple(g), want):
            assert torch.equal(a, c)


def test_rows_beyond_2_31_elements():
    """Three rows 1.1e9 elements apart."""
    C, ld = 300, 1_100_000_000
    big = [torch.empty(2 * ld + C, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x, y = (t.as_strided((3, C), (ld, 1)) for t in big)
    src, w, b, _ = _make(3, 3, C, "bf16")
    x.copy_(src)
    B.layer_norm(x, w, b, out=y)
    assert torch.equal(y, B.layer_norm(src, w, b))
