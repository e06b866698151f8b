"""Layer norm without a GPU: the reference's gradient against central differences,
and every refusal of the entry points and helpers (all pointers here are fake)."""
import numpy as np
import pytest
import torch

import norm_reference as R
from cnn_convolution_forward_amd import binding as B

X, Y, W, D, M, K, WS = (0x10000000 * i for i in range(1, 8))


@pytest.mark.parametrize("n,C", [(1, 1), (3, 2), (4, 9)])
def test_reference_gradient(n, C):
    """Central differences along random directions: third derivatives of O(1) data leave less than 1e-7."""
    rng = np.random.default_rng(C)
    x, w, b, dy = rng.standard_normal((n, C)), rng.standard_normal(C), rng.standard_normal(C), rng.standard_normal((n, C))
    f = lambda x, w, b: (R.norm(x, w, b, 0.1)[0][0] * dy).sum()
    (_, mean, rstd), _ = R.norm(x, w, b, 0.1)
    grads = R.norm_grad(x, w, dy, mean, rstd)[0]
    for i, g in enumerate(grads):
        d = rng.standard_normal(g.shape)
        up, dn = [x, w, b], [x, w, b]
        up[i], dn[i] = up[i] + 1e-5 * d, dn[i] - 1e-5 * d
        num = (f(*up) - f(*dn)) / 2e-5
        assert abs(num - (g * d).sum()) <= 1e-6 * (np.abs(g * d).sum() + 1), i


def _f(dtype=1, rows=10, C=24, eps=1e-5, x=X, ldx=24, w=W, b=D, y=Y, ldy=24, m=M, k=K):
    return B.conv_norm_fwd(dtype, rows, C, eps, x, ldx, w, b, y, ldy, m, k)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(dtype=2), 2), (dict(dtype=257), 2), (dict(rows=-1), 2), (dict(C=0), 2),
    (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2), (dict(ldx=23), 2), (dict(ldy=1), 2),
    (dict(x=X + 1), 2), (dict(w=W + 2), 2), (dict(m=M + 1), 2), (dict(rows=1 << 30), 4), (dict(C=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21), 4),
    (dict(y=X), 5), (dict(y=X + 48 * 9 + 46), 5), (dict(m=K), 5), (dict(m=W), 5), (dict(k=Y), 5), (dict(y=D), 5)])
def test_forward_refusals(kw, status):
    assert _f(**kw) == status


def test_backward_refusals():
    need = B.conv_norm_bwd_workspace_bytes(1, 10, 24)
    assert need > 0 and B.conv_norm_bwd_workspace_bytes(3, 10, 24) == 0 and B.conv_norm_bwd_workspace_bytes(1, -1, 24) == 0
    dy, dx, dw, db = (X + 0x01000000 * i for i in range(1, 5))

    def f(dtype=1, rows=10, C=24, x=X, ldx=24, w=W, m=M, k=K, dy=dy, dx=dx, lddx=24, dw=dw, db=db, ws=WS, n=need):
        return B.conv_norm_bwd(dtype, rows, C, x, ldx, w, m, k, dy, 24, dx, lddx, dw, db, ws, n)

    assert f(x=None) == 1 and f(m=None) == 1 and f(k=None) == 1 and f(dy=None) == 1 and f(dx=None) == 1
    assert f(dtype=-1) == 2 and f(ldx=5) == 2 and f(lddx=23) == 2 and f(dw=dw + 1) == 2 and f(C=0) == 2
    assert f(rows=1 << 30) == 4
    assert f(ws=None) == 6 and f(n=need - 1) == 6 and f(ws=WS + 4) == 6
    assert f(dx=X) == 5 and f(dx=dy + 4) == 5 and f(dw=W) == 5 and f(db=dw + 8) == 5 and f(ws=X) == 5 and f(dx=M) == 5


def test_no_rows_forward_does_nothing():
    assert _f(rows=0, x=None, y=None, m=None, k=None) == 0


def test_helpers_refuse():
    x = torch.zeros(5, 8)
    with pytest.raises(ValueError):
        B.layer_norm(x)                                  # not on a GPU
    with pytest.raises(ValueError):
        B.layer_norm(torch.zeros(2, 3, 4, 5))
    with pytest.raises(TypeError):
        B.layer_norm(x.double())
