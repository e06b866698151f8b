"""Layer norm and its gradients in float64, with bounds on the error of a float32
evaluation beside each value.

U = 2**-23 stands for one float32 operation, as in seq_reference.  A sum over a
row has at most 32 terms in a thread (one of every 256 in rows too wide for
that), and ten more steps to join threads.
"""
import numpy as np

from seq_reference import U


def depth(C):
    return 42 + C // 256


def norm(x, w, b, eps):
    """y, mean, rstd and their error bounds."""
    C = x.shape[1]
    mean = x.mean(1, keepdims=True)
    em = (depth(C) + 2) * U * np.abs(x).mean(1, keepdims=True)
    c = x - mean
    ec = em + U * np.abs(c)
    var = (c * c).mean(1, keepdims=True)
    ev = (2 * np.abs(c) * ec + ec * ec).mean(1, keepdims=True) + (depth(C) + 4) * U * var
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1 / np.sqrt(var + eps)
        er = rstd * (0.5 * ev / (var + eps) + 4 * U)
    y = c * rstd * w + b
    ey = np.abs(w) * (ec * rstd + np.abs(c) * er) + 3 * U * np.abs(c * rstd * w) + U * np.abs(y)
    return (y, mean[:, 0], rstd[:, 0]), (ey, em[:, 0], er[:, 0])


def norm_grad(x, w, dy, mean, rstd):
    """dx, dweight, dbias for the mean and rstd as given, and their error bounds."""
    n, C = x.shape
    k = rstd[:, None]
    h = (x - mean[:, None]) * k
    eh = 3 * U * np.abs(h)
    e = w * dy
    s0, s1 = e.mean(1, keepdims=True), (e * h).mean(1, keepdims=True)
    d = (depth(C) + 4) * U
    es0 = d * np.abs(e).mean(1, keepdims=True)
    es1 = (d * np.abs(e * h) + np.abs(e) * eh).mean(1, keepdims=True)
    dx = k * (e - s0 - h * s1)
    parts = np.abs(e) + np.abs(s0) + np.abs(h * s1)
    edx = k * (es0 + np.abs(h) * es1 + np.abs(s1) * eh + 5 * U * parts)
    # a group's own rows one after another (at most 512 workgroups), then the groups, then the workgroups
    r = (n // 512 + 1 + 16 + 64 + 10) * U
    return (dx, (dy * h).sum(0), dy.sum(0)), (edx, (np.abs(dy) * eh + (r + U) * np.abs(dy * h)).sum(0), r * np.abs(dy).sum(0))
