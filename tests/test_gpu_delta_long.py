"""The gated delta rule cut into segments with heads of more than 96 channels, where the joining takes four waves and a
segment's sums two workgroups, and many value heads to a key head; against the float64 reference with test_gpu_delta's bounds."""
import numpy as np
import pytest

from cnn_convolution_forward_amd import binding as B
from test_gpu_delta import Case, _whole
from test_gpu_delta_sizes import INF, NAN, _forward, _held

pytestmark = pytest.mark.gpu


def _is_cut(dt, lens, H, Hv, dk, dv, packed, f):
    """Whether a batch takes more workspace than its blocks do: the segments' matrices."""
    code = 1 if dt == "bf16" else 0
    par = B.DeltaParams(H, Hv, dk, dv, 1, 1.0, 1e-6)
    n = sum(lens)
    seq = B.SeqParams(code, len(lens), max(lens), Hv * dv, 64 if packed else None, n)
    blocks = n // 64 + len(lens) if packed else len(lens) * -(-max(lens) // 64)
    return f(seq, par) > blocks * f(B.SeqParams(code, 1, 64, Hv * dv, None, 0), par)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens,H,Hv,dk,dv,packed,unit", [
    ([1100], 1, 1, 128, 128, False, True), ([1500, 0, 700], 1, 2, 113, 127, True, True), ([1300], 1, 2, 100, 33, False, False),
    ([64 * 9] * 2, 1, 1, 97, 128, False, True), ([1, 2000, 65], 1, 1, 127, 101, True, False)])
def test_wide_heads_in_segments(dt, lens, H, Hv, dk, dv, packed, unit):
    for f in (B.conv_delta_fwd_workspace_bytes, B.conv_delta_bwd_workspace_bytes):
        assert _is_cut(dt, lens, H, Hv, dk, dv, packed, f)
    c = Case(dt, lens, H, Hv, dk, dv, packed=packed, unit=unit, slices=3 * packed, g=lambda r, s: -np.exp(r.uniform(-9, -2, s)))
    first = _whole(c)
    again = B.delta_rule(*c.data(), s0=c.s0, with_states=True, **c.opts())
    assert all(bool((a == b).all()) for a, b in zip(first[:2], again[:2]))


@pytest.mark.parametrize("dt,unit,bad", [("bf16", True, INF), ("f32", False, INF), ("f32", True, NAN)])
def test_values_that_are_not_finite_in_segments(dt, unit, bad):
    """In the first, a middle and the last segment: in front of them, and beside them in other columns and heads, all stays right."""
    assert _is_cut(dt, [1100], 1, 2, 32, 40, False, B.conv_delta_fwd_workspace_bytes)
    c = Case(dt, [1100], 1, 2, 32, 40, unit=unit, seed=39, g=lambda r, s: -np.exp(r.uniform(-9, -2, s)))
    clean = _forward(c)
    for token in (5, 200, 500, 1099):
        for name, head in (("q", 0), ("k", 0), ("v", 1), ("g", 1), ("b", 0)):
            _held(c, clean, name, token, head, bad, token // 32 * 32)


def test_what_is_not_cut():
    assert not _is_cut("bf16", [448], 1, 1, 128, 128, False, B.conv_delta_fwd_workspace_bytes)
    assert not _is_cut("bf16", [1000] * 8, 4, 16, 128, 128, False, B.conv_delta_fwd_workspace_bytes)


@pytest.mark.parametrize("dt,H,Hv,dk,dv", [("bf16", 1, 16, 32, 32), ("f32", 2, 16, 24, 20), ("bf16", 3, 24, 64, 40)])
def test_many_value_heads_to_a_key_head(dt, H, Hv, dk, dv):
    _whole(Case(dt, [100] * 2, H, Hv, dk, dv))
