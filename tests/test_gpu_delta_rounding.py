"""bf16 outputs of the gated delta rule: products of 22 bits and one rounding at the end.  The bounds are those of
float32 outputs (delta_reference), and half a step of bf16 on top: 2**-8 of a value at most.  Values that all but
cancel show anything coarser."""
import pytest

import delta_reference as R
from cnn_convolution_forward_amd import binding as B
from test_gpu_delta import Case, _check, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,H,Hv,dk,dv,packed,unit", [
    ([200], 1, 2, 16, 40, False, True), ([130] * 3, 2, 2, 16, 32, False, False), ([70, 0, 1, 129], 1, 2, 24, 31, True, True),
    ([700], 1, 1, 16, 64, False, True), ([150], 1, 2, 128, 128, False, True)])
def test_whole_sequences_are_rounded_once(lens, H, Hv, dk, dv, packed, unit):
    c = Case("bf16", lens, H, Hv, dk, dv, packed=packed, unit=unit, seed=21, g=lambda r, s: -r.uniform(0, 0.05, s))
    y, _ = B.delta_rule(*c.data(), s0=c.s0, **c.opts())
    y = _np(y).reshape(c.off[-1], Hv, dv)
    grow = 2 * dk ** 0.5 if max(lens) > 448 else 1.0          # as in test_gpu_delta
    for i, h, hk, r, q, k, v, g, b, _, _ in c.sequences():
        ref, hist = R.forward(q, k, v, g, b, _np(c.s0)[i, h], c.scale)
        _check(y[r, h], ref, R.forward_bounds(q, k, v, g, b, hist, c.scale, c.ku(), False, grow)[0], True, "sequence %d head %d" % (i, h))


def test_a_float32_call_rounded_at_the_end():
    """The same values as float32 tensors: what the bf16 call returns is, but for a few values next to a border, that result rounded."""
    c = Case("bf16", [256] * 2, 2, 2, 64, 64, seed=4)
    q, k, v, g, b = c.data()
    y, sT = B.delta_rule(*c.data(), s0=c.s0, **c.opts())
    y32, sT32 = B.delta_rule(q.float(), k.float(), v.float(), g, b, s0=c.s0, **c.opts())
    # Both are within 2**-20 of a sum's usual size before they are rounded.  Borders lie 2**-8 of a value apart or more, so a value of
    # that size falls to the other side once in 2**11, one 2**n times smaller 2**n times as often; those are 2**-n of all, and
    # with n up to 11 they add up to less than 12 * 2**-11.
    assert float((y != y32.bfloat16()).float().mean()) < 12 * 2.0 ** -11
    assert float((sT - sT32).norm()) <= 2.0 ** -18 * float(sT32.norm())
