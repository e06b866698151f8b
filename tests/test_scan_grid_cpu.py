"""The recurrence's grid: within what a launch can hold for every batch that the
entry points accept, with a place for every sequence.  scan_grid.h is host
arithmetic, so it is compiled and called here."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from cnn_convolution_forward_amd import binding as B

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "cnn_convolution_forward_amd", "csrc")
SOURCE = """
#include "scan_grid.h"
extern "C" void grid(int B, int nct, int per, long long through, long long *out) {
    const convfwd::ScanGrid g = convfwd::scan_grid(B, nct, per, through);
    out[0] = g.groups, out[1] = g.nb, out[2] = g.size;
}
"""
LIMIT = 1 << 23         # (rows/64 + B) * ceil(C/64) stays below it


@pytest.fixture(scope="module")
def grid(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("grid")
    (d / "g.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "g.so"), str(d / "g.cpp")], check=True)
    f = ctypes.CDLL(str(d / "g.so")).grid

    def call(B_, T, C, channels, tokens, rows=None):
        """Of equal sequences, or of a packed batch of `rows` rows."""
        f.argtypes = [ctypes.c_int] * 3 + [ctypes.c_longlong, ctypes.POINTER(ctypes.c_longlong)]
        out = (ctypes.c_longlong * 3)()
        nct, per = -(-C // channels), max(1, -(-T // tokens))
        total = 0 if rows is None or per == 1 else rows // tokens + B_
        f(B_, nct, per, total, out)
        return nct, per, total, list(out)

    return call


def _check(got, B_):
    nct, per, total, (groups, nb, size) = got
    assert 0 < size * 512 < 1 << 32, got
    assert groups % nct == 0 and groups <= max(64, nct)
    if total:
        assert size == nct * total
    else:
        assert size == groups * nb * per
        assert groups // nct * nb >= B_          # batches g = 0 .. G-1 hold g, g + G, ..., g + (nb-1) G: all below G nb


@pytest.mark.parametrize("B_,T,C", [(65, 8_000_000, 1), (65, 1 << 22, 1), (127, 4_000_000, 1), (64, (1 << 23) - 64, 1), (1, (1 << 29) - 128, 64),
                                    (2, (1 << 28) - 128, 64), (4193, 127_000, 3), (33, 1 << 23, 65), (1 << 21, 64, 1),
                                    (1, 64, 1 << 20), (300, 1600, 1 << 18)])
def test_accepted_edges_can_be_launched(grid, B_, T, C):
    accepted = (B_ * T // 64 + B_) * -(-C // 64) < LIMIT and B_ * T < 1 << 30
    assert (B.conv_scan_bwd_workspace_bytes(B.SeqParams(0, B_, T, C, None, 0)) > 0) == accepted
    if accepted:
        for channels in (64, 128):
            for tokens in (64, 128):
                _check(grid(B_, T, C, channels, tokens), B_)


def test_accepted_batches_can_be_launched(grid):
    rng, n = random.Random(3), 0
    while n < 2000:
        B_ = int(2 ** rng.uniform(0, 21))
        C = int(2 ** rng.uniform(0, 14))
        most = min((1 << 30) - 1, (LIMIT // -(-C // 64) - B_) * 64)          # rows about the limit
        if most < B_:
            continue
        T = max(1, int(most * rng.uniform(0.9, 1.0)) // B_)
        rows = B_ * T
        seq = B.SeqParams(0, B_, T, C, None, 0)
        if not B.conv_scan_bwd_workspace_bytes(seq):
            continue
        n += 1
        channels, tokens = rng.choice((64, 128)), rng.choice((64, 128))
        _check(grid(B_, T, C, channels, tokens), B_)
        _check(grid(B_, T, C, channels, tokens, rows), B_)


def test_one_workgroup_too_many_is_refused():
    """2^23 workgroups of 512 threads: the recurrence refuses the batch on the host."""
    X, G, I, Y, D, H, WS = (0x100000000000 * i for i in range(1, 8))
    seq = B.SeqParams(0, 1, ((1 << 23) - 1) * 64, 64, None, 0)
    call = lambda s: B.conv_scan_fwd(s, 8.0, X, 64, G, 64, I, 64, D, None, Y, 64, H, None, WS, 1)
    assert B.conv_scan_fwd_workspace_bytes(seq) == 0 and call(seq) == 4
    assert B.conv_scan_bwd(seq, 8.0, X, 64, G, 64, I, 64, D, H, Y, 64, None, WS, 64, WS * 2, 64, WS * 3, 64, D * 5, None, WS * 4, 1) == 4
    less = B.SeqParams(0, 1, ((1 << 23) - 2) * 64, 64, None, 0)
    assert B.conv_scan_fwd_workspace_bytes(less) > 0 and call(less) == 6         # only its workspace is too small


def test_batches_with_rows_to_fill_leave_room_for_a_workgroup(grid):
    """CONV_SEQ_FILL takes at least one workgroup more: the batch that leaves no room is refused."""
    full, off = (1 << 23) - 1, 0x100000000000                  # = 47 * 178481
    seq = lambda fill, B_: B.SeqParams(fill, B_, 1, 47 * 64, off, 0)
    assert B.conv_scan_fwd_workspace_bytes(seq(0, 178481)) == 0        # no workspace: one chunk each
    call = lambda s: B.conv_scan_fwd(s, -1.0, None, 64, None, 64, None, 64, off * 2, None, None, 64, None, None, None, 0)
    assert call(seq(0, 178481)) == 2 and call(seq(B.SEQ_FILL, 178481)) == 4 and call(seq(B.SEQ_FILL, 178480)) == 2      # 2: the scale
    for B_ in (178480, 178479, 89240, 59493):
        nct, per, total, (groups, nb, size) = grid(B_, 1, 47 * 64, 64, 128, 0)
        assert size < full or B_ * nct == full
