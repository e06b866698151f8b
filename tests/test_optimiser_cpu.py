"""The AdamW helper's handling of lists of tensors, without a GPU: stand-ins that
have a tensor's addresses and types, and a recorder in place of the entry point."""
import ctypes

import pytest
import torch

from cnn_convolution_forward_amd import binding as B


class Fake:
    """What the helper asks of a GPU tensor."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, address, n, dtype=torch.float32, index=0):
        self.address, self.n, self.dtype, self.index = address, n, dtype, index
        self.device = torch.device("cuda", index)

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def data_ptr(self):
        return self.address

    def get_device(self):
        return self.index


@pytest.fixture
def calls(monkeypatch):
    """What each conv_adamw_step call would have read: gradient type and addresses; `status` is returned."""
    seen, status = [], [0]

    def step(o, table, count, stream=None):
        seen.append((o.grad_dtype, [table[i].g for i in range(count)], o.step))
        return status[0]

    monkeypatch.setattr(B, "conv_adamw_step", step)
    monkeypatch.setattr(B, "_stream_of", lambda t: None)
    seen_status = lambda v: status.__setitem__(0, v)
    return seen, seen_status


def _optimiser():
    row = lambda k, dtype=torch.float32: [Fake(0x10000 * k + 0x1000 * i, 10 + i, dtype) for i in range(3)]
    return B.AdamW(row(1), row(2), row(3), row(4))


BAD = {
    "another type": [Fake(0x90000, 10, torch.bfloat16), Fake(0x91000, 11), Fake(0x92000, 12, torch.bfloat16)],
    "all of one type but a size": [Fake(0x90000, 10, torch.bfloat16), Fake(0x91000, 11, torch.bfloat16), Fake(0x92000, 9, torch.bfloat16)],
    "a size": [Fake(0x90000, 10), Fake(0x91000, 12), Fake(0x92000, 12)],
    "too few": [Fake(0x90000, 10)],
}


@pytest.mark.parametrize("kind", sorted(BAD))
def test_refused_gradients_leave_the_optimiser_as_it_was(calls, kind):
    seen, _ = calls
    opt = _optimiser()
    kept = list(opt.grads)
    with pytest.raises((TypeError, ValueError)):
        opt.step(BAD[kind])
    assert not seen and opt.steps == 0
    opt.step()
    assert seen == [(0, [g.address for g in kept], 1)]
    assert all(a is b for a, b in zip(opt.grads, kept)), "the gradients in use must be held"


def test_step_that_fails_keeps_the_gradients_before_it(calls):
    seen, status = calls
    opt = _optimiser()
    kept = list(opt.grads)
    status(5)
    with pytest.raises(B.ConvError):
        opt.step([Fake(0x90000 + 0x1000 * i, 10 + i, torch.bfloat16) for i in range(3)])
    status(0)
    opt.step()
    assert seen[0][0] == 1 and seen[1] == (0, [g.address for g in kept], 1) and opt.steps == 1
    assert all(a is b for a, b in zip(opt.grads, kept))


def test_gradients_of_another_type_are_taken_whole(calls):
    seen, _ = calls
    opt = _optimiser()
    new = [Fake(0x90000 + 0x1000 * i, 10 + i, torch.bfloat16) for i in range(3)]
    opt.step(iter(new))
    opt.step()
    assert seen == [(1, [g.address for g in new], 1), (1, [g.address for g in new], 2)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lengths", [(2, 4), (3, 2), (3,), (3, 3, 3), (0, 6)])
def test_state_values_needs_two_lists_of_all_tensors(bits, lengths, monkeypatch):
    """Six tensors in another split would take m for v."""
    row = lambda k, dtype=torch.float32: [Fake(0x10000 * k + 0x1000 * i, 10, dtype) for i in range(3)]
    one = lambda k: [Fake(0x10000 * k + 0x1000 * i, 1) for i in range(3)]
    kinds = (torch.float32, torch.float32) if bits == 32 else (torch.int8, torch.uint8)
    scales = {} if bits == 32 else {"m_scale": one(5), "v_scale": one(6)}
    opt = B.AdamW(row(1), row(2), row(3, kinds[0]), row(4, kinds[1]), bits=bits, **scales)
    monkeypatch.setattr(Fake, "copy_", lambda self, t: None, raising=False)
    monkeypatch.setattr(B, "conv_adamw_state_values", lambda *a: 0)
    monkeypatch.setattr(B, "_stream_of", lambda t: None)
    with pytest.raises(ValueError):
        opt.state_values(out=tuple([Fake(0x90000 + 0x1000 * i, 10) for i in range(n)] for n in lengths))
    good = (row(7), row(8))
    assert opt.state_values(out=good) is good
