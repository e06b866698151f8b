"""Every tensor of a call has to be on one GPU, the current one, and a caller's
workspace has to be memory of that GPU.  Without a GPU: stand-ins that have a
tensor's type, shape and place."""
import pytest
import torch

from cnn_convolution_forward_amd import binding as B


class Fake:
    is_cuda = True

    def __init__(self, shape, dtype=torch.float32, index=0, dense=True):
        self.shape, self.dtype, self.index, self.dense = torch.Size(shape), dtype, index, dense
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")
        self.is_cuda = index >= 0

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.dense

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 4

    def data_ptr(self):
        return 0x1000


@pytest.mark.parametrize("index", [1, -1])
def test_tensors_of_another_device_are_refused(index, monkeypatch):
    x = Fake((2, 5, 8))
    with pytest.raises(ValueError, match="gate"):
        B._ld(Fake((2, 5, 8), index=index), x.shape, x, "gate")
    with pytest.raises(ValueError, match="decay"):
        B._dense(Fake((8,), index=index), (8,), torch.float32, "decay", 0)
    with pytest.raises(ValueError, match="offsets"):
        B.make_seq(Fake((5, 8)), Fake((3,), torch.int32, index), 5)
    with pytest.raises(ValueError, match="workspace"):
        B._workspace(Fake((1 << 20,), index=index), 0, x)
    row = lambda i=0: [Fake((10,), index=i), Fake((10,))]
    with pytest.raises(ValueError, match="grads"):
        B.AdamW(row(), [Fake((10,)), Fake((10,), index=index)], row(), row())
    with pytest.raises(ValueError, match="m must"):
        B.AdamW(row(), row(), row(index), row())
    with pytest.raises(ValueError, match="grad_scale"):
        B.AdamW(row(), row(), row(), row(), grad_scale=Fake((1,), index=index))
    monkeypatch.setattr(B, "_queries", (lambda: 0, lambda d: 0x5000 + d))
    assert B._stream_of(x) == 0x5000
    with pytest.raises(ValueError, match="current device"):
        B._stream_of(Fake((1,), index=index))


def test_workspace_is_memory_of_its_size():
    """An expanded tensor has more elements than memory."""
    x = Fake((2, 5, 8))
    with pytest.raises(ValueError, match="workspace"):
        B._workspace(Fake((1 << 20,), dense=False), 0, x)
    assert B._workspace(Fake((100,)), 0, x)[:2] == (0x1000, 400)
    assert B._workspace(None, 0, x) == (None, 0, None)
