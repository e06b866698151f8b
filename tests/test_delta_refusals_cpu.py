"""Heads that are not there, and heads without channels, are refused by the gated delta rule's helpers like any other shape."""
import pytest
import torch

from cnn_convolution_forward_amd import binding as B


@pytest.mark.parametrize("q,v", [((2, 5, 2, 0), (2, 5, 4, 6)), ((2, 5, 0, 8), (2, 5, 4, 6)), ((2, 5, 2, 8), (2, 5, 0, 6)), ((2, 5, 2, 8), (2, 5, 4, 0))])
def test_no_heads_or_channels(q, v):
    q, v = torch.zeros(q), torch.zeros(v)
    with pytest.raises(ValueError, match="head"):
        B.make_delta(q, v)
    with pytest.raises(ValueError, match="head"):
        B.make_delta(q[0], v[0], offsets=torch.tensor([0, 5], dtype=torch.int32), max_len=5)
    with pytest.raises(ValueError, match="head"):
        B.make_delta(q[:, 0], v[:, 0], step=True)
