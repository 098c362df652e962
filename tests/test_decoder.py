"""The feature decoder's buffers, without a GPU."""
import pytest
import torch

from differentiable_tile_gaussian_amd import decoder


def test_buffers_after_a_failed_allocation(monkeypatch):
    """An allocation that fails leaves the decoder able to try again with the same rows."""
    net = decoder.FeatureDecoder(32, 64, 12, blocks=2, device="cpu")
    net._reserve(100)
    real, left = torch.empty, [5]

    def empty(*a, **k):
        left[0] -= 1
        if left[0] == 0:
            raise torch.OutOfMemoryError("no memory")
        return real(*a, **k)
    monkeypatch.setattr(torch, "empty", empty)
    with pytest.raises(torch.OutOfMemoryError):
        net._reserve(300)
    net._reserve(300)
    sized = [net.h, net.u, net.f, net.y, net.du, net.da, net.dh, *net.h8, *net.a8, *net.z8, *net.u8]
    assert all(t.shape[0] == 300 for t in sized) and all(r.numel() == 300 for r in net.rstd)
