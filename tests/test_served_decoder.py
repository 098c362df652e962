"""What the 4-bit decoder computes from.  Without a GPU the library's calls stand in as recorders of
the parameters that reach them."""
import pytest
import torch

from differentiable_tile_gaussian_amd import decoder


@pytest.fixture
def calls(monkeypatch):
    """Values of the weights, biases and norms that a forward pass hands to the library."""
    seen = []

    class Packed:
        def __init__(self, rows, cols):
            self.values = torch.full((rows, cols), float("nan"))

    monkeypatch.setattr(decoder.gs, "mx4_empty", lambda rows, cols, device: Packed(rows, cols))
    monkeypatch.setattr(decoder.gs, "gs_mx4_pack", lambda x, q: q.values.copy_(x))
    monkeypatch.setattr(decoder.gs, "gs_rmsnorm_fwd", lambda x, weight, eps, y, **k: seen.append(weight.clone()))
    monkeypatch.setattr(decoder.gs, "gs_linear_fwd",
                        lambda x, w, y, bias=None, **k: seen.extend((w.values.clone(), bias.clone())))
    return seen


def forward(calls, served, rows=5):
    calls.clear()
    served.forward(torch.zeros(rows, served.net.width))
    return list(calls)


def same(a, b):
    return len(a) == len(b) and all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("blocks", [0, 2])
def test_it_serves_one_state_of_the_network(calls, blocks):
    """Steps of training behind its construction change nothing that it computes from, until refresh()."""
    net = decoder.FeatureDecoder(32, 64, 12, blocks=blocks, device="cpu")
    served = decoder.ServedDecoder(net)
    first = forward(calls, served)
    assert len(first) == 3 * (2 * blocks + 1) - blocks
    for p in net.parameters.values():
        p.add_(1.0)
    assert same(forward(calls, served), first)
    served.refresh()
    assert same(forward(calls, served), [v + 1.0 for v in first])


def test_a_refresh_keeps_its_buffers(calls):
    """A captured forward pass reads the buffers that were there: a refresh writes into them."""
    net = decoder.FeatureDecoder(32, 64, 12, device="cpu")
    served = decoder.ServedDecoder(net)
    packed, vectors = dict(served.w4), dict(served.vectors)
    net.parameters["w3"] = net.parameters["w3"] + 1.0          # replaced, not changed in place
    net.parameters["b3"] = net.parameters["b3"] + 1.0
    served.refresh()
    assert all(served.w4[k] is v for k, v in packed.items()) and all(served.vectors[k] is v for k, v in vectors.items())
    assert torch.equal(packed["w3"].values, net.parameters["w3"]) and torch.equal(vectors["b3"], net.parameters["b3"])


@pytest.mark.gpu
def test_its_results_are_those_of_one_state():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(7)
    net = decoder.FeatureDecoder(48, 96, 20, blocks=2, seed=3)
    x, base = (torch.randn(300, c, generator=g).cuda() for c in (48, 20))
    served = decoder.ServedDecoder(net)
    before = served.forward(x, base).clone()
    for p in net.parameters.values():
        p.add_(0.2 * torch.randn(p.shape, generator=g).cuda())
    assert torch.equal(served.forward(x, base), before)
    served.refresh()
    after = served.forward(x, base).clone()
    assert torch.equal(after, decoder.ServedDecoder(net).forward(x, base)) and not torch.equal(after, before)
