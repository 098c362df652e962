"""The feature decoder: its gradients against 64-bit automatic differentiation of the same
network without 8-bit storage, its training through the rasteriser, and the plane layout."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def plain(params, x, base, blocks):
    """The network in float64."""
    def norm(h, w):
        return h * (h.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * w
    h, f = x, 0.0
    for i in range(blocks):
        h = h + f
        z = norm(h, params[f"norm.{i}"]) @ params[f"w1.{i}"].t() + params[f"b1.{i}"]
        f = z * torch.sigmoid(z) @ params[f"w2.{i}"].t() + params[f"b2.{i}"]
    return norm(h + f, params["norm.head"]) @ params["w3"].t() + params["b3"] + base


@pytest.mark.parametrize("rows,width,hidden,outputs,blocks", [(1000, 32, 64, 12, 1), (333, 35, 80, 59, 2), (64, 256, 512, 48, 1)])
def test_gradients_against_automatic_differentiation(cuda, rows, width, hidden, outputs, blocks):
    """An e4m3 value is within 2^-4 of its own; the errors of a sum of many are independent, so
    a gradient tensor as a whole is expected within 2^-4 / sqrt(3) (uniform errors) of a few
    such roundings: the bound is 2^-3 of its norm, and the result's is 2^-4."""
    print("decoder", rows, width, hidden, outputs, blocks, flush=True)
    from differentiable_tile_gaussian_amd.decoder import FeatureDecoder
    g = torch.Generator().manual_seed(rows)
    net = FeatureDecoder(width, hidden, outputs, blocks, seed=rows)
    for k, v in net.parameters.items():
        if v.dim() == 1:
            v.add_(0.1 * torch.randn(v.shape, generator=g).cuda())
    net.refresh()
    x, base, dy = (torch.randn(rows, c, generator=g).cuda() for c in (width, outputs, outputs))
    y = net.forward(x, base)
    dx = net.backward(dy)
    p64 = {k: (net.w16[k] if v.dim() == 2 else v).cpu().double().requires_grad_() for k, v in net.parameters.items()}
    x64 = x.cpu().double().requires_grad_()
    y64 = plain(p64, x64, base.cpu().double(), blocks)
    (y64 * dy.cpu().double()).sum().backward()

    def off(a, b):
        return float((a.cpu().double() - b).norm() / b.norm())
    assert off(y, y64.detach()) < 2.0 ** -4
    assert off(dx, x64.grad) < 2.0 ** -3
    for k, v in net.grads.items():
        assert off(v, p64[k].grad) < 2.0 ** -3, k


def test_training_through_the_rasteriser(cuda):
    import examples.train_decoder as ex
    losses = ex.train(gaussians=3000, steps=60, size=96)
    print("decoder losses", losses[0], losses[-1])
    assert losses[-1] < 0.7 * losses[0]


@pytest.mark.parametrize("n", [1, 63, 64, 200])
def test_rows_and_planes(cuda, n):
    from differentiable_tile_gaussian_amd import gs
    from differentiable_tile_gaussian_amd.decoder import planes_to_rows, rows_to_planes
    planar = torch.randn(23, n, device="cuda")
    blocked = gs.to_blocked(planar, 1)
    assert torch.equal(planes_to_rows(blocked, n, 11, 12), planar[11:].t())
    rows = torch.randn(n, 12, device="cuda")
    rows_to_planes(rows, blocked, 11)
    back = gs.from_blocked(blocked, n, 1)
    assert torch.equal(back[11:], rows.t()) and torch.equal(back[:11], planar[:11])
