"""Shared features, served weights and clipping in the decoder, the pipeline and the example, against
64-bit forms and automatic differentiation."""
import math

import numpy as np
import pytest
import torch

from tests import more_ref as more
from tests.test_gpu_decoder import plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from differentiable_tile_gaussian_amd import gs as _gs
    return _gs


def off(a, b):
    return float((a.cpu().double() - b).norm() / b.norm())


def mx4_values(w):
    return torch.from_numpy(more.mx4_decode(*more.mx4_encode(w.cpu().double().numpy())))


@pytest.mark.parametrize("rows,entries,width,hidden,outputs,blocks", [(1000, 40, 32, 64, 12, 1), (333, 500, 35, 80, 59, 2)])
def test_table_gradients_against_automatic_differentiation(gs, rows, entries, width, hidden, outputs, blocks):
    """As the decoder's own gradients: 8-bit roundings, independent over a sum, 2^-3 of the norm."""
    print("table", rows, entries, width, flush=True)
    from differentiable_tile_gaussian_amd.decoder import FeatureDecoder, FeatureTable
    g = torch.Generator().manual_seed(rows)
    net, table = FeatureDecoder(width, hidden, outputs, blocks, seed=rows), FeatureTable(entries, width, scale=0.7, seed=rows)
    index = torch.randint(0, entries, (rows,), generator=g)
    base, dy = (torch.randn(rows, outputs, generator=g).cuda() for _ in range(2))
    y = net.forward(table.forward(index.cuda()), base)
    table.backward(net.backward(dy))
    p64 = {k: (net.w16[k] if v.dim() == 2 else v).cpu().double() for k, v in net.parameters.items()}
    t64 = table.parameters["table"].cpu().double().requires_grad_()
    y64 = plain(p64, 0.7 * t64[index], base.cpu().double(), blocks)
    (y64 * dy.cpu().double()).sum().backward()
    assert off(y, y64.detach()) < 2.0 ** -4
    assert off(table.grads["table"], t64.grad) < 2.0 ** -3
    table.forward(index[:100].int().cuda())                                  # fewer rows, the other type
    table.backward(torch.ones(100, width, device="cuda"))
    want = torch.zeros(entries).index_add_(0, index[:100], torch.full((100,), float(np.float32(0.7))))
    assert torch.allclose(table.grads["table"].cpu(), want[:, None].expand(-1, width), rtol=1e-6, atol=0)


@pytest.mark.parametrize("rows,width,hidden,outputs,blocks", [(1000, 32, 64, 12, 1), (333, 35, 80, 59, 2), (64, 256, 512, 48, 1), (50, 48, 64, 5, 0)])
def test_served_decoder(gs, rows, width, hidden, outputs, blocks):
    """The network of the 4-bit weights' values; what is between its layers is within 2^-4 of its own in 8
    bits, and over a sum of many such within 2^-4 of the norm."""
    print("served", rows, width, hidden, outputs, blocks, flush=True)
    from differentiable_tile_gaussian_amd.decoder import FeatureDecoder, ServedDecoder
    g = torch.Generator().manual_seed(rows)
    net = FeatureDecoder(width, hidden, outputs, blocks, seed=rows)
    for v in net.parameters.values():
        if v.dim() == 1:
            v.add_(0.1 * torch.randn(v.shape, generator=g).cuda())
    x, base = (torch.randn(rows, c, generator=g).cuda() for c in (width, outputs))
    served = ServedDecoder(net)
    p64 = {k: mx4_values(v) if v.dim() == 2 else v.cpu().double() for k, v in net.parameters.items()}
    want = plain(p64, x.cpu().double(), base.cpu().double(), blocks)
    assert off(served.forward(x, base), want) < 2.0 ** -4
    assert off(served.forward(x), want - base.cpu().double()) < 2.0 ** -4
    assert torch.equal(served.forward(x[:7], base[:7]), served.forward(x, base)[:7])


def test_pipeline_clips_before_the_update(gs):
    from differentiable_tile_gaussian_amd import scenes
    from differentiable_tile_gaussian_amd.pipeline import Pipeline
    scene = scenes.random_scene(3, 1500, 1)
    cam = gs.make_camera(scenes.identity_camera(96, 96, 110.0))
    params = torch.from_numpy(scene.params).cuda()
    target = torch.rand(3, 96, 96, generator=torch.Generator().manual_seed(4)).cuda()
    # fixed-point sums: the two pipelines have the same gradients bit for bit
    one, two = (Pipeline(params, 1, 96, 96, cfg=gs.GsConfig(gs.GS_GRAD_SUMS_FIXED)) for _ in range(2))
    one.forward(cam)
    one.backward(cam, target)
    grads = one.planar(one.grads)
    norm = math.sqrt(float(grads.double().square().sum()))
    extra = torch.full((7,), 3.0 * norm / math.sqrt(7.0), device="cuda")   # with it the norm is sqrt(10) times as large
    assert abs(float(one.clip(norm, [extra])) - math.sqrt(10.0) * norm) < 1e-6 * norm
    want = grads.double() / math.sqrt(10.0)
    assert bool(((one.planar(one.grads).double() - want).abs() <= want.abs() * 2.0 ** -22).all())
    assert torch.allclose(extra.double(), torch.full_like(extra, 3.0 * norm / math.sqrt(70.0)).double(), rtol=1e-6)
    two.step(cam, target, max_grad_norm=norm / 2)
    got = two.planar(two.grads)
    assert bool(((got.double() - grads.double() / 2).abs() <= grads.double().abs() * 2.0 ** -23).all())
    # the update is Adam's on the clipped gradient: its moments say so
    assert torch.allclose(two.planar(two.m), got * 0.1, rtol=1e-5, atol=0)
    three = Pipeline(params, 1, 96, 96, cfg=gs.GsConfig(gs.GS_GRAD_SUMS_FIXED))
    three.step_views([cam, cam], [target, target], max_grad_norm=norm * 2)
    assert abs(float(three.grad_norm) - norm) < 1e-4 * norm


@pytest.mark.parametrize("kw", [dict(codebook=50, max_norm=0.5, serve=True), dict(max_norm=1e9), dict(codebook=5000)])
def test_the_example_runs(gs, kw):
    import examples.train_decoder as ex
    losses = ex.train(gaussians=2000, steps=4, size=64, **kw)
    assert len(losses) == 4 + bool(kw.get("serve")) and all(math.isfinite(x) for x in losses)
