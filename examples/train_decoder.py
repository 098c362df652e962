"""Trains a feature decoder through the rasteriser: every Gaussian has a learned feature row,
a network decodes the rows into colour coefficients, and the gradient of the image loss comes
back through the blend and the colour planes into the network and the features.

    python examples/train_decoder.py [--gaussians N] [--steps K]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from differentiable_tile_gaussian_amd import gs, scenes  # noqa: E402
from differentiable_tile_gaussian_amd.decoder import FeatureDecoder, planes_to_rows, rows_to_planes  # noqa: E402
from differentiable_tile_gaussian_amd.pipeline import Pipeline  # noqa: E402

COLOUR = 11   # the first colour plane


def train(gaussians=20_000, steps=100, width=32, hidden=64, sh_degree=1, size=256, seed=0, log=None):
    """Fits the colours of a random scene, seen from one camera, starting from grey; returns
    the losses of all steps."""
    scene = scenes.random_scene(seed, gaussians, sh_degree)
    cam = gs.make_camera(scenes.identity_camera(size, size, 1.2 * size))
    params = torch.from_numpy(scene.params).cuda()
    target = Pipeline(params, sh_degree, size, size).forward(cam).clone()

    count = 3 * (sh_degree + 1) ** 2
    base = torch.zeros(gaussians, count, device="cuda")
    base[:, :3] = 0.5
    pl = Pipeline(params, sh_degree, size, size)
    net = FeatureDecoder(width, hidden, count, seed=seed)
    features = torch.randn(gaussians, width, generator=torch.Generator().manual_seed(seed)).cuda()
    learned = [features, *net.parameters.values()]
    adam = torch.optim.Adam(learned, lr=5e-3)
    dy = torch.empty(gaussians, count, device="cuda")
    losses = []
    for step in range(steps):
        rows_to_planes(net.forward(features, base), pl.params, COLOUR)
        pl.forward(cam)
        pl.backward(cam, target)
        # the loss's gradient is that of a mean over the image: scaled to the rows' own size
        planes_to_rows(pl.grads, gaussians, COLOUR, count, out=dy).mul_(3.0 * size * size)
        features.grad = net.backward(dy).float()
        for name, p in net.parameters.items():
            p.grad = net.grads[name]
        adam.step()
        net.refresh()
        losses.append(float(pl.loss[0]))
        if log and step % 10 == 0:
            log(f"step {step}: loss {losses[-1]:.5f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--gaussians", type=int, default=20_000)
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    out = train(a.gaussians, a.steps, log=lambda s: print(s, flush=True))
    print(f"loss {out[0]:.5f} -> {out[-1]:.5f} in {len(out)} steps")
