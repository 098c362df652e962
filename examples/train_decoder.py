"""Trains a feature decoder through the rasteriser: every Gaussian has a learned feature row,
a network decodes the rows into colour coefficients, and the gradient of the image loss comes
back through the blend and the colour planes into the network and the features.  With
--codebook E the Gaussians share E rows, with --clip X the gradients are clipped to the global
norm X, and --serve renders the trained network's colours from weights in 4 bits.

    python examples/train_decoder.py [--gaussians N] [--steps K] [--codebook E] [--clip X] [--serve]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from differentiable_tile_gaussian_amd import gs, scenes  # noqa: E402
from differentiable_tile_gaussian_amd.decoder import (FeatureDecoder, FeatureTable, GradientClip, ServedDecoder,  # noqa: E402
                                                      planes_to_rows, rows_to_planes)
from differentiable_tile_gaussian_amd.pipeline import Pipeline  # noqa: E402

COLOUR = 11   # the first colour plane


def train(gaussians=20_000, steps=100, width=32, hidden=64, sh_degree=1, size=256, seed=0, log=None, codebook=0,
          max_norm=None, serve=False):
    """Fits the colours of a random scene, seen from one camera, starting from grey; returns
    the losses of all steps, and with serve then that of the image from 4-bit weights."""
    scene = scenes.random_scene(seed, gaussians, sh_degree)
    cam = gs.make_camera(scenes.identity_camera(size, size, 1.2 * size))
    params = torch.from_numpy(scene.params).cuda()
    target = Pipeline(params, sh_degree, size, size).forward(cam).clone()

    count = 3 * (sh_degree + 1) ** 2
    base = torch.zeros(gaussians, count, device="cuda")
    base[:, :3] = 0.5
    pl = Pipeline(params, sh_degree, size, size)
    net = FeatureDecoder(width, hidden, count, seed=seed)
    generator = torch.Generator().manual_seed(seed)
    table = FeatureTable(codebook, width, seed=seed) if codebook else None
    if table:
        features = table.parameters["table"]
        index = torch.randint(0, codebook, (gaussians,), generator=generator).cuda()
    else:
        features = torch.randn(gaussians, width, generator=generator).cuda()
    learned = [features, *net.parameters.values()]
    adam = torch.optim.Adam(learned, lr=5e-3)
    dy = torch.empty(gaussians, count, device="cuda")
    features.grad = table.grads["table"] if table else torch.zeros_like(features)
    clip = GradientClip([features.grad, *net.grads.values()], max_norm) if max_norm else None
    losses = []
    for step in range(steps):
        rows_to_planes(net.forward(table.forward(index) if table else features, base), pl.params, COLOUR)
        pl.forward(cam)
        pl.backward(cam, target)
        # the loss's gradient is that of a mean over the image: scaled to the rows' own size
        planes_to_rows(pl.grads, gaussians, COLOUR, count, out=dy).mul_(3.0 * size * size)
        dx = net.backward(dy)
        if table:
            table.backward(dx)
        else:
            features.grad.copy_(dx)
        for name, p in net.parameters.items():
            p.grad = net.grads[name]
        if clip:
            clip()
        adam.step()
        net.refresh()
        losses.append(float(pl.loss[0]))
        if log and step % 10 == 0:
            log(f"step {step}: loss {losses[-1]:.5f}")
    if serve:
        y = ServedDecoder(net).forward(table.forward(index) if table else features, base)
        rows_to_planes(y, pl.params, COLOUR)
        pl.forward(cam)
        pl.backward(cam, target)
        losses.append(float(pl.loss[0]))
        if log:
            log(f"from 4-bit weights: loss {losses[-1]:.5f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--gaussians", type=int, default=20_000)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--codebook", type=int, default=0)
    ap.add_argument("--clip", type=float, default=None)
    ap.add_argument("--serve", action="store_true")
    a = ap.parse_args()
    out = train(a.gaussians, a.steps, log=lambda s: print(s, flush=True), codebook=a.codebook, max_norm=a.clip, serve=a.serve)
    print(f"loss {out[0]:.5f} -> {out[a.steps - 1]:.5f} in {a.steps} steps")
