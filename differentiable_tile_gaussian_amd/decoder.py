"""A network that decodes a feature row per Gaussian into some of its parameters.

Residual feed-forward blocks over the rows and a linear head, every operator a library call
(gs_rmsnorm_*, gs_linear_*, gs_mx8_*); torch holds the buffers.  Per block, with h the residual
stream and f the block's branch:

    h = h + f_previous;  a = norm(h);  u = silu(a W1^T + b1);  f = u W2^T + b2

and at the end h = h + f, a = norm(h), y = a W3^T + b3 + base.  What the backward pass reads
again is kept in 8 bits (MX8): a and u (the layers' inputs), the pre-activations and h; the two
layers that follow read a and u in that form in the forward pass too, so that the gradients
are those of what was computed.  The residual stream and the gradients between layers are
bfloat16, weights' gradients float32.
"""
from __future__ import annotations

import torch

from . import gs

EPS = 1e-6


class FeatureDecoder:
    """parameters and grads: name -> float32 tensor (w1.i [hidden][width], b1.i, w2.i
    [width][hidden], b2.i, norm.i, and w3, b3, norm.head).  Change parameters in place, then
    call refresh()."""

    def __init__(self, width, hidden, outputs, blocks=1, device="cuda", seed=0):
        self.width, self.hidden, self.outputs, self.blocks, self.device = width, hidden, outputs, blocks, device
        g = torch.Generator().manual_seed(seed)

        def weight(n, k, scale=1.0):
            return (torch.randn(n, k, generator=g) * (scale * k ** -0.5)).to(device)
        p = {}
        for i in range(blocks):
            p[f"norm.{i}"] = torch.ones(width, device=device)
            p[f"w1.{i}"], p[f"b1.{i}"] = weight(hidden, width), torch.zeros(hidden, device=device)
            p[f"w2.{i}"], p[f"b2.{i}"] = weight(width, hidden), torch.zeros(width, device=device)
        p["norm.head"] = torch.ones(width, device=device)
        p["w3"], p["b3"] = weight(outputs, width, 0.1), torch.zeros(outputs, device=device)
        self.parameters = p
        self.grads = {k: torch.zeros_like(v) for k, v in p.items()}
        self.w16 = {}
        self.rows = -1
        self.refresh()

    def refresh(self):
        """Rounds the weights to the bfloat16 the products read."""
        for k, v in self.parameters.items():
            if v.dim() == 2:
                self.w16[k] = v.to(torch.bfloat16)

    def _reserve(self, rows):
        if rows == self.rows:
            return
        self.rows = -1   # until all of them are there
        w, n, dev, bf = self.width, self.hidden, self.device, torch.bfloat16

        def buf(cols, dtype=bf):
            return torch.empty((rows, cols), dtype=dtype, device=dev)
        count = self.blocks + 1
        self.h = buf(w)
        self.h8 = [gs.mx8_empty(rows, w, dev) for _ in range(count)]
        self.a8 = [gs.mx8_empty(rows, w, dev) for _ in range(count)]
        self.rstd = [torch.empty(rows, device=dev) for _ in range(count)]
        self.z8 = [gs.mx8_empty(rows, n, dev) for _ in range(self.blocks)]
        self.u8 = [gs.mx8_empty(rows, n, dev) for _ in range(self.blocks)]
        self.u, self.f = buf(n), buf(w)
        self.y = buf(self.outputs, torch.float32)
        self.du, self.da, self.dh = buf(n), buf(w), buf(w)
        self.ws = torch.empty(max(gs.gs_workspace_bytes(gs.GS_WS_LINEAR_BWD, rows, W=w, H=n),
                                  gs.gs_workspace_bytes(gs.GS_WS_LINEAR_BWD, rows, W=n, H=w),
                                  gs.gs_workspace_bytes(gs.GS_WS_LINEAR_BWD, rows, W=w, H=self.outputs),
                                  gs.gs_workspace_bytes(gs.GS_WS_RMSNORM_BWD, rows, W=w)),
                              dtype=torch.uint8, device=dev)
        self.rows = rows

    def forward(self, x, base=None):
        """x [rows][width] (float32 or bfloat16) -> [rows][outputs] float32, plus base if given
        (float32, the same size).  The result is overwritten by the next call."""
        self._reserve(x.shape[0])
        p, w = self.parameters, self.w16
        branch = None
        for i in range(self.blocks + 1):
            last = i == self.blocks
            gs.gs_rmsnorm_fwd(x if i == 0 else self.h, p["norm.head" if last else f"norm.{i}"], EPS, self.a8[i],
                              self.rstd[i], residual=branch, h=self.h, ckpt=self.h8[i])
            if last:
                break
            gs.gs_linear_fwd(self.a8[i], w[f"w1.{i}"], self.u, bias=p[f"b1.{i}"], act="silu", z=self.z8[i])
            gs.gs_mx8_pack(self.u, self.u8[i])
            gs.gs_linear_fwd(self.u8[i], w[f"w2.{i}"], self.f, bias=p[f"b2.{i}"])
            branch = self.f
        gs.gs_linear_fwd(self.a8[-1], w["w3"], self.y, bias=p["b3"], residual=base)
        return self.y

    def backward(self, dy):
        """dy [rows][outputs] (float32 or bfloat16): fills grads and returns the gradient of x
        (bfloat16, overwritten by the next call) for the last forward."""
        p, w, g = self.parameters, self.w16, self.grads
        gs.gs_linear_bwd(dy, self.a8[-1], w["w3"], self.da, g["w3"], g["b3"], self.ws)
        gs.gs_rmsnorm_bwd(self.da, self.h8[-1], p["norm.head"], self.rstd[-1], self.dh, g["norm.head"], self.ws)
        for i in reversed(range(self.blocks)):
            gs.gs_linear_bwd(self.dh, self.u8[i], w[f"w2.{i}"], self.du, g[f"w2.{i}"], g[f"b2.{i}"], self.ws)
            gs.gs_linear_bwd(self.du, self.a8[i], w[f"w1.{i}"], self.da, g[f"w1.{i}"], g[f"b1.{i}"], self.ws, act="silu",
                             z=self.z8[i])
            gs.gs_rmsnorm_bwd(self.da, self.h8[i], p[f"norm.{i}"], self.rstd[i], self.dh, g[f"norm.{i}"], self.ws,
                              dres=self.dh)
        return self.dh


def planes_to_rows(blocked, n, first, count, out=None):
    """Planes first .. first + count - 1 of a blocked parameter array ([groups][P][64]) as rows
    [n][count]."""
    rows = blocked[:, first:first + count].transpose(1, 2).reshape(-1, count)[:n]
    return rows.contiguous() if out is None else out.copy_(rows)


def rows_to_planes(rows, blocked, first):
    """Writes rows [n][count] into planes first .. of a blocked parameter array."""
    n, count = rows.shape
    full = n // 64
    blocked[:full, first:first + count].copy_(rows[:full * 64].view(full, 64, count).transpose(1, 2))
    if n % 64:
        blocked[full, first:first + count, :n % 64].copy_(rows[full * 64:].t())
