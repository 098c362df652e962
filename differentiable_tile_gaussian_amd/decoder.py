"""A network that decodes a feature row per Gaussian into some of its parameters.

Residual feed-forward blocks over the rows and a linear head, every operator a library call
(gs_rmsnorm_*, gs_linear_*, gs_mx8_*; gs_lookup_* for rows that Gaussians share, gs_clip_grads before an
update, gs_mx4_* to serve the trained network); torch holds the buffers.  Per block, with h the residual
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


class FeatureTable:
    """Feature rows that Gaussians share (a codebook): forward(index) gives a decoder its rows, times
    `scale`, and backward(dx) takes their gradient back to the table.  parameters and grads: "table",
    [entries][width] float32.  A Gaussian whose index is outside the table has a row of zeros."""

    def __init__(self, entries, width, scale=1.0, device="cuda", seed=0):
        self.entries, self.width, self.scale, self.device = entries, width, scale, device
        g = torch.Generator().manual_seed(seed)
        self.parameters = {"table": torch.randn(entries, width, generator=g).to(device)}
        self.grads = {"table": torch.zeros_like(self.parameters["table"])}
        self.rows = -1

    def forward(self, index):
        """index [rows] (int32 or int64) -> [rows][width] bfloat16, overwritten by the next call."""
        rows = index.shape[0]
        if rows != self.rows:
            self.rows = -1   # until both are there
            self.x = torch.empty((rows, self.width), dtype=torch.bfloat16, device=self.device)
            self.ws = gs.workspace(gs.GS_WS_LOOKUP_BWD, n=rows, W=self.width, H=self.entries, device=self.device)
            self.rows = rows
        self.index = index
        gs.gs_lookup_fwd(self.parameters["table"], index, self.x, scale=self.scale)
        return self.x

    def backward(self, dx):
        """dx [rows][width] (float32 or bfloat16): fills grads for the last forward's index."""
        gs.gs_lookup_bwd(dx, self.index, self.grads["table"], self.ws, scale=self.scale)


class ServedDecoder:
    """A trained FeatureDecoder's forward pass with its weights in 4 bits (MX4), an eighth of their
    float32 size.  Between its layers there are 8 bits (MX8), written by the norm and by the first
    layer of a block as the next layer reads them; nothing is kept for a backward pass.  It serves the
    network as it was when this was made: weights, biases and norms are copies, which refresh()
    renews after further training."""

    def __init__(self, net):
        self.net, self.rows = net, -1
        self.w4, self.vectors = {}, {}
        for name, v in net.parameters.items():
            if v.dim() == 2:
                self.w4[name] = gs.mx4_empty(*v.shape, v.device)
            else:
                self.vectors[name] = torch.empty_like(v)
        self.refresh()

    def refresh(self):
        """Takes the network's present parameters, into the buffers that are there."""
        for name, v in self.net.parameters.items():
            if v.dim() == 2:
                gs.gs_mx4_pack(v, self.w4[name])
            else:
                self.vectors[name].copy_(v.detach())

    def _reserve(self, rows):
        if rows == self.rows:
            return
        self.rows = -1   # until all of them are there
        n, dev = self.net, self.net.device
        self.h, self.f = (torch.empty((rows, n.width), dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.a8, self.u8 = gs.mx8_empty(rows, n.width, dev), gs.mx8_empty(rows, n.hidden, dev)
        self.y = torch.empty((rows, n.outputs), device=dev)
        self.rows = rows

    def forward(self, x, base=None):
        """As FeatureDecoder.forward."""
        self._reserve(x.shape[0])
        n, p, w = self.net, self.vectors, self.w4
        branch = None
        for i in range(n.blocks):
            gs.gs_rmsnorm_fwd(x if i == 0 else self.h, p[f"norm.{i}"], EPS, self.a8, residual=branch, h=self.h)
            gs.gs_linear_fwd(self.a8, w[f"w1.{i}"], self.u8, bias=p[f"b1.{i}"], act="silu")
            gs.gs_linear_fwd(self.u8, w[f"w2.{i}"], self.f, bias=p[f"b2.{i}"])
            branch = self.f
        gs.gs_rmsnorm_fwd(self.h if n.blocks else x, p["norm.head"], EPS, self.a8, residual=branch)
        gs.gs_linear_fwd(self.a8, w["w3"], self.y, bias=p["b3"], residual=base)
        return self.y


class GradientClip:
    """Clipping by the global norm of gradients in buffers that stay where they are (a decoder's
    and a table's grads, with others): calling it scales all of them by min(1, max_norm / norm) and
    returns the norm (device tensor of one value, overwritten by the next call)."""

    def __init__(self, tensors, max_norm):
        self.lists, self.max_norm = gs.Matrices(tensors), max_norm
        device = self.lists.tensors[0].device if self.lists.tensors else "cuda"
        self.norm = torch.zeros(1, device=device)
        self.ws = gs.workspace(gs.GS_WS_CLIP_GRADS, device=device)

    def __call__(self):
        gs.gs_clip_grads(self.lists, self.max_norm, self.norm, self.ws)
        return self.norm


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
