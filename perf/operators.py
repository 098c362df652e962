"""Cases, plain forms and inputs of the operators a network over Gaussians is made of.

Such a network maps one feature row per Gaussian (or per 16x16 image tile) to Gaussian
parameters and is trained through the rasteriser's parameter gradients.  Its operators:

  linear       y = act(x W^T + b) + r, optionally keeping x W^T + b in 8 bits
  linear_grad  the gradients of x, W and b, from 8-bit or bfloat16 checkpoints
  norm         h = x + r and its root-mean-square norm, in bfloat16 or 8 bits with scales
  norm_grad    the gradients of h and of the norm's weight
  pack         a matrix to 8 bits with scales and back

The 8-bit format (MX8): e4m3 elements, and for each 32 columns of a row one power-of-two
scale 2^e with the smallest e >= -126 for which the block's largest finite magnitude is at
most 448 2^e.

`run` computes an operator from elementary torch operations in 32 bits (`own` false) or by
the library's calls (`own` true); `exact` computes it from its definition in 64 bits.
"""
import math

import torch
import torch.nn.functional as F

own = False

EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu")
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu

# Rows: 1,024 is the smallest scene of the benchmark, 1,000,003 its one-million scene made
# ragged, 3,000,000 its 720p stress scene, 8,160 the 16x16 tiles of its 1920x1080 images.
# 59 is the number of parameters of a Gaussian at SH degree 3 and 48 its colour coefficients.
TILES = 8160


def _linear(rows, inner, outer, act="none", x8=False, ckpt=False, residual=False, f32=False):
    return {"op": "linear", "rows": rows, "inner": inner, "outer": outer, "act": act, "x8": x8, "ckpt": ckpt,
            "residual": residual, "f32": f32}


def _linear_grad(rows, inner, outer, act="none", ckpt=False, f32=False):
    return {"op": "linear_grad", "rows": rows, "inner": inner, "outer": outer, "act": act, "ckpt": ckpt, "f32": f32}


def _norm(rows, cols, residual=False, y8=False, ckpt=False, f32=False):
    return {"op": "norm", "rows": rows, "cols": cols, "residual": residual, "y8": y8, "ckpt": ckpt, "f32": f32}


def _norm_grad(rows, cols, ckpt=False, dres=False, f32=False):
    return {"op": "norm_grad", "rows": rows, "cols": cols, "ckpt": ckpt, "dres": dres, "f32": f32}


def _pack(rows, cols, f32=False):
    return {"op": "pack", "rows": rows, "cols": cols, "f32": f32}


def listed():
    return [
        # one image's appearance code through a wide layer when a single view is rendered
        {"name": "linear_view"} | _linear(1, 1024, 1024, "silu"),
        # a hidden layer over every Gaussian: 8-bit input from the norm, pre-activation kept in 8 bits
        {"name": "linear_gaussians"} | _linear(1_000_003, 128, 128, "silu", x8=True, ckpt=True),
        # the second layer of a wide block over the tiles of a 1080p image, with its residual
        {"name": "linear_tiles"} | _linear(TILES, 4096, 1024, x8=True, residual=True),
        # the output layer to the colour coefficients: float32 gradients from the rasteriser
        {"name": "linear_grad_colours"} | _linear_grad(100_003, 64, 48, f32=True),
        # the hidden layer over every Gaussian, backward from its 8-bit checkpoints
        {"name": "linear_grad_gaussians"} | _linear_grad(1_000_003, 128, 128, "silu", ckpt=True),
        # the first layer of the wide block over the tiles, backward from its 8-bit checkpoints
        {"name": "linear_grad_tiles"} | _linear_grad(TILES, 1024, 4096, "gelu", ckpt=True),
        # float32 features of the smallest scene: latency
        {"name": "norm_scene"} | _norm(1024, 64, y8=True, f32=True),
        # the residual stream of a large scene, kept in 8 bits beside the 8-bit norm
        {"name": "norm_gaussians"} | _norm(3_000_000, 128, residual=True, y8=True, ckpt=True),
        # a tile stream whose width is no multiple of 32
        {"name": "norm_grad_tiles"} | _norm_grad(TILES, 1000, dres=True),
        # the residual stream's gradient over every Gaussian, from its 8-bit checkpoint
        {"name": "norm_grad_gaussians"} | _norm_grad(1_000_003, 128, ckpt=True, dres=True),
        # parameter rows of every Gaussian (59 float32 values, an odd width)
        {"name": "pack_parameters"} | _pack(1_000_003, 59, f32=True),
        # a wide block's activations
        {"name": "pack_activations"} | _pack(TILES, 4096),
    ]


def _size(rng, low, high):
    """Log-uniform in [low, high]; every other one a multiple of 16 where that fits."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and n >= 16:
        n = n // 16 * 16
    return min(max(n, low), high)


def draw(rng):
    op = rng.choice(("linear", "linear_grad", "norm", "norm_grad", "pack"))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("linear", "linear_grad"):
        if rng.random() < 0.6:    # rows are Gaussians
            inner, outer = _size(rng, 3, 256), _size(rng, 3, 256)
            rows = _size(rng, 1, min(1_000_003, 1_000_003 * 256 // (inner + outer)))
        else:                     # rows are image tiles or views
            inner, outer = _size(rng, 256, 2048), _size(rng, 256, 4096)
            rows = _size(rng, 1, min(TILES, TILES * 4096 * 1024 // (inner * outer)))
        act = rng.choice(ACTS)
        if op == "linear":
            return _linear(rows, inner, outer, act, x8=flag(), ckpt=flag(), residual=flag(), f32=rng.random() < 0.25)
        return _linear_grad(rows, inner, outer, act, ckpt=flag(), f32=rng.random() < 0.25)
    if rng.random() < 0.6:
        cols = _size(rng, 3, 256)
        rows = _size(rng, 1, min(1_000_003, 1_000_003 * 128 // cols))
    else:
        cols = _size(rng, 256, 4096)
        rows = _size(rng, 1, min(4 * TILES, TILES * 4096 * 4 // cols))
    if op == "norm":
        return _norm(rows, cols, residual=flag(), y8=flag(), ckpt=flag(), f32=rng.random() < 0.25)
    if op == "norm_grad":
        return _norm_grad(rows, cols, ckpt=flag(), dres=flag(), f32=rng.random() < 0.25)
    return _pack(rows, cols, f32=flag())


# ---------------------------------------------------------------- the 8-bit format, plain

def quantise(v):
    """float32 [M][C] -> (e4m3 [M][C], e8m0 [M][ceil(C / 32)])."""
    m, c = v.shape
    nb = (c + 31) // 32
    b = F.pad(v, (0, nb * 32 - c)).view(m, nb, 32)
    top = torch.where(torch.isfinite(b), b, 0.0).abs().amax(-1)
    # the exponent field of the smallest 2^e with top <= 1.75 2^(e + 8)
    e = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(1, 254)
    q = (b * ((254 - e) << 23).view(torch.float32).unsqueeze(-1)).to(E4M3)
    return q.view(m, nb * 32)[:, :c], e.to(torch.uint8).view(E8M0)


def dequantise(q, s):
    return q.float() * s.float().repeat_interleave(32, dim=1)[:, :q.shape[1]]


def _pitched(q, s):
    """The same matrix with rows that start at multiples of 16 bytes."""
    m, c = q.shape
    store = torch.zeros((m, (c + 15) // 16 * 16), dtype=torch.uint8, device=q.device).view(E4M3)
    store[:, :c].view(torch.uint8).copy_(q.view(torch.uint8))
    return store[:, :c], s.contiguous()


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    def grads(m, c):
        # loss gradients per Gaussian: a third of the rows is outside the view, the others
        # spread over orders of magnitude around 1 / (3 W H)
        seen = torch.rand(m, 1, generator=g, device="cuda") > 1.0 / 3.0
        return normal(m, c) * torch.exp(normal(m, 1) - 13.0) * seen

    def stream(m, c):
        # features: columns of different spread around a small offset
        return normal(m, c) * torch.exp(0.5 * normal(1, c)) + normal(1, c, scale=0.2)

    op, m = case["op"], case["rows"]
    wide = torch.float32 if case["f32"] else torch.bfloat16
    s = {"case": case}
    if op in ("linear", "linear_grad"):
        k, n = case["inner"], case["outer"]
        s["w"] = normal(n, k, scale=k ** -0.5).bfloat16()
        x = stream(m, k)
        if op == "linear":
            s["b"] = normal(n, scale=0.1)
            s["x"] = _pitched(*quantise(x)) if case["x8"] else x.bfloat16()
            s["r"] = stream(m, n).to(wide) if case["residual"] else None
        else:
            z = normal(m, n, scale=1.5)
            s["x"] = _pitched(*quantise(x)) if case["ckpt"] else x.bfloat16()
            s["z"] = None if case["act"] == "none" else _pitched(*quantise(z)) if case["ckpt"] else z.bfloat16()
            s["dy"] = grads(m, n).to(wide)
        return s
    c = case["cols"]
    x = stream(m, c)
    if op == "pack":
        s["x"] = x.to(wide)
        return s
    s["w"] = 1.0 + normal(c, scale=0.2)
    if op == "norm":
        s["x"] = x.to(wide)
        s["r"] = stream(m, c).to(wide) if case["residual"] else None
    else:
        s["rstd"] = torch.rsqrt(x.square().mean(1) + EPS)
        s["h"] = _pitched(*quantise(x)) if case["ckpt"] else x.to(wide)
        s["dy"] = grads(m, c).to(wide)
        s["dres"] = grads(m, c).to(wide) if case["dres"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _values(t):
    return dequantise(*t) if isinstance(t, tuple) else t.float()


def _eight(v):
    q, s = quantise(v)
    return {"q": q, "scale": s}


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0.0).float()
    if act == "silu":
        g = 1.0 / (1.0 + torch.exp(-z))
        return g * (1.0 + z * (1.0 - g))
    c = 2.0 * math.sqrt(2.0 / math.pi)
    g = 1.0 / (1.0 + torch.exp(-c * (z + 0.044715 * z * z * z)))
    return g * (1.0 + z * (1.0 - g) * c * (1.0 + 3.0 * 0.044715 * z * z))


def _plain(s):
    case = s["case"]
    op = case["op"]
    wide = torch.float32 if case["f32"] else torch.bfloat16
    if op == "linear":
        z = _values(s["x"]) @ s["w"].float().t() + s["b"]
        y = _act(z, case["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        out = {"y": y.to(wide)}
        if case["ckpt"]:
            out["z"] = _eight(z)
        return out
    if op == "linear_grad":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _act_slope(_values(s["z"]), case["act"])
        return {"dx": (dz @ s["w"].float()).bfloat16(), "dw": (dz.t() @ _values(s["x"])).bfloat16(), "db": dz.sum(0)}
    if op == "norm":
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        y = h * rstd.unsqueeze(1) * s["w"]
        out = {"y": _eight(y) if case["y8"] else y.bfloat16(), "rstd": rstd}
        if s["r"] is not None:
            out["h"] = h.to(wide)
        if case["ckpt"]:
            out["ckpt"] = _eight(h)
        return out
    if op == "norm_grad":
        rstd = s["rstd"].unsqueeze(1)
        dy, xhat = s["dy"].float(), _values(s["h"]) * rstd
        u = dy * s["w"]
        dh = rstd * (u - xhat * (u * xhat).mean(1, keepdim=True))
        if s["dres"] is not None:
            dh = dh + s["dres"].float()
        return {"dh": dh.to(wide), "dw": (dy * xhat).sum(0)}
    q, e = quantise(s["x"].float())
    return {"q": q, "scale": e, "back": dequantise(q, e).bfloat16()}


# ---------------------------------------------------------------- the library's calls

def _library(s):
    from differentiable_tile_gaussian_amd import gs

    case = s["case"]
    op, m = case["op"], case["rows"]
    wide = torch.float32 if case["f32"] else torch.bfloat16

    def matrix(t):
        return gs.Mx8(*t) if isinstance(t, tuple) else t

    def empty(rows, cols, dtype):
        return torch.empty((rows, cols), dtype=dtype, device="cuda")

    def eight(t):
        return {"q": t.q, "scale": t.scales}

    if op == "linear":
        y = empty(m, case["outer"], wide)
        z = gs.mx8_empty(m, case["outer"]) if case["ckpt"] else None
        gs.gs_linear_fwd(matrix(s["x"]), s["w"], y, bias=s["b"], act=case["act"], residual=s["r"], z=z)
        return {"y": y} if z is None else {"y": y, "z": eight(z)}
    if op == "linear_grad":
        if "ws" not in s:
            s["ws"] = gs.workspace(gs.GS_WS_LINEAR_BWD, n=m, W=case["inner"], H=case["outer"])
        dx = empty(m, case["inner"], torch.bfloat16)
        dw = empty(case["outer"], case["inner"], torch.bfloat16)
        db = torch.empty(case["outer"], dtype=torch.float32, device="cuda")
        gs.gs_linear_bwd(s["dy"], matrix(s["x"]), s["w"], dx, dw, db, s["ws"], act=case["act"], z=matrix(s["z"]))
        return {"dx": dx, "dw": dw, "db": db}
    if op == "norm":
        c = case["cols"]
        y = gs.mx8_empty(m, c) if case["y8"] else empty(m, c, torch.bfloat16)
        h = empty(m, c, wide) if s["r"] is not None else None
        ckpt = gs.mx8_empty(m, c) if case["ckpt"] else None
        rstd = torch.empty(m, dtype=torch.float32, device="cuda")
        gs.gs_rmsnorm_fwd(s["x"], s["w"], EPS, y, rstd, residual=s["r"], h=h, ckpt=ckpt)
        out = {"y": eight(y) if case["y8"] else y, "rstd": rstd}
        if h is not None:
            out["h"] = h
        if ckpt is not None:
            out["ckpt"] = eight(ckpt)
        return out
    if op == "norm_grad":
        c = case["cols"]
        if "ws" not in s:
            s["ws"] = gs.workspace(gs.GS_WS_RMSNORM_BWD, n=m, W=c)
        dh = empty(m, c, wide)
        dw = torch.empty(c, dtype=torch.float32, device="cuda")
        gs.gs_rmsnorm_bwd(s["dy"], matrix(s["h"]), s["w"], s["rstd"], dh, dw, s["ws"], dres=s["dres"])
        return {"dh": dh, "dw": dw}
    q = gs.mx8_empty(m, case["cols"])
    back = empty(m, case["cols"], torch.bfloat16)
    gs.gs_mx8_pack(s["x"], q)
    gs.gs_mx8_unpack(q, back)
    return eight(q) | {"back": back}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- the work of one pass

def _bytes(rows, cols, kind):
    if kind == 1:
        return rows * (cols + (cols + 31) // 32)
    return rows * cols * kind


def work(case):
    op, m = case["op"], case["rows"]
    wide = 4 if case["f32"] else 2
    if op == "linear":
        k, n = case["inner"], case["outer"]
        b = _bytes(m, k, 1 if case["x8"] else 2) + _bytes(m, n, wide) * (1 + case["residual"])
        b += (_bytes(m, n, 1) if case["ckpt"] else 0) + 2 * n * k + 4 * n
        return {"bytes": b, "flops": 2 * m * n * k}
    if op == "linear_grad":
        k, n = case["inner"], case["outer"]
        kept = 1 if case["ckpt"] else 2
        b = _bytes(m, n, wide) + _bytes(m, k, kept) + _bytes(m, k, 2) + 4 * n * k + 4 * n
        b += 0 if case["act"] == "none" else _bytes(m, n, kept)
        return {"bytes": b, "flops": 4 * m * n * k}
    c = case["cols"]
    if op == "norm":
        b = _bytes(m, c, wide) * (3 if case["residual"] else 1) + _bytes(m, c, 1 if case["y8"] else 2)
        b += (_bytes(m, c, 1) if case["ckpt"] else 0) + 4 * m + 4 * c
        return {"bytes": b, "flops": 5 * m * c}
    if op == "norm_grad":
        b = _bytes(m, c, wide) * (3 if case["dres"] else 2) + _bytes(m, c, 1 if case["ckpt"] else wide) + 4 * m + 8 * c
        return {"bytes": b, "flops": 10 * m * c}
    return {"bytes": _bytes(m, c, wide) + _bytes(m, c, 1) + _bytes(m, c, 2), "flops": 3 * m * c}


# ---------------------------------------------------------------- the definition in 64 bits

def _grid64(v):
    """The nearest e4m3 value (ties to the even one) of |v| <= 448, in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3.0)
    return torch.round(v / step) * step


def _eight64(v):
    m, c = v.shape
    block = torch.arange(c, device=v.device) // 32
    top = torch.zeros((m, (c + 31) // 32), dtype=torch.float64, device=v.device)
    top.scatter_reduce_(1, block.expand(m, c), v.abs(), "amax")
    frac, e = torch.frexp(top / 448.0)
    e = torch.where(frac == 0.5, e - 1, e)
    e = torch.where(frac == 0.0, torch.full_like(e, -126), e).clamp(min=-126)
    scale = torch.exp2(e.double())
    return _grid64(v / scale[:, block]), scale


def _values64(t):
    if not isinstance(t, tuple):
        return t.double()
    q, s = t
    col = torch.arange(q.shape[1], device=q.device) // 32
    return q.double() * s.double()[:, col]


def _act64(z, act):
    """The activation and its slope."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).double()
    if act == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg + z * sg * (1.0 - sg)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 0.134145 * z * z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def eight(v):
        q, scale = _eight64(v)
        return {"q": q, "scale": scale}

    if op == "linear":
        z = torch.matmul(_values64(s["x"]), s["w"].double().t().contiguous()) + s["b"].double()
        y = _act64(z, case["act"])[0]
        if s["r"] is not None:
            y = y + s["r"].double()
        return {"y": y, "z": eight(z)} if case["ckpt"] else {"y": y}
    if op == "linear_grad":
        dz = s["dy"].double()
        if s["z"] is not None:
            dz = dz * _act64(_values64(s["z"]), case["act"])[1]
        return {"dx": torch.matmul(dz, s["w"].double()), "dw": torch.matmul(dz.t().contiguous(), _values64(s["x"])),
                "db": dz.sum(0)}
    if op == "norm":
        h = s["x"].double() + (0.0 if s["r"] is None else s["r"].double())
        rstd = 1.0 / torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / case["cols"] + EPS)
        y = h * s["w"].double() * rstd[:, None]
        out = {"y": eight(y) if case["y8"] else y, "rstd": rstd}
        if s["r"] is not None:
            out["h"] = h
        if case["ckpt"]:
            out["ckpt"] = eight(h)
        return out
    if op == "norm_grad":
        # the gradient of y = h rstd w along its row: the part along h is taken out
        h, rstd, dy, w = _values64(s["h"]), s["rstd"].double(), s["dy"].double(), s["w"].double()
        along = torch.matmul(dy * h, w) * rstd ** 3 / case["cols"]
        dh = dy * w * rstd[:, None] - h * along[:, None]
        if s["dres"] is not None:
            dh = dh + s["dres"].double()
        return {"dh": dh, "dw": torch.matmul(rstd, dy * h)}
    q, scale = _eight64(s["x"].double())
    col = torch.arange(case["cols"], device=q.device) // 32
    return {"q": q, "scale": scale, "back": q * scale[:, col]}
