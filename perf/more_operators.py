"""Cases, plain forms and inputs of further operators for networks over Gaussians: shared
features, 4-bit weights and the clipping of a step's gradients.

A network over Gaussians may take its feature rows from a table that many Gaussians share
(a codebook, a code per view), is trained with the norm of all gradients bounded, and is
served from weights in 4 bits.  Its operators:

  lookup       y[i] = scale table[index[i]]; a zero row where the index is outside the table
  lookup_grad  dtable[t] = scale times the sum of dy[i] over the rows i with index[i] = t
  clip         n = the Euclidean norm of all gradients together; each times min(1, max / n)
  pack4        a matrix to 4 bits with scales and back
  linear4      y = act(x W^T + b) + r with W in 4 bits, x in bfloat16, 8 or 4 bits

The 4-bit format (MX4): e2m1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign; two to a byte,
the even column in the low half), and for each 32 columns of a row one power-of-two scale 2^e
with the smallest e >= -126 for which the block's largest magnitude is at most 6 2^e.  Rows
are stored in whole blocks.  The 8-bit format (MX8) is e4m3 elements with 448 in 6's place.

`run` computes an operator from elementary torch operations in 32 bits (64 for the sums over
many rows; `own` false) or by the library's calls (`own` true); `exact` computes it from its
definition in 64 bits.
"""
import math

import torch
import torch.nn.functional as F

own = False

ACTS = ("none", "relu", "silu", "gelu")
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# Rows: 1,024 is the smallest scene of the benchmark, 1,000,003 its one-million scene made
# ragged, 3,000,000 its 720p stress scene, 8,160 the 16x16 tiles of its 1920x1080 images.
# A Gaussian has 59 parameters at SH degree 3, of which 48 are colour coefficients.
TILES = 8160


def _lookup(rows, entries, cols, f32=False, t16=False, wide=False):
    return {"op": "lookup", "rows": rows, "entries": entries, "cols": cols, "f32": f32, "t16": t16, "wide": wide}


def _lookup_grad(rows, entries, cols, f32=False, wide=False):
    return {"op": "lookup_grad", "rows": rows, "entries": entries, "cols": cols, "f32": f32, "wide": wide}


def _clip(gaussians, degree, blocks, width, hidden, outputs, over=True):
    return {"op": "clip", "gaussians": gaussians, "degree": degree, "blocks": blocks, "width": width, "hidden": hidden,
            "outputs": outputs, "over": over}


def _pack4(rows, cols, f32=False):
    return {"op": "pack4", "rows": rows, "cols": cols, "f32": f32}


def _linear4(rows, inner, outer, act="none", x="bf16", y="bf16", residual=False):
    return {"op": "linear4", "rows": rows, "inner": inner, "outer": outer, "act": act, "x": x, "y": y, "residual": residual}


def listed():
    return [
        # the smallest scene's features from a small codebook: latency
        {"name": "lookup_scene"} | _lookup(1024, 64, 32, f32=True),
        # every Gaussian of a large scene from a codebook of 2^16 float32 rows, as the network's bfloat16 input
        {"name": "lookup_gaussians"} | _lookup(1_000_003, 65536, 128, wide=True),
        # a middling scene's colour features, gradients in float32 from the rasteriser's planes
        {"name": "lookup_grad_scene"} | _lookup_grad(100_003, 4096, 48, f32=True),
        # the codebook's gradient over every Gaussian of a large scene
        {"name": "lookup_grad_gaussians"} | _lookup_grad(1_000_003, 65536, 128, wide=True),
        # a decoder's gradients alone, many of them small: latency
        {"name": "clip_network"} | _clip(0, 0, 4, 128, 256, 48),
        # those of a stress scene's Gaussians and a decoder together
        {"name": "clip_gaussians"} | _clip(3_000_000, 3, 1, 128, 128, 48),
        # a wide layer's float32 weight to 4 bits
        {"name": "pack4_weight"} | _pack4(1024, 4096, f32=True),
        # the hidden activations of every Gaussian
        {"name": "pack4_gaussians"} | _pack4(1_000_003, 128),
        # one image's appearance code through a wide layer when a single view is rendered
        {"name": "linear4_view"} | _linear4(1, 1024, 1024, "silu"),
        # a hidden layer over every Gaussian, from the norm's 8 bits to the next layer's
        {"name": "linear4_gaussians"} | _linear4(1_000_003, 128, 128, "silu", x="mx8", y="mx8"),
        # the second layer of a wide block over the tiles of a 1080p image, with its residual
        {"name": "linear4_tiles"} | _linear4(TILES, 4096, 1024, x="mx8", residual=True),
        # the first one, with its input in 4 bits
        {"name": "linear4_tiles_x4"} | _linear4(TILES, 1024, 4096, "gelu", x="mx4"),
    ]


def _size(rng, low, high):
    """Log-uniform in [low, high]; every other one a multiple of 16 where that fits."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and n >= 16:
        n = n // 16 * 16
    return min(max(n, low), high)


def draw(rng):
    op = rng.choice(("lookup", "lookup_grad", "clip", "pack4", "linear4"))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("lookup", "lookup_grad"):
        cols = _size(rng, 3, 512)
        rows = _size(rng, 1, min(1_000_003, 1_000_003 * 64 // cols))
        entries = _size(rng, 1, min(1 << 18, (1 << 22) // cols))
        if op == "lookup":
            return _lookup(rows, entries, cols, f32=flag(), t16=flag(), wide=flag())
        return _lookup_grad(rows, entries, cols, f32=flag(), wide=flag())
    if op == "clip":
        blocks = rng.choice((0, 1, 2, 3, 4))
        gaussians = 0 if blocks and rng.random() < 0.4 else _size(rng, 1, 2_000_000)
        return _clip(gaussians, rng.choice((0, 1, 2, 3)), blocks, _size(rng, 16, 256), _size(rng, 16, 1024),
                     _size(rng, 3, 59), over=flag())
    if op == "pack4":
        cols = _size(rng, 3, 4096)
        rows = _size(rng, 1, min(1_000_003, 1_000_003 * 64 // cols))
        return _pack4(rows, cols, f32=flag())
    if rng.random() < 0.6:    # rows are Gaussians
        inner, outer = _size(rng, 3, 256), _size(rng, 3, 256)
        rows = _size(rng, 1, min(1_000_003, 1_000_003 * 200 // (inner + outer)))
    else:                     # rows are image tiles or views
        inner, outer = _size(rng, 256, 4096), _size(rng, 256, 4096)
        rows = _size(rng, 1, min(TILES, TILES * 1024 * 3500 // (inner * outer)))
    return _linear4(rows, inner, outer, rng.choice(ACTS), x=rng.choice(("bf16", "mx8", "mx4")),
                    y=rng.choice(("bf16", "f32", "mx8")), residual=flag())


# ---------------------------------------------------------------- the formats, plain

def _blocks(v):
    """The 32-column blocks of [M][C] (zeros behind the last column)."""
    m, c = v.shape
    return F.pad(v, (0, -c % 32)).view(m, -1, 32)


def quantise8(v):
    """float32 [M][C] -> (e4m3 [M][C], e8m0 [M][ceil(C / 32)])."""
    b = _blocks(v)
    # the exponent field of the smallest 2^e with the largest magnitude <= 1.75 2^(e + 8)
    e = (((b.abs().amax(-1).view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(1, 254)
    q = (b * ((254 - e) << 23).view(torch.float32).unsqueeze(-1)).to(E4M3)
    return q.view(v.shape[0], -1)[:, :v.shape[1]], e.to(torch.uint8).view(E8M0)


def quantise4(v):
    """float32 [M][C] -> (e2m1 codes, uint8 [M][32 ceil(C / 32)], e8m0 [M][ceil(C / 32)])."""
    b = _blocks(v)
    # 6 = 1.5 2^2
    e = (((b.abs().amax(-1).view(torch.int32) + 0x3FFFFF) >> 23) - 2).clamp(1, 254)
    r = b * ((254 - e) << 23).view(torch.float32).unsqueeze(-1)
    a = r.abs()
    # how many midpoints are passed; a midpoint itself goes to the even code
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = code | (torch.signbit(r).to(torch.uint8) << 3)
    return code.view(v.shape[0], -1), e.to(torch.uint8).view(E8M0)


def dequantise8(q, s):
    return q.float() * s.float().repeat_interleave(32, dim=1)[:, :q.shape[1]]


def dequantise4(code, s, c):
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=code.device)
    return (table[code.long()] * s.float().repeat_interleave(32, dim=1))[:, :c]


def _stored8(v):
    """(q, scales) with rows that start at multiples of 16 bytes."""
    q, s = quantise8(v)
    m, c = q.shape
    store = torch.zeros((m, (c + 15) // 16 * 16), dtype=torch.uint8, device=q.device).view(E4M3)
    store[:, :c].view(torch.uint8).copy_(q.view(torch.uint8))
    return {"q": store[:, :c], "scales": s.contiguous(), "cols": c}


def _stored4(v):
    """Two codes to a byte, the even column in the low half."""
    code, s = quantise4(v)
    return {"q": (code[:, 0::2] | code[:, 1::2] << 4).contiguous(), "scales": s.contiguous(), "cols": v.shape[1]}


# ---------------------------------------------------------------- inputs

def _shapes(case):
    """The decoder's parameters: per block two layers and a norm, and the head."""
    w, h, o = case["width"], case["hidden"], case["outputs"]
    if not case["blocks"]:
        return []
    return [(w,), (h, w), (h,), (w, h), (w,)] * case["blocks"] + [(w,), (o, w), (o,)]


def _planes(case):
    return 11 + 3 * (case["degree"] + 1) ** 2


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

    def kept(v, kind):
        return {"mx8": _stored8, "mx4": _stored4, "bf16": torch.Tensor.bfloat16, "f32": torch.Tensor.float}[kind](v)

    op, s = case["op"], {"case": case}
    wide = torch.float32 if case.get("f32") else torch.bfloat16
    if op in ("lookup", "lookup_grad"):
        m, t, c = case["rows"], case["entries"], case["cols"]
        # entries are used unevenly (an entry's share falls with its rank, ranks are scattered over
        # the table), and one row in fifty has none
        rank = (torch.rand(m, generator=g, device="cuda") ** 3 * t).long().clamp(max=t - 1)
        index = torch.randperm(t, generator=g, device="cuda")[rank]
        index[torch.rand(m, generator=g, device="cuda") < 0.02] = -1
        s["index"] = index if case["wide"] else index.int()
        s["scale"] = c ** 0.5 if op == "lookup" else 0.25
        if op == "lookup":
            s["table"] = stream(t, c).to(torch.bfloat16 if case["t16"] else torch.float32)
        else:
            s["dy"] = grads(m, c).to(wide)
        return s
    if op == "clip":
        n, p = case["gaussians"], _planes(case)
        list_ = [grads(shape[0], shape[1] if len(shape) > 1 else 1).view(shape) for shape in _shapes(case)]
        if n:
            # the parameter gradients as the rasteriser keeps them: groups of 64 Gaussians, p planes each;
            # what is behind the last Gaussian is no gradient
            blocked = grads((n + 63) // 64 * 64, p).view(-1, 64, p).transpose(1, 2).contiguous()
            if n % 64:
                blocked[-1, :, n % 64:] = float("nan")
            s["blocked"] = blocked
            s["blocked_out"] = torch.zeros_like(blocked)
        s["grads"], s["out"] = list_, [torch.empty_like(x) for x in list_]
        count = sum(x.numel() for x in list_) + n * p
        s["max"] = (count * 2.0 / 3.0) ** 0.5 * math.exp(-12.0) * (0.5 if case["over"] else 8.0)
        return s
    m = case["rows"]
    if op == "pack4":
        s["x"] = stream(m, case["cols"]).to(wide)
        return s
    k, n = case["inner"], case["outer"]
    s["w"] = _stored4(normal(n, k, scale=k ** -0.5))
    s["b"] = normal(n, scale=0.1)
    s["x"] = kept(stream(m, k), case["x"])
    s["r"] = stream(m, n).to(torch.float32 if case["y"] == "f32" else torch.bfloat16) if case["residual"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _codes(t):
    q = t["q"]
    return torch.stack((q & 15, q >> 4), dim=2).view(q.shape[0], -1)


def _values(t):
    if not isinstance(t, dict):
        return t.float()
    return dequantise8(t["q"], t["scales"]) if t["q"].dtype == E4M3 else dequantise4(_codes(t), t["scales"], t["cols"])


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain(s):
    case = s["case"]
    op = case["op"]
    wide = torch.float32 if case.get("f32") else torch.bfloat16
    if op in ("lookup", "lookup_grad"):
        there = (s["index"] >= 0) & (s["index"] < case["entries"])
        index = torch.where(there, s["index"], 0).long()
        if op == "lookup":
            rows = s["table"][index].float() * s["scale"]
            return {"y": torch.where(there[:, None], rows, 0.0).to(wide)}
        dy = torch.where(there[:, None], s["dy"], 0.0).double()
        total = torch.zeros((case["entries"], case["cols"]), dtype=torch.float64, device=dy.device)
        return {"dtable": (total.index_add_(0, index, dy) * s["scale"]).float()}
    if op == "clip":
        n = case["gaussians"]
        every = list(s["grads"])
        if n:
            full = n // 64
            every += [s["blocked"][:full], s["blocked"][full:, :, :n % 64]]
        norm = sum(x.double().square().sum() for x in every).sqrt()
        factor = (s["max"] / norm).clamp(max=1.0).float()
        out = {"norm": norm.float(), "grads": [x * factor for x in s["grads"]]}
        if n:
            clipped = s["blocked"] * factor
            if n % 64:
                clipped[-1, :, n % 64:] = 0.0
            out["blocked"] = clipped
        return out
    if op == "pack4":
        code, e = quantise4(s["x"].float())
        return {"scale": e, "back": dequantise4(code, e, case["cols"]).bfloat16()}
    y = _act(_values(s["x"]) @ _values(s["w"]).t() + s["b"], case["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    if case["y"] == "mx8":
        q, e = quantise8(y)
        return {"y": q, "scale": e}
    return {"y": y if case["y"] == "f32" else y.bfloat16()}


# ---------------------------------------------------------------- the library's calls

def _library(s):
    from differentiable_tile_gaussian_amd import gs

    case = s["case"]
    op = case["op"]
    wide = torch.float32 if case.get("f32") else torch.bfloat16

    def matrix(t):
        if not isinstance(t, dict):
            return t
        return gs.Mx8(t["q"], t["scales"]) if t["q"].dtype == E4M3 else gs.Mx4(t["q"], t["scales"], t["cols"])

    def empty(rows, cols, dtype):
        return torch.empty((rows, cols), dtype=dtype, device="cuda")

    if op == "lookup":
        y = empty(case["rows"], case["cols"], wide)
        gs.gs_lookup_fwd(s["table"], s["index"], y, scale=s["scale"])
        return {"y": y}
    if op == "lookup_grad":
        if "ws" not in s:
            s["ws"] = gs.workspace(gs.GS_WS_LOOKUP_BWD, n=case["rows"], W=case["cols"], H=case["entries"])
        dtable = empty(case["entries"], case["cols"], torch.float32)
        gs.gs_lookup_bwd(s["dy"], s["index"], dtable, s["ws"], scale=s["scale"])
        return {"dtable": dtable}
    if op == "clip":
        n = case["gaussians"]
        if "ws" not in s:   # the buffers of a step stay where they are
            s["ws"] = gs.workspace(gs.GS_WS_CLIP_GRADS)
            s["lists"] = [gs.Matrices(list_ + (gs.blocked_matrices(blocked, n, case["degree"]) if n else []))
                          for list_, blocked in ((s["grads"], s.get("blocked")), (s["out"], s.get("blocked_out")))]
        norm = torch.empty(1, dtype=torch.float32, device="cuda")
        gs.gs_clip_grads(s["lists"][0], s["max"], norm, s["ws"], out=s["lists"][1])
        out = {"norm": norm[0], "grads": s["out"]}
        return out | {"blocked": s["blocked_out"]} if n else out
    if op == "pack4":
        q = gs.mx4_empty(case["rows"], case["cols"])
        back = empty(case["rows"], case["cols"], torch.bfloat16)
        gs.gs_mx4_pack(s["x"], q)
        gs.gs_mx4_unpack(q, back)
        return {"scale": q.scales, "back": back}
    m, n = case["rows"], case["outer"]
    y = gs.mx8_empty(m, n) if case["y"] == "mx8" else empty(m, n, torch.float32 if case["y"] == "f32" else torch.bfloat16)
    gs.gs_linear_fwd(matrix(s["x"]), matrix(s["w"]), y, bias=s["b"], act=case["act"], residual=s["r"])
    return {"y": y.q, "scale": y.scales} if case["y"] == "mx8" else {"y": y}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- the work of one pass

def _bytes(rows, cols, kind):
    nb = (cols + 31) // 32
    return rows * {"mx8": cols + nb, "mx4": 17 * nb, "bf16": 2 * cols, "f32": 4 * cols}[kind]


def work(case):
    op = case["op"]
    kind = "f32" if case.get("f32") else "bf16"
    if op in ("lookup", "lookup_grad"):
        m, t, c = case["rows"], case["entries"], case["cols"]
        # a forward has to read the entries that are used, at most one a row
        table = _bytes(min(t, m) if op == "lookup" else t, c, "bf16" if case.get("t16") else "f32")
        return {"bytes": _bytes(m, c, kind) + table + m * (8 if case["wide"] else 4), "flops": m * c}
    if op == "clip":
        count = sum(math.prod(shape) for shape in _shapes(case)) + case["gaussians"] * _planes(case)
        return {"bytes": 8 * count + 4, "flops": 3 * count}
    m = case["rows"]
    if op == "pack4":
        c = case["cols"]
        return {"bytes": _bytes(m, c, kind) + _bytes(m, c, "mx4") + _bytes(m, c, "bf16"), "flops": 3 * m * c}
    k, n = case["inner"], case["outer"]
    b = _bytes(m, k, case["x"]) + _bytes(n, k, "mx4") + _bytes(m, n, case["y"]) + 4 * n
    b += _bytes(m, n, "f32" if case["y"] == "f32" else "bf16") if case["residual"] else 0
    return {"bytes": b, "flops": 2 * m * n * k}


# ---------------------------------------------------------------- the definition in 64 bits

def _nearest64(v, digits, lowest):
    """The nearest value with `digits` digits behind the leading one (ties to the even one), spaced
    evenly below 2^lowest, in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.exp2(torch.clamp(e - 1, min=lowest).double() - digits)
    return torch.round(v / step) * step


def _scaled64(v, largest, digits, lowest):
    """Elements and scales of 32-column blocks."""
    m, c = v.shape
    block = torch.arange(c, device=v.device) // 32
    top = torch.zeros((m, (c + 31) // 32), dtype=torch.float64, device=v.device)
    top.scatter_reduce_(1, block.expand(m, c), v.abs(), "amax")
    frac, e = torch.frexp(top / largest)
    e = torch.where(frac == 0.5, e - 1, e)
    e = torch.where(frac == 0.0, torch.full_like(e, -126), e).clamp(min=-126)
    scale = torch.exp2(e.double())
    return _nearest64(v / scale[:, block], digits, lowest), scale


def _values64(t):
    if not isinstance(t, dict):
        return t.double()
    q, c = t["q"], t["cols"]
    col = torch.arange(c, device=q.device)
    if q.dtype == E4M3:
        v = q.double()
    else:
        code = ((q[:, col // 2] >> (col % 2 * 4).to(torch.uint8)) & 15).double()
        mag = code % 8
        # one digit behind the point; two values below 1
        v = torch.where(mag < 2, mag * 0.5, (1.0 + mag % 2 * 0.5) * torch.exp2(torch.floor(mag / 2) - 1.0))
        v = torch.where(code >= 8, -v, v)
    return v * t["scales"].double()[:, col // 32]


def _act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        table = torch.cat((s["table"].double(), torch.zeros_like(s["table"][:1]).double()))
        return {"y": table[s["index"].long()] * s["scale"]}      # -1: the row of zeros behind the table
    if op == "lookup_grad":
        # rows in the order of their entries: an entry's sum is a difference of running sums
        order = torch.argsort(s["index"], stable=True)
        ends = torch.searchsorted(s["index"][order].long(), torch.arange(-1, case["entries"], device="cuda"), right=True)
        running = F.pad(s["dy"][order].double().cumsum(0), (0, 0, 1, 0))
        return {"dtable": (running[ends[1:]] - running[ends[:-1]]) * s["scale"]}
    if op == "clip":
        n = case["gaussians"]
        every = [x.double() for x in s["grads"]]
        parts = [torch.linalg.vector_norm(x) for x in every]
        if n:
            blocked = s["blocked"].double()
            blocked.view(-1, 64)[torch.isnan(blocked.view(-1, 64))] = 0.0   # the padding alone
            parts.append(torch.linalg.vector_norm(blocked))
        norm = torch.linalg.vector_norm(torch.stack(parts))
        by = torch.minimum(s["max"] / norm, torch.ones_like(norm))
        out = {"norm": norm, "grads": [x * by for x in every]}
        return out | {"blocked": blocked * by} if n else out
    if op == "pack4":
        q, scale = _scaled64(s["x"].double(), 6.0, 1.0, 0)
        col = torch.arange(case["cols"], device=q.device) // 32
        return {"scale": scale, "back": q * scale[:, col]}
    z = torch.matmul(_values64(s["x"]), _values64(s["w"]).t().contiguous()) + s["b"].double()
    y = _act64(z, case["act"])
    if s["r"] is not None:
        y = y + s["r"].double()
    if case["y"] != "mx8":
        return {"y": y}
    q, scale = _scaled64(y, 448.0, 3.0, -6)
    return {"y": q, "scale": scale}
