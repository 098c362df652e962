"""Plain 64-bit forms of the network operators, on the CPU, and the tolerances their tests use.

MX8 is encoded here by a search in the sorted list of e4m3 values, element by element of the
definition: the block's exponent, then the nearest value with ties to the even code.
"""
import math

import numpy as np
import torch

U24 = 2.0 ** -24        # float32 unit roundoff
UBF = 2.0 ** -8         # bfloat16 unit roundoff (8 significant bits)


def e4m3_table():
    """The 127 non-negative finite e4m3 values by code."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


_TABLE = e4m3_table()
_HALF = (_TABLE[1:] + _TABLE[:-1]) / 2


def e4m3_codes(v):
    """Codes of the nearest e4m3 values of a float64 array with |v| <= 448 (NaN: 0x7f)."""
    a = np.abs(v)
    code = np.searchsorted(_HALF, a, side="left")          # a on a midpoint stays below
    tie = (code < 126) & (a == _HALF[np.minimum(code, 125)]) & (code % 2 == 1)
    code = np.where(tie, code + 1, code)
    code = np.where(np.isnan(v), 0x7f, code)
    return (code | np.where(np.signbit(v) & ~np.isnan(v), 0x80, 0)).astype(np.uint8)


def mx8_scale_bytes(v):
    """[rows][blocks] scale bytes of a float64 matrix."""
    rows, cols = v.shape
    nb = (cols + 31) // 32
    out = np.zeros((rows, nb), np.uint8)
    for b in range(nb):
        blk = v[:, 32 * b:32 * b + 32]
        top = np.where(np.isfinite(blk), np.abs(blk), 0.0).max(1) if rows else np.zeros(0)
        for i in range(rows):
            e = -126
            if top[i] > 0.0:
                e = max(math.frexp(top[i])[1] - 12, -126)
                while top[i] > 448.0 * 2.0 ** e:
                    e += 1
            out[i, b] = e + 127
    return out


def mx8_encode(v):
    """(codes [rows][cols], scale bytes) of a float64 matrix; non-finite elements are NaN."""
    s = mx8_scale_bytes(v)
    scale = np.exp2(s.astype(np.float64) - 127.0).repeat(32, axis=1)[:, :v.shape[1]]
    with np.errstate(invalid="ignore"):
        r = np.where(np.isfinite(v), v / scale, np.nan)
    return e4m3_codes(r), s


def mx8_decode(codes, s):
    mag = np.where((codes & 0x7f) == 0x7f, np.nan, np.append(_TABLE, np.nan)[codes & 0x7f])
    scale = np.exp2(s.astype(np.float64) - 127.0)
    scale[s == 255] = np.nan
    return np.where(codes & 0x80, -mag, mag) * scale.repeat(32, axis=1)[:, :codes.shape[1]]


def activation(z, act):
    """(act(z), act'(z)) in float64."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        g = torch.sigmoid(z)
        return z * g, g * (1 + z * (1 - g))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t ** 2) * c * (1 + 3 * 0.044715 * z ** 2)


def linear(x, w, b, act, r=None):
    z = x @ w.t() + b
    y = activation(z, act)[0]
    return z, y if r is None else y + r


def linear_grads(dy, z, act, x, w):
    dz = dy if act == "none" else dy * activation(z, act)[1]
    return dz, dz @ w, dz.t() @ x, dz.sum(0)


def rmsnorm(x, r, w, eps):
    h = x if r is None else x + r
    rstd = (h.square().mean(1) + eps) ** -0.5
    return h, rstd, h * rstd[:, None] * w


def rmsnorm_grads(dy, h, w, rstd, dres=None):
    xhat = h * rstd[:, None]
    u = dy * w
    dh = rstd[:, None] * (u - xhat * (u * xhat).mean(1, keepdim=True))
    return dh if dres is None else dh + dres, (dy * xhat).sum(0)


def rounding(dtype):
    """Relative rounding error of one store to dtype."""
    return UBF if dtype == torch.bfloat16 else U24
