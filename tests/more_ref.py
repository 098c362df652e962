"""Plain 64-bit forms of the lookup, the clipping and the MX4 operators, on the CPU.

MX4 is encoded by a search in the list of e2m1 values, element by element of the definition."""
import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_HALF = (E2M1[1:] + E2M1[:-1]) / 2


def e2m1_codes(v):
    """Codes of the nearest e2m1 values of a float64 array with |v| <= 6."""
    a = np.abs(v)
    code = np.searchsorted(_HALF, a, side="left")          # a on a midpoint stays below
    tie = (code < 7) & (a == _HALF[np.minimum(code, 6)]) & (code % 2 == 1)
    return (np.where(tie, code + 1, code) | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def mx4_scale_bytes(v):
    """[rows][blocks] scale bytes of a float64 matrix; 255 for a block with an infinity or a NaN."""
    rows, cols = v.shape
    out = np.zeros((rows, (cols + 31) // 32), np.uint8)
    for b in range(out.shape[1]):
        blk = v[:, 32 * b:32 * b + 32]
        for i in range(rows):
            if not np.isfinite(blk[i]).all():
                out[i, b] = 255
                continue
            top, e = np.abs(blk[i]).max(), -126
            if top > 0.0:
                e = max(math.frexp(top)[1] - 5, -126)
                while top > 6.0 * 2.0 ** e:
                    e += 1
            out[i, b] = e + 127
    return out


def mx4_encode(v):
    """(codes [rows][cols], scale bytes) of a float64 matrix; codes of a NaN block are zero."""
    s = mx4_scale_bytes(v)
    scale = np.exp2(s.astype(np.float64) - 127.0).repeat(32, axis=1)[:, :v.shape[1]]
    bad = (s == 255).repeat(32, axis=1)[:, :v.shape[1]]
    return np.where(bad, 0, e2m1_codes(np.where(bad, 0.0, v) / scale)).astype(np.uint8), s


def mx4_decode(codes, s):
    scale = np.exp2(s.astype(np.float64) - 127.0)
    scale[s == 255] = np.nan
    mag = E2M1[codes & 7]
    return np.where(codes & 8, -mag, mag) * scale.repeat(32, axis=1)[:, :codes.shape[1]]


def mx4_bytes(codes, behind=0):
    """Two codes to a byte in whole blocks; `behind`: the codes behind the last column."""
    rows, cols = codes.shape
    whole = np.full((rows, (cols + 31) // 32 * 32), behind, np.uint8)
    whole[:, :cols] = codes
    return whole[:, 0::2] | whole[:, 1::2] << 4


def mx4_codes(q, cols):
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out[:, :cols]


def lookup(table, index, scale):
    """(rows, rows of the magnitudes) in float64."""
    there = (index >= 0) & (index < table.shape[0])
    y = torch.where(there[:, None], table[torch.where(there, index, 0)], 0.0) * scale
    return y, y.abs()


def lookup_grad(dy, index, entries, scale):
    """(sums, sums of magnitudes, rows of each entry) in float64."""
    there = (index >= 0) & (index < entries)
    at, rows = index[there], dy[there]
    total = torch.zeros(entries, dy.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(total)
    total.index_add_(0, at, rows)
    mag.index_add_(0, at, rows.abs())
    return total * scale, mag * abs(scale), torch.bincount(at, minlength=entries)


def clip(grads, max_norm):
    """(norm, clipped) in float64."""
    norm = math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))
    f = 1.0 if norm <= max_norm else max_norm / norm
    return norm, [g.double() * f for g in grads]
