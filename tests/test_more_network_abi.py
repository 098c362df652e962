"""Refusals of the lookup, the clipping and the MX4 operators: every argument check answers on the
host, before anything is enqueued, with a message naming the argument (no GPU is touched); and
hand-worked values of the tests' own MX4 encoding."""
import ctypes as C

import numpy as np
import pytest
import torch

from tests import more_ref as ref

F32, BF16, MX8, MX4 = 0, 1, 2, 4


@pytest.fixture(scope="module")
def gs():
    from differentiable_tile_gaussian_amd import gs as _gs
    return _gs


class Mats:
    """gs_matrix values at made-up, distinct addresses."""

    def __init__(self, gs):
        self.gs, self.next = gs, 1 << 20

    def __call__(self, rows, cols, kind=BF16, **kw):
        self.next += 1 << 20
        ld = (cols + 31) // 32 * 32 if kind == MX4 else cols
        m = self.gs.GsMatrix(self.next, self.next + (1 << 19) if kind in (MX8, MX4) else None, rows, cols, ld, (cols + 31) // 32,
                             kind)
        for k, v in kw.items():
            setattr(m, k, v)
        return m


def refused(gs, status, text, code=None):
    code = gs.GS_ERR_INVALID_ARG if code is None else code
    assert status == code and text in gs.gs_last_error(), (status, gs.gs_last_error())


def test_mx4_arguments(gs):
    L, m, R = gs.lib(), Mats(gs), C.byref
    x, q = m(4, 40), m(4, 40, MX4)

    def pack(x=x, q=q):
        return L.gs_mx4_pack(R(x), R(q), None)
    refused(gs, pack(q=m(4, 40, MX4, ld=40)), "q: ld must be a multiple of 32")
    refused(gs, pack(q=m(4, 40, MX4, ld=32)), "q: ld out of range")
    refused(gs, pack(q=m(4, 40, MX4, ld=(1 << 21) + 32)), "q: ld must be")
    refused(gs, pack(q=m(4, 40, MX4, data=(1 << 20) + 8)), "q: data is misaligned")
    refused(gs, pack(q=m(4, 40, MX4, scales=None)), "q: scales is null")
    refused(gs, pack(q=m(4, 40, MX4, scales_ld=1)), "q: scales_ld")
    refused(gs, pack(q=m(4, 40, MX4, scales_ld=(1 << 21) + 1)), "q: scales_ld")
    refused(gs, pack(q=m(4, 41, MX4)), "q is 4 x 41")
    refused(gs, pack(q=m(4, 40, MX8)), "q: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, pack(x=m(4, 40, MX4)), "x: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, pack(x=m(4, 40, F32, data=q.data)), "output is one of the inputs")
    refused(gs, pack(x=m(4, 40, 5)), "x: unknown type")
    refused(gs, L.gs_mx4_unpack(R(x), R(x), None), "q: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, L.gs_mx4_unpack(R(q), R(q), None), "x: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, L.gs_mx4_unpack(None, R(x), None), "q is null")
    assert pack(m(0, 40, data=None), m(0, 40, MX4, data=None)) == gs.GS_OK
    # the operators that do not take it
    refused(gs, L.gs_mx8_pack(R(m(4, 40)), R(q), None), "q: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, L.gs_linear_bwd(R(m(4, 24)), None, 0, R(m(4, 40)), R(m(24, 40, MX4)), None, None, None, 16, 1 << 40, None),
            "w: this type", gs.GS_ERR_UNSUPPORTED)


def test_linear_mx4_arguments(gs):
    L, m, R = gs.lib(), Mats(gs), C.byref
    x, w, y = m(4, 40, MX4), m(24, 40, MX4), m(4, 24)

    def fwd(x=x, w=w, act=0, r=None, z=None, y=y):
        return L.gs_linear_fwd(R(x), R(w), None, act, R(r) if r else None, R(z) if z else None, R(y), None)
    refused(gs, fwd(z=m(4, 24, MX8)), "z: not kept", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(x=m(4, 40, F32)), "x: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(w=m(24, 40)), "x: this type", gs.GS_ERR_UNSUPPORTED)          # x in MX4 needs w in MX4
    refused(gs, fwd(x=m(4, 40), w=m(24, 40), y=m(4, 24, MX8)), "y: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(y=m(4, 24, MX4)), "y: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(w=m(24, 41, MX4)), "w is 24 x 41, expected 24 x 40")
    refused(gs, fwd(w=m(0, 40, MX4)), "w: rows")
    refused(gs, fwd(act=4), "activation")
    refused(gs, fwd(r=m(4, 40)), "residual is 4 x 40")
    refused(gs, fwd(y=m(4, 24, data=x.data)), "an output is one of the inputs")
    refused(gs, fwd(r=m(4, 24, F32, data=y.data)), "needs its type")
    assert fwd(x=m(0, 40, MX4, data=None), y=m(0, 24, data=None)) == gs.GS_OK


def test_lookup_arguments(gs):
    L, m, R = gs.lib(), Mats(gs), C.byref
    table, y = m(10, 24, F32), m(4, 24)

    def fwd(table=table, index=64, size=4, scale=1.0, y=y):
        return L.gs_lookup_fwd(R(table) if table else None, index, size, C.c_float(scale), R(y) if y else None, None)
    refused(gs, fwd(table=None), "table is null")
    refused(gs, fwd(table=m(0, 24, F32)), "table: rows")
    refused(gs, fwd(table=m(10, 24, MX8)), "table: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(y=None), "y is null")
    refused(gs, fwd(y=m(4, 25)), "y is 4 x 25, expected 4 x 24")
    refused(gs, fwd(y=m(4, 24, MX8)), "y: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(index=None), "index is null")
    refused(gs, fwd(index=66), "index is misaligned")
    refused(gs, fwd(index=68, size=8), "index is misaligned")
    refused(gs, fwd(size=2), "index_bytes")
    refused(gs, fwd(scale=float("nan")), "scale")
    refused(gs, fwd(scale=float("inf")), "scale")
    refused(gs, fwd(y=m(4, 24, F32, data=table.data)), "output is one of the inputs")
    assert fwd(index=None, y=m(0, 24, data=None)) == gs.GS_OK

    def bwd(dy=y, index=64, size=4, dtable=table, ws=16, nbytes=1 << 30):
        return L.gs_lookup_bwd(R(dy), index, size, C.c_float(1.0), R(dtable), ws, nbytes, None)
    need = gs.gs_workspace_bytes(gs.GS_WS_LOOKUP_BWD, 4, W=24, H=10)
    refused(gs, bwd(dy=m(4, 25)), "dy is 4 x 25")
    refused(gs, bwd(dtable=m(10, 24, MX8)), "dtable: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, bwd(dtable=m(10, 24, F32, data=y.data)), "output is one of the inputs")
    refused(gs, bwd(ws=None), "lookup_bwd workspace", gs.GS_ERR_CAPACITY)
    refused(gs, bwd(nbytes=need - 1), "lookup_bwd workspace", gs.GS_ERR_CAPACITY)
    assert gs.gs_workspace_bytes(gs.GS_WS_LOOKUP_BWD, -1, W=24, H=10) == 0
    assert gs.gs_workspace_bytes(gs.GS_WS_LOOKUP_BWD, 4, W=0, H=10) == 0


@pytest.mark.parametrize("cols", [1, 48, 600])
def test_a_lookup_workspace_serves_fewer_rows(gs, cols):
    rows = sorted(set(range(0, 9000)) | set(range(0, 400_000, 997)) | {(1 << 20) - 1, 1 << 20, (1 << 20) + 1})
    for entries in (1, 4096, 1 << 20):
        sizes = [gs.gs_workspace_bytes(gs.GS_WS_LOOKUP_BWD, r, W=cols, H=entries) for r in rows]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_clip_arguments(gs):
    L, m = gs.lib(), Mats(gs)

    def clip(grads, out=(), count=None, top=1.0, norm=64, ws=64, nbytes=1 << 30):
        a = (gs.GsMatrix * max(len(grads), 1))(*grads)
        o = (gs.GsMatrix * len(out))(*out) if out else None
        return L.gs_clip_grads(a, o, len(grads) if count is None else count, top, norm, ws, nbytes, None)
    g = [m(4, 24, F32), m(1, 7, BF16)]
    refused(gs, clip(g, count=-1), "count")
    refused(gs, clip(g, count=1025), "count")
    refused(gs, L.gs_clip_grads(None, None, 1, 1.0, 64, 64, 1 << 30, None), "grads is null")
    refused(gs, clip(g, norm=None), "norm is null")
    for bad in (0.0, -1.0, float("nan")):
        refused(gs, clip(g, top=bad), "max_norm")
    refused(gs, clip([g[0], m(4, 24, MX8)]), "grads[1]: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, clip(g, [m(4, 24, F32), m(1, 8)]), "out[1] is 1 x 8, expected 1 x 7")
    refused(gs, clip(g, [m(4, 24, MX8), m(1, 7)]), "out[0]: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, clip(g, [m(4, 24, BF16, data=g[0].data), m(1, 7)]), "out[0] in place")
    refused(gs, clip([g[0], g[0]], [g[0], g[0]]), "out[1] shares its data with entry 0")
    refused(gs, clip([g[0], g[0]], [m(4, 24, F32), g[0]]), "out[1] shares its data with entry 0")
    refused(gs, clip([m(4, 24, F32), g[0]], [g[0], m(4, 24, F32)]), "out[1] shares its data with entry 0")
    refused(gs, clip(g, ws=None), "clip_grads workspace", gs.GS_ERR_CAPACITY)
    refused(gs, clip(g, nbytes=gs.gs_workspace_bytes(gs.GS_WS_CLIP_GRADS) - 1), "clip_grads workspace", gs.GS_ERR_CAPACITY)


def test_binding_refuses(gs):
    x = torch.zeros(4, 40, dtype=torch.bfloat16)
    q = gs.mx4_empty(4, 40, device="cpu")
    assert q.shape == (4, 40) and q.q.shape == (4, 32) and q.scales.shape == (4, 2)
    for bad, text in ((gs.Mx4(q.q, q.scales, 65), "whole blocks"), (gs.Mx4(q.q, q.scales[:, :1], 40), "whole blocks|adjacent"),
                      (gs.Mx4(q.q.view(torch.int8), q.scales, 40), "uint8"), (q, "device memory")):
        with pytest.raises(ValueError, match=text):
            gs._struct(bad, "q")
    with pytest.raises(ValueError, match="index"):
        gs._index(torch.zeros(4, dtype=torch.int16), 4)
    with pytest.raises(ValueError, match="index"):
        gs._index(torch.zeros(4, dtype=torch.int32), 4)         # not in device memory
    with pytest.raises(ValueError, match="tensor"):
        gs.Matrices([q])
    with pytest.raises(ValueError, match="contiguous"):
        gs.Matrices([torch.zeros(3, 4, 5)[:, :2]])
    with pytest.raises(ValueError, match="device memory"):
        gs.Matrices([x])


@pytest.mark.parametrize("numel", [0, 1, 7, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, (3 << 20) + 5])
def test_tensors_as_matrices(gs, numel):
    parts = gs._as_matrices(torch.arange(numel, dtype=torch.float32), "t")
    assert all(p.dim() == 2 and p.shape[1] <= 1 << 20 for p in parts)
    assert torch.equal(torch.cat([p.reshape(-1) for p in parts]) if parts else torch.zeros(0), torch.arange(numel).float())


@pytest.mark.parametrize("n", [1, 63, 64, 65, 200])
def test_blocked_arrays_as_matrices(gs, n):
    t = gs.empty_blocked(n, 1, device="cpu")
    t.fill_(float("nan"))
    planes = torch.arange(23 * n, dtype=torch.float32).view(23, n)
    for i in range(n):
        t[i // 64, :, i % 64] = planes[:, i]
    parts = gs.blocked_matrices(t, n, 1)
    assert sorted(torch.cat([p.reshape(-1) for p in parts]).tolist()) == list(range(23 * n))


def test_the_reference_encoding_pins():
    v = np.zeros((1, 65))
    v[0, :9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.01]     # scale 1: ties go to the even code
    v[0, 32], v[0, 64] = 6.01, np.inf
    codes, s = ref.mx4_encode(v)
    assert list(codes[0, :9]) == [7, 0, 2, 2, 4, 4, 6, 6, 15] and list(s[0]) == [127, 128, 255]
    assert codes[0, 32] == 5                                           # 6.01 / 2 -> 3
    assert np.isnan(ref.mx4_decode(codes, s)[0, 64]) and ref.mx4_decode(codes, s)[0, 32] == 6.0
    assert list(ref.mx4_bytes(codes)[0, :5]) == [0x07, 0x22, 0x44, 0x66, 0x0f]
    assert np.array_equal(ref.mx4_codes(ref.mx4_bytes(codes, 9), 65), codes)
    assert list(ref.mx4_encode(np.zeros((1, 1)))[1][0]) == [1]
