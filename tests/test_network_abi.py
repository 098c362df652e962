"""Refusals of the network operators: every argument check answers on the host, before
anything is enqueued, with a message naming the argument (no GPU is touched)."""
import ctypes as C

import numpy as np
import pytest
import torch

from tests import network_ref as ref

F32, BF16, MX8 = 0, 1, 2


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
        m = self.gs.GsMatrix(self.next, self.next + (1 << 19) if kind == MX8 else None, rows, cols, cols, (cols + 31) // 32,
                             kind)
        for k, v in kw.items():
            setattr(m, k, v)
        return m


def refused(gs, status, text, code=None):
    code = gs.GS_ERR_INVALID_ARG if code is None else code
    assert status == code and text in gs.gs_last_error(), (status, gs.gs_last_error())


def test_matrix_fields(gs):
    L, m = gs.lib(), Mats(gs)
    q = m(4, 40, MX8)
    R = C.byref

    def pack(x, out=None):
        return L.gs_mx8_pack(R(x) if x is not None else None, R(out or q), None)
    refused(gs, pack(None), "x is null")
    refused(gs, pack(m(-1, 40)), "x: rows")
    refused(gs, pack(m(1 << 31, 40)), "x: rows")
    refused(gs, pack(m(4, 0)), "x: cols")
    refused(gs, pack(m(4, (1 << 20) + 1)), "x: more than 2^20", gs.GS_ERR_UNSUPPORTED)
    refused(gs, pack(m(4, 40, ld=39)), "x: ld")
    refused(gs, pack(m(4, 40, type=3)), "x: unknown type")
    refused(gs, pack(m(4, 40, MX8)), "x: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, pack(m(4, 40, data=None)), "x: data is null")
    refused(gs, pack(m(4, 40, data=(1 << 20) + 1)), "x: data is misaligned")
    refused(gs, pack(m(4, 40, F32, data=(1 << 20) + 2)), "x: data is misaligned")
    refused(gs, pack(m(4, 40), m(4, 41, MX8)), "q is 4 x 41, expected 4 x 40")
    refused(gs, pack(m(4, 40), m(4, 40, MX8, scales=None)), "q: scales is null")
    refused(gs, pack(m(4, 40), m(4, 40, MX8, scales_ld=1)), "q: scales_ld")
    x = m(4, 40)
    refused(gs, pack(x, m(4, 40, MX8, data=x.data)), "output is one of the inputs")
    assert L.gs_mx8_pack(R(m(0, 40, data=None)), R(m(0, 40, MX8, data=None)), None) == gs.GS_OK   # nothing to do
    refused(gs, L.gs_mx8_unpack(R(m(4, 40)), R(m(4, 40)), None), "q: this type", gs.GS_ERR_UNSUPPORTED)


def test_norm_arguments(gs):
    L, m, R = gs.lib(), Mats(gs), C.byref
    x, y = m(4, 40), m(4, 40)

    def fwd(x=x, r=None, w=16, eps=1e-6, h=None, ck=None, y=y):
        return L.gs_rmsnorm_fwd(R(x), R(r) if r else None, w, C.c_float(eps), R(h) if h else None, R(ck) if ck else None, R(y),
                                None, None)
    refused(gs, fwd(w=None), "weight")
    refused(gs, fwd(eps=0.0), "eps")
    refused(gs, fwd(eps=float("nan")), "eps")
    refused(gs, fwd(r=m(4, 41)), "residual is 4 x 41")
    refused(gs, fwd(h=m(3, 40)), "h is 3 x 40")
    refused(gs, fwd(h=m(4, 40, MX8)), "h: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(ck=m(4, 40)), "ckpt: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(y=x), "an output is one of the inputs")
    refused(gs, fwd(h=y), "an output is one of the inputs")
    refused(gs, fwd(h=m(4, 40, F32, data=x.data)), "needs its type")

    def bwd(dy=x, h=m(4, 40, MX8), w=16, rstd=16, dres=None, dh=y, dw=16, ws=16, nbytes=1 << 30):
        return L.gs_rmsnorm_bwd(R(dy), R(h), w, rstd, R(dres) if dres else None, R(dh), dw, ws, nbytes, None)
    refused(gs, bwd(rstd=None), "rstd")
    refused(gs, bwd(h=m(4, 41)), "h is 4 x 41")
    refused(gs, bwd(dh=x), "output is one of the inputs")
    refused(gs, bwd(dh=m(4, 40, MX8)), "dh: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, bwd(ws=None), "rmsnorm_bwd workspace", gs.GS_ERR_CAPACITY)
    need = gs.gs_workspace_bytes(gs.GS_WS_RMSNORM_BWD, 4, W=40)
    assert need >= 160
    refused(gs, bwd(nbytes=need - 1), "rmsnorm_bwd workspace", gs.GS_ERR_CAPACITY)


def test_linear_arguments(gs):
    L, m, R = gs.lib(), Mats(gs), C.byref
    x, w, y = m(4, 40), m(24, 40), m(4, 24)

    def fwd(x=x, w=w, act=0, r=None, z=None, y=y):
        return L.gs_linear_fwd(R(x), R(w), None, act, R(r) if r else None, R(z) if z else None, R(y), None)
    refused(gs, fwd(x=m(4, 40, F32)), "x: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(w=m(24, 41)), "w is 24 x 41, expected 24 x 40")
    refused(gs, fwd(w=m(24, 40, F32)), "w: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(w=m(0, 40)), "w: rows")
    refused(gs, fwd(act=4), "activation")
    refused(gs, fwd(act=-1), "activation")
    refused(gs, fwd(r=m(4, 40)), "residual is 4 x 40")
    refused(gs, fwd(z=m(5, 24, MX8)), "z is 5 x 24")
    refused(gs, fwd(y=m(4, 24, MX8)), "y: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, fwd(y=m(4, 24, data=x.data)), "an output is one of the inputs")
    refused(gs, fwd(r=m(4, 24, F32, data=y.data)), "needs its type")

    def bwd(dy=m(4, 24), z=None, act=0, x=x, w=w, dx=m(4, 40), dw=m(24, 40, F32), ws=16, nbytes=1 << 40):
        return L.gs_linear_bwd(R(dy), R(z) if z else None, act, R(x), R(w), R(dx) if dx else None, R(dw) if dw else None, None,
                               ws, nbytes, None)
    refused(gs, bwd(act=2), "z is null")
    refused(gs, bwd(dy=m(4, 40)), "dy is 4 x 40")
    refused(gs, bwd(dy=m(4, 24, MX8)), "dy: this type", gs.GS_ERR_UNSUPPORTED)
    refused(gs, bwd(dx=m(4, 24)), "dx is 4 x 24")
    refused(gs, bwd(dw=m(40, 24)), "dw is 40 x 24")
    refused(gs, bwd(dx=x), "output is one of the inputs")
    refused(gs, bwd(dw=w), "output is one of the inputs")
    need = gs.gs_workspace_bytes(gs.GS_WS_LINEAR_BWD, 4, W=40, H=24)
    refused(gs, bwd(nbytes=need - 1), "linear_bwd workspace", gs.GS_ERR_CAPACITY)
    refused(gs, bwd(ws=None), "linear_bwd workspace", gs.GS_ERR_CAPACITY)


def test_workspaces(gs):
    ws = gs.gs_workspace_bytes
    assert ws(gs.GS_WS_LINEAR_BWD, -1, W=8, H=8) == 0 and ws(gs.GS_WS_LINEAR_BWD, 8, W=0, H=8) == 0
    assert ws(gs.GS_WS_LINEAR_BWD, 8, W=8, H=(1 << 20) + 1) == 0 and ws(gs.GS_WS_RMSNORM_BWD, 8, W=0) == 0
    assert ws(gs.GS_WS_RMSNORM_BWD, 0, W=64) > 0 and ws(gs.GS_WS_LINEAR_BWD, 0, W=64, H=64) > 0


def test_binding_refuses(gs):
    x = torch.zeros(4, 40, dtype=torch.bfloat16)
    for bad, text in ((x, "device memory"), (x.half(), "float32, bfloat16"), (x.t(), "adjacent"), (x[0], "adjacent|matrix")):
        with pytest.raises(ValueError, match=text):
            gs.gs_mx8_pack(bad, gs.mx8_empty(4, 40, device="cpu"))
    with pytest.raises(ValueError, match="Mx8"):
        gs.gs_mx8_unpack(gs.Mx8(x, x), x)
    with pytest.raises(ValueError, match="act"):
        gs._activation("tanh")
    with pytest.raises(ValueError, match="bias"):
        gs._floats(torch.zeros(3), 4, "bias")


def test_the_reference_encoding_pins():
    """Hand-worked MX8 values: the tests' own reference against the definition."""
    v = np.zeros((1, 33))
    v[0, :6] = [448.0, 1.0, 17.0, 19.0, -2.0 ** -10, 3 * 2.0 ** -10]
    v[0, 32] = 449.0
    codes, s = ref.mx8_encode(v)
    # scale 1: 448 = 0x7e, 1 = 0x38, 17 -> 16 and 19 -> 20 (ties to even), 2^-10 -> 0, 3 2^-10 -> 2^-8
    assert list(codes[0, :6]) == [0x7e, 0x38, 0x58, 0x5a, 0x80, 0x02] and list(s[0]) == [127, 128]
    assert codes[0, 32] == 0x76                                         # 449 / 2 = 224.5 -> 224
    assert ref.mx8_decode(codes, s)[0, 32] == 448.0
    assert list(ref.mx8_encode(np.zeros((1, 1)))[1][0]) == [1]


@pytest.mark.parametrize("k,n", [(64, 48), (128, 128), (256, 64), (64, 256), (99, 113), (200, 200), (1024, 4096), (4096, 40)])
def test_a_workspace_serves_fewer_rows(gs, k, n):
    """Sizes do not fall as rows are added, so that one made for the most rows serves all calls."""
    rows = sorted({r + d for r in (0, 128, 512, 1280, 16384, 20480, 32768, 65536, 131072, 1 << 20) for d in (-1, 0, 1, 127, 128)
                   if r + d >= 0} | set(range(0, 140_000, 997)))
    for call, kw in ((gs.GS_WS_LINEAR_BWD, dict(W=k, H=n)), (gs.GS_WS_RMSNORM_BWD, dict(W=k))):
        sizes = [gs.gs_workspace_bytes(call, r, **kw) for r in rows]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), [(r, a, b) for r, a, b in zip(rows, sizes, sizes[1:]) if a > b][:3]
