"""The network operators (MX8 storage, RMS norm, linear layers and their gradients) on the GPU
against plain 64-bit forms on the CPU.

Tolerances, per element, from the arithmetic: a float32 sum of n terms is within n 2^-23 of
the sum of their magnitudes (any order; the matrix cores may truncate), a store to bfloat16
within 2^-8 and to float32 within 2^-24 of the value, the sigmoid and square root within 8
units of 2^-24 plus |z| 2^-24 for the exponent's argument.  MX8 encodings of given values are
compared bit for bit; those of computed values to half an e4m3 step of the scale used.
"""
import zlib

import numpy as np
import pytest
import torch

from tests import network_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6
SUM = 2.0 ** -23


@pytest.fixture(scope="module")
def gs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from differentiable_tile_gaussian_amd import gs as _gs
    return _gs


def rng(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g) * scale


def strided(t, pad, offset):
    """The same device matrix with `pad` more elements between rows, starting `offset`
    elements into its buffer; the rest of the buffer holds NaN (or 0x7f bytes)."""
    rows, cols = t.shape
    store = torch.empty(rows * (cols + pad) + offset, dtype=t.dtype, device="cuda")
    if t.element_size() == 1:
        store.view(torch.uint8).fill_(0x7f)
    else:
        store.fill_(float("nan"))
    out = store[offset:].view(rows, cols + pad)[:, :cols]
    out.view(torch.uint8 if t.element_size() == 1 else t.dtype).copy_(
        t.view(torch.uint8 if t.element_size() == 1 else t.dtype))
    return out


def mx8_of(gs, v, pad=0, offset=0):
    """Device Mx8 and its float64 values of a float32 host matrix."""
    codes, s = ref.mx8_encode(v.double().numpy())
    q = torch.from_numpy(codes).view(torch.float8_e4m3fn).cuda()
    sc = torch.from_numpy(s).view(torch.float8_e8m0fnu).cuda()
    return gs.Mx8(strided(q, pad, offset), strided(sc, pad % 3, offset % 5)), torch.from_numpy(ref.mx8_decode(codes, s))


def given(gs, v, kind, pad=0, offset=0):
    """Device matrix of the type and its float64 values."""
    if kind == "mx8":
        return mx8_of(gs, v, pad, offset)
    t = v.to(torch.bfloat16 if kind == "bf16" else torch.float32)
    return strided(t.cuda(), pad, offset), t.double()


def output(gs, rows, cols, kind, pad=0, offset=0):
    if kind is None:
        return None
    if kind == "mx8":
        return gs.Mx8(strided(torch.zeros(rows, cols, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), pad,
                              offset),
                      strided(torch.zeros(rows, (cols + 31) // 32, dtype=torch.uint8, device="cuda")
                              .view(torch.float8_e8m0fnu), pad % 3, offset % 5))
    dt = torch.bfloat16 if kind == "bf16" else torch.float32
    return strided(torch.full((rows, cols), float("nan"), dtype=dt, device="cuda"), pad, offset)


def untouched(t, rows, cols):
    """Whether the buffer's elements outside the matrix still hold the filler."""
    base = t._base if t._base is not None else t
    b = base.view(torch.uint8) if base.element_size() == 1 else base
    mask = torch.ones(b.numel(), dtype=torch.bool, device="cuda")
    v = mask[t.storage_offset():].as_strided((rows, cols), (t.stride(0), 1))
    v.zero_()
    rest = b.reshape(-1)[mask]
    return bool((rest == 0x7f).all() if b.dtype == torch.uint8 else torch.isnan(rest).all())


def within(got, want, tol, what):
    got, want, tol = got.double().cpu(), want.double(), torch.as_tensor(tol, dtype=torch.float64)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), [int(i) for i in bad.nonzero()[0]],
                           float(got[bad][0]), float(want[bad][0]))


def check_mx8(m, v, tol, what):
    """A computed MX8 matrix: every scale right for values within tol of v, every element
    within half an e4m3 step of v."""
    codes = m.q.view(torch.uint8).cpu().numpy()
    s = m.scales.view(torch.uint8).cpu().numpy()
    lo = ref.mx8_scale_bytes(np.maximum(np.abs(v.numpy()) - tol.numpy(), 0.0))
    hi = ref.mx8_scale_bytes(np.abs(v.numpy()) + tol.numpy())
    assert ((s >= lo) & (s <= hi)).all(), what
    step = np.exp2(s.astype(np.float64) - 127).repeat(32, axis=1)[:, :codes.shape[1]]
    half = np.maximum(np.abs(v.numpy()) * 2.0 ** -4, step * 2.0 ** -10)
    within(torch.from_numpy(ref.mx8_decode(codes, s)), v, torch.from_numpy(half) + tol, what)


def check_stored(m, kind, v, tol, what):
    if kind == "mx8":
        check_mx8(m, v, tol, what)
    else:
        within(m, v, tol * (1 + ref.UBF) + v.abs() * ref.rounding(m.dtype), what)


# ------------------------------------------------------------------------------- MX8

SPECIAL = [0.0, -0.0, 448.0, 448.1, 449.0, 464.0, 480.0, 512.0, float("inf"), float("-inf"), float("nan"), 1e-45, 1e-38,
           3.4028234e38, -3.4028234e38, 2.0 ** -126, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 17.0, 18.0, 19.0, -17.0,
           1.0625, 1.1875, 0.0, 1.0, -1.0]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (3, 31, 0, 0), (5, 32, 0, 0), (7, 33, 1, 1), (64, 59, 0, 0),
                                                  (33, 128, 8, 0), (9, 257, 3, 3), (4, 513, 0, 0), (2, 4100, 0, 1),
                                                  (1025, 64, 0, 0)])
def test_mx8_pack_and_unpack_bit_for_bit(gs, kind, rows, cols, pad, offset):
    print("mx8", kind, rows, cols, pad, offset, flush=True)
    g = rng("mx8", rows, cols)
    v = normal(g, rows, cols) * torch.exp2(torch.randint(-40, 40, (rows, 1), generator=g).float())
    flat = v.view(-1)
    at = torch.randperm(flat.numel(), generator=g)[:min(len(SPECIAL), max(flat.numel() // 40, 1))]
    flat[at] = torch.tensor(SPECIAL[:len(at)])
    if rows > 2:
        v[1] = 0.0                                          # a row of empty blocks
    x, x64 = given(gs, v, kind, pad, offset)
    q = output(gs, rows, cols, "mx8", pad, offset)
    gs.gs_mx8_pack(x, q)
    codes, s = ref.mx8_encode(x64.numpy())
    got = q.q.view(torch.uint8).cpu().numpy()
    nan = (codes & 0x7f) == 0x7f
    assert np.array_equal(q.scales.view(torch.uint8).cpu().numpy(), s)
    assert np.array_equal(got[~nan], codes[~nan]) and ((got[nan] & 0x7f) == 0x7f).all()
    assert untouched(q.q, rows, cols) and untouched(q.scales, rows, (cols + 31) // 32)
    for out_kind in ("f32", "bf16"):
        back = output(gs, rows, cols, out_kind, pad, offset)
        gs.gs_mx8_unpack(q, back)
        want = torch.from_numpy(ref.mx8_decode(codes, s))
        want = want.float() if out_kind == "f32" else want.float().bfloat16()
        assert torch.equal(torch.nan_to_num(back.cpu().float(), 1.0, 2.0, 3.0), torch.nan_to_num(want.float(), 1.0, 2.0, 3.0))
        assert untouched(back, rows, cols)


def test_mx8_unpack_reads_the_scale_range(gs):
    codes = torch.arange(128, dtype=torch.uint8).repeat(2, 1)
    codes[1] |= 0x80
    for bytes_ in ([0, 1, 127, 247], [255, 0, 254, 100]):
        s = torch.tensor([bytes_, bytes_], dtype=torch.uint8)
        q = gs.Mx8(codes.view(torch.float8_e4m3fn).cuda(), s.view(torch.float8_e8m0fnu).cuda())
        out = torch.empty(2, 128, device="cuda")
        gs.gs_mx8_unpack(q, out)
        want = torch.from_numpy(ref.mx8_decode(codes.numpy(), s.numpy())).float()
        assert torch.equal(torch.nan_to_num(out.cpu(), 1.0, 2.0, 3.0), torch.nan_to_num(want, 1.0, 2.0, 3.0))


# ------------------------------------------------------------------------------- RMS norm

NORM_SHAPES = [(1, 1, 0, 0), (1, 64, 0, 0), (5, 3, 0, 0), (130, 32, 0, 0), (67, 59, 0, 0), (1025, 64, 8, 0), (300, 128, 0, 0),
               (41, 200, 1, 1), (18, 256, 0, 0), (9, 1000, 0, 0), (6, 1024, 0, 0), (5, 2047, 3, 0), (3, 4096, 0, 0),
               (7, 4097, 0, 0), (2, 9001, 5, 1), (5000, 128, 0, 0)]


def norm_tol(cols):
    """Relative error of rstd in float32: the sum's chain, the mean, the root."""
    return (cols / 64 + 24) * ref.U24


@pytest.mark.parametrize("rows,cols,pad,offset", NORM_SHAPES)
@pytest.mark.parametrize("xk,rk,hk,ck,yk", [("f32", None, None, False, "f32"), ("bf16", "bf16", "bf16", True, "mx8"),
                                            ("bf16", "f32", "f32", False, "bf16"), ("f32", "bf16", "bf16", True, "mx8")])
def test_rmsnorm_forward(gs, rows, cols, pad, offset, xk, rk, hk, ck, yk):
    print("rmsnorm_fwd", rows, cols, xk, rk, hk, ck, yk, flush=True)
    g = rng("norm", rows, cols)
    v = normal(g, rows, cols) * torch.exp(normal(g, rows, 1))
    if rows > 4:
        v[3] = 0.0
    x, x64 = given(gs, v, xk, pad, offset)
    r, r64 = given(gs, normal(g, rows, cols) * (torch.arange(rows) != 3)[:, None], rk, pad, offset) if rk else (None, None)
    w = (1 + 0.2 * normal(g, cols))
    y, h, ckpt = (output(gs, rows, cols, k, pad, offset) for k in (yk, hk, "mx8" if ck else None))
    rstd = torch.full((rows,), float("nan"), device="cuda")
    gs.gs_rmsnorm_fwd(x, w.cuda(), EPS, y, rstd, residual=r, h=h, ckpt=ckpt)
    h64, rstd64, y64 = ref.rmsnorm(x64, r64, w.double(), EPS)
    t = norm_tol(cols)
    within(rstd, rstd64, rstd64 * t, "rstd")
    check_stored(y, yk, y64, y64.abs() * (t + 4 * ref.U24) + (h64.abs() + x64.abs()) * rstd64[:, None] * w.abs() * ref.U24, "y")
    htol = x64.abs() * ref.U24 * 2
    if h is not None:
        check_stored(h, hk, h64, htol, "h")
        assert untouched(h, rows, cols)
    if ckpt is not None:
        check_mx8(ckpt, h64, htol, "ckpt")
    if yk != "mx8":
        assert untouched(y, rows, cols)


@pytest.mark.parametrize("cols", [3, 9, 59, 96, 513, 1000, 1025, 2047, 4095, 4097])
def test_rmsnorm_forward_in_place(gs, cols):
    g = rng("inplace", cols)
    x, r = (normal(g, 50, cols).bfloat16().cuda() for _ in range(2))
    w = torch.ones(cols, device="cuda")
    y, h = (torch.empty(50, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gs.gs_rmsnorm_fwd(x, w, EPS, y, residual=r, h=h)
    r2, y2 = r.clone(), torch.empty_like(y)
    gs.gs_rmsnorm_fwd(x, w, EPS, y2, residual=r2, h=r2)
    assert torch.equal(r2, h) and torch.equal(y2, y)


@pytest.mark.parametrize("rows,cols,pad,offset", NORM_SHAPES)
@pytest.mark.parametrize("dk,hk,rk,ok", [("bf16", "mx8", "bf16", "bf16"), ("f32", "f32", None, "f32"),
                                         ("bf16", "bf16", "f32", "f32"), ("f32", "mx8", "f32", "bf16")])
def test_rmsnorm_backward(gs, rows, cols, pad, offset, dk, hk, rk, ok):
    print("rmsnorm_bwd", rows, cols, dk, hk, rk, ok, flush=True)
    g = rng("normgrad", rows, cols)
    h, h64 = given(gs, normal(g, rows, cols), hk, pad, offset)
    dy, dy64 = given(gs, normal(g, rows, cols, scale=1e-5) * (torch.rand(rows, 1, generator=g) > 0.3), dk, pad, offset)
    dres, dres64 = given(gs, normal(g, rows, cols, scale=1e-5), rk, pad, offset) if rk else (None, None)
    w = 1 + 0.2 * normal(g, cols)
    rstd = torch.rsqrt(h64.square().mean(1) + EPS).float()
    dh = output(gs, rows, cols, ok, pad, offset)
    dw = torch.full((cols,), float("nan"), device="cuda")
    ws = gs.workspace(gs.GS_WS_RMSNORM_BWD, n=rows, W=cols)
    gs.gs_rmsnorm_bwd(dy, h, w.cuda(), rstd.cuda(), dh, dw, ws, dres=dres)
    dh64, dw64 = ref.rmsnorm_grads(dy64, h64, w.double(), rstd.double(), dres64)
    xhat, u = h64 * rstd.double()[:, None], dy64 * w.double()
    scale = rstd.double()[:, None] * (u.abs() + xhat.abs() * (u * xhat).abs().mean(1, keepdim=True))
    if dres64 is not None:
        scale = scale + dres64.abs()
    check_stored(dh, ok, dh64, scale * (cols / 64 + 32) * ref.U24, "dh")
    within(dw, dw64, (dy64 * xhat).abs().sum(0) * (min(rows, 512) + 64) * ref.U24, "dw")
    assert untouched(dh, rows, cols)
    # the same bits again, without the weight's gradient and in place of dres
    if dres is not None and rk == ok:
        gs.gs_rmsnorm_bwd(dy, h, w.cuda(), rstd.cuda(), dres, None, ws, dres=dres)
        assert torch.equal(dres, dh)


def test_rmsnorm_gradient_against_differences(gs):
    g = rng("normdiff")
    rows, cols = 4, 37
    x, w, dy = normal(g, rows, cols), 1 + 0.2 * normal(g, cols), normal(g, rows, cols)
    rstd = torch.empty(rows, device="cuda")
    y, dh, dw = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda")
    gs.gs_rmsnorm_fwd(x.cuda(), w.cuda(), EPS, y, rstd)
    gs.gs_rmsnorm_bwd(dy.cuda(), x.cuda(), w.cuda(), rstd, dh, dw, gs.workspace(gs.GS_WS_RMSNORM_BWD, n=rows, W=cols))

    def loss(x_, w_):
        return float((ref.rmsnorm(x_, None, w_, EPS)[2] * dy.double()).sum())
    d = 1e-5
    for i in range(rows):
        for j in range(0, cols, 5):
            e = torch.zeros(rows, cols, dtype=torch.float64)
            e[i, j] = d
            num = (loss(x.double() + e, w.double()) - loss(x.double() - e, w.double())) / (2 * d)
            assert abs(num - float(dh[i, j])) < 1e-4
    for j in range(cols):
        e = torch.zeros(cols, dtype=torch.float64)
        e[j] = d
        num = (loss(x.double(), w.double() + e) - loss(x.double(), w.double() - e)) / (2 * d)
        assert abs(num - float(dw[j])) < 1e-4


# ------------------------------------------------------------------------------- linear layers

# rows, in, out: single values, single rows, widths across the tiles' edges, narrow and wide
LINEAR_SHAPES = [(1, 1, 1), (1, 1024, 1024), (2, 64, 48), (17, 35, 59), (64, 32, 64), (1000, 128, 128), (513, 64, 48),
                 (300, 257, 130), (129, 1024, 384), (4097, 96, 200), (64, 300, 2000), (33, 256, 256), (2050, 3, 3),
                 (5, 4096, 40), (700, 512, 640), (257, 129, 65), (1, 5000, 7)]
# widths of more than two column groups against one, and results of 65 to 128 and of more tiles
LINEAR_SHAPES += [(300, 200, 33), (300, 33, 200), (513, 256, 64), (513, 64, 256), (300, 7, 200), (300, 200, 7),
                  (1100, 80, 1000), (1030, 83, 1001), (2100, 48, 1104), (2100, 45, 1101)]
PITCHES = [(0, 0), (3, 1), (8, 0)]


@pytest.mark.parametrize("rows,k,n", LINEAR_SHAPES + [(3200, 2048, 2048)])
@pytest.mark.parametrize("xk,act,rk,zk,yk,pitch", [("bf16", "none", None, None, "f32", 0), ("mx8", "silu", None, "mx8", "bf16", 0),
                                                   ("mx8", "gelu", "bf16", "bf16", "bf16", 1),
                                                   ("bf16", "relu", "f32", "mx8", "f32", 2),
                                                   ("bf16", "silu", "bf16", "f32", "bf16", 1)])
def test_linear_forward(gs, rows, k, n, xk, act, rk, zk, yk, pitch):
    print("linear_fwd", rows, k, n, xk, act, rk, zk, yk, flush=True)
    pad, off = PITCHES[pitch]
    g = rng("linear", rows, k, n)
    x, x64 = given(gs, normal(g, rows, k), xk, pad, off)
    w, w64 = given(gs, normal(g, n, k, scale=k ** -0.5), "bf16", pad, off)
    b = 0.3 * normal(g, n)
    r, r64 = given(gs, normal(g, rows, n), rk, pad, off) if rk else (None, None)
    y, z = output(gs, rows, n, yk, pad, off), output(gs, rows, n, zk, pad, off)
    gs.gs_linear_fwd(x, w, y, bias=b.cuda(), act=act, residual=r, z=z)
    z64, y64 = ref.linear(x64, w64, b.double(), act, r64)
    ztol = (x64.abs() @ w64.abs().t() + b.abs().double()) * (k + 2) * SUM
    ytol = 1.2 * ztol + z64.abs() * (z64.abs() + 16) * ref.U24 + (0 if r64 is None else r64.abs() * 2 * ref.U24)
    check_stored(y, yk, y64, ytol, "y")
    assert untouched(y, rows, n)
    if z is not None:
        check_stored(z, zk, z64, ztol, "z")
        if zk == "mx8":
            assert untouched(z.q, rows, n) and untouched(z.scales, rows, (n + 31) // 32)
    if rk == yk:                                          # y in place of the residual
        gs.gs_linear_fwd(x, w, r, bias=b.cuda(), act=act, residual=r)
        assert torch.equal(r, y)


@pytest.mark.parametrize("rows,k,n", LINEAR_SHAPES)
@pytest.mark.parametrize("dk,xk,zk,act,dxk,dwk,pitch", [("f32", "bf16", None, "none", "bf16", "f32", 0),
                                                        ("bf16", "bf16", None, "none", "f32", "f32", 1),
                                                        ("bf16", "mx8", "mx8", "silu", "bf16", "bf16", 0),
                                                        ("f32", "mx8", "bf16", "gelu", "f32", "f32", 1),
                                                        ("bf16", "bf16", "f32", "relu", "bf16", "f32", 2)])
def test_linear_backward(gs, rows, k, n, dk, xk, zk, act, dxk, dwk, pitch):
    print("linear_bwd", rows, k, n, dk, xk, zk, act, dxk, dwk, flush=True)
    pad, off = PITCHES[pitch]
    g = rng("lineargrad", rows, k, n)
    x, x64 = given(gs, normal(g, rows, k), xk, pad, off)
    w, w64 = given(gs, normal(g, n, k, scale=k ** -0.5), "bf16", pad, off)
    dy, dy64 = given(gs, normal(g, rows, n, scale=1e-6) * (torch.rand(rows, 1, generator=g) > 0.3), dk, pad, off)
    z, z64 = given(gs, normal(g, rows, n, scale=2.0), zk, pad, off) if zk else (None, None)
    dx, dw = output(gs, rows, k, dxk, pad, off), output(gs, n, k, dwk, pad, off)
    db = torch.full((n,), float("nan"), device="cuda")
    ws = gs.workspace(gs.GS_WS_LINEAR_BWD, n=rows, W=k, H=n)
    gs.gs_linear_bwd(dy, x, w, dx, dw, db, ws, act=act, z=z)
    dz64, dx64, dw64, db64 = ref.linear_grads(dy64, z64, act, x64, w64)
    # dz: exact for a bfloat16 dy without activation, else rounded once
    rdz = 0.0 if (dk == "bf16" and act == "none") else ref.UBF
    slope = 0.0 if act == "none" else 1.0
    dztol = dy64.abs() * slope * (0 if z64 is None else z64.abs() + 24) * ref.U24
    check_stored(dx, dxk, dx64, (dz64.abs() @ w64.abs()) * (rdz + (n + 2) * SUM) + dztol @ w64.abs(), "dx")
    check_stored(dw, dwk, dw64, (dz64.abs().t() @ x64.abs()) * (rdz + (rows + 2) * SUM) + dztol.t() @ x64.abs(), "dw")
    within(db, db64, dz64.abs().sum(0) * (min(rows, 1024) + 64) * ref.U24 + dztol.sum(0), "db")
    assert untouched(dx, rows, k) and untouched(dw, n, k)
    # each output alone gives the same bits
    for want in range(3):
        one = [torch.full_like(t, float("nan")) if i == want else None for i, t in enumerate((dx, dw, db))]
        gs.gs_linear_bwd(dy, x, w, *one, ws, act=act, z=z)
        assert torch.equal(one[want], (dx, dw, db)[want]), want


@pytest.mark.parametrize("n", [7, 16, 40, 65, 67, 79, 80, 130, 200, 300])
@pytest.mark.parametrize("rows", [100, 20000])
def test_linear_in_place_of_the_residual(gs, rows, n):
    """The same bits with y in place of the residual, at widths whose last columns are taken
    from inside the row, with the column groups in one block and in several."""
    print("linear in place", rows, n, flush=True)
    g = rng("inplacelinear", rows, n)
    x, w = normal(g, rows, 20).bfloat16().cuda(), normal(g, n, 20).bfloat16().cuda()
    for dt in (torch.bfloat16, torch.float32):
        r = normal(g, rows, n).to(dt).cuda()
        y = torch.empty_like(r)
        gs.gs_linear_fwd(x, w, y, act="silu", residual=r)
        gs.gs_linear_fwd(x, w, r, act="silu", residual=r)
        assert torch.equal(r, y)


def test_linear_gradient_against_differences(gs):
    g = rng("lineardiff")
    rows, k, n = 3, 7, 5
    x, w = normal(g, rows, k).bfloat16(), normal(g, n, k).bfloat16()
    b, dy = normal(g, n), normal(g, rows, n).bfloat16()
    for act in ("silu", "gelu"):
        y, z = torch.empty(rows, n, device="cuda"), torch.empty(rows, n, device="cuda")
        gs.gs_linear_fwd(x.cuda(), w.cuda(), y, bias=b.cuda(), act=act, z=z)
        dx, dw, db = torch.empty(rows, k, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
        gs.gs_linear_bwd(dy.cuda(), x.cuda(), w.cuda(), dx, dw, db, gs.workspace(gs.GS_WS_LINEAR_BWD, n=rows, W=k, H=n), act=act,
                         z=z)
        args = [t.double() for t in (x, w, b)]

        def loss(x_, w_, b_):
            return float((ref.linear(x_, w_, b_, act)[1] * dy.double()).sum())
        for i, got in enumerate((dx, dw, db)):
            got = got.cpu().double()
            for j in range(got.numel()):
                e = torch.zeros_like(args[i]).view(-1)
                e[j] = 1e-5
                lo, hi = ([a + s * e.view(a.shape) if m == i else a for m, a in enumerate(args)] for s in (-1, 1))
                num = (loss(*hi) - loss(*lo)) / 2e-5
                # dz rounds to bfloat16: 2^-8 of sums of magnitudes below 16
                assert abs(num - float(got.view(-1)[j])) < 16 * ref.UBF


# ------------------------------------------------------------------------------- edges

def test_no_rows(gs):
    def empty(c, dt=torch.bfloat16):
        return torch.empty(0, c, dtype=dt, device="cuda")
    gs.gs_mx8_pack(empty(40), gs.mx8_empty(0, 40))
    gs.gs_mx8_unpack(gs.mx8_empty(0, 40), empty(40))
    w = torch.ones(40, device="cuda")
    gs.gs_rmsnorm_fwd(empty(40), w, EPS, empty(40))
    dw = torch.full((40,), 7.0, device="cuda")
    gs.gs_rmsnorm_bwd(empty(40), empty(40), w, torch.empty(0, device="cuda"), empty(40), dw,
                      gs.workspace(gs.GS_WS_RMSNORM_BWD, n=0, W=40))
    assert (dw == 0).all()
    for k, n in ((40, 24), (500, 300)):
        wt = torch.ones(n, k, dtype=torch.bfloat16, device="cuda")
        gs.gs_linear_fwd(empty(k), wt, empty(n))
        dwt, db = torch.full((n, k), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
        gs.gs_linear_bwd(empty(n), empty(k), wt, empty(k), dwt, db, gs.workspace(gs.GS_WS_LINEAR_BWD, n=0, W=k, H=n),
                         act="silu", z=empty(n))
        assert (dwt == 0).all() and (db == 0).all()


@pytest.mark.parametrize("k,n", [(64, 64), (320, 96)])
def test_rows_do_not_mix(gs, k, n):
    """NaN and infinity in one row reach that row alone; in 8 bits, that element alone."""
    g = rng("nan", k, n)
    x, w = normal(g, 40, k).bfloat16().cuda(), normal(g, n, k).bfloat16().cuda()
    y = [torch.empty(40, n, device="cuda") for _ in range(2)]
    z = [gs.mx8_empty(40, n) for _ in range(2)]
    gs.gs_linear_fwd(x, w, y[0], z=z[0])
    x2 = x.clone()
    x2[11, 5], x2[30, 0] = float("nan"), float("inf")
    gs.gs_linear_fwd(x2, w, y[1], z=z[1])
    keep = torch.ones(40, dtype=torch.bool)
    keep[[11, 30]] = False
    assert torch.equal(y[0][keep], y[1][keep]) and not torch.isfinite(y[1][[11, 30]]).any()
    assert torch.equal(z[0].q.view(torch.uint8)[keep], z[1].q.view(torch.uint8)[keep])
    h = torch.randn(8, 64, device="cuda")
    h2 = h.clone()
    h2[2, 3] = float("inf")
    q = [gs.mx8_empty(8, 64) for _ in range(2)]
    for a, b in zip((h, h2), q):
        gs.gs_mx8_pack(a, b)
    differ = q[0].q.view(torch.uint8) != q[1].q.view(torch.uint8)
    top = h[2, :32].abs().argmax() == 3
    assert differ.sum() == 1 or top


def test_offsets_past_32_bits(gs):
    """Rows so far apart that element offsets pass 2^31 and byte offsets 2^32."""
    rows, k, n, ld = 5, 48, 40, (1 << 29) + 72
    g = rng("far")

    def far(cols, dt):
        return torch.empty(rows * ld, dtype=dt, device="cuda").view(rows, ld)[:, :cols]
    store_x, store_y = far(k, torch.bfloat16), far(n, torch.bfloat16)
    x = normal(g, rows, k).bfloat16()
    store_x.copy_(x)
    w = normal(g, n, k).bfloat16().cuda()
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    gs.gs_linear_fwd(x.cuda(), w, y, act="silu")
    gs.gs_linear_fwd(store_x, w, store_y, act="silu")
    assert torch.equal(store_y, y)
    ws = gs.workspace(gs.GS_WS_LINEAR_BWD, n=rows, W=k, H=n)
    out = [[torch.empty(rows, k, dtype=torch.bfloat16, device="cuda"), torch.empty(n, k, device="cuda"),
            torch.empty(n, device="cuda")] for _ in range(2)]
    gs.gs_linear_bwd(y, x.cuda(), w, *out[0], ws)
    gs.gs_linear_bwd(store_y, store_x, w, *out[1], ws)
    assert all(torch.equal(a, b) for a, b in zip(*out))
    wn = torch.ones(k, device="cuda")
    a, b = torch.empty(rows, k, device="cuda"), torch.empty(rows, k, device="cuda")
    gs.gs_rmsnorm_fwd(x.cuda(), wn, EPS, a)
    gs.gs_rmsnorm_fwd(store_x, wn, EPS, b)
    assert torch.equal(a, b)
    q = [gs.mx8_empty(rows, k) for _ in range(2)]
    gs.gs_mx8_pack(x.cuda(), q[0])
    gs.gs_mx8_pack(store_x, q[1])
    assert torch.equal(q[0].q.view(torch.uint8), q[1].q.view(torch.uint8))


def _block(gs, x, w1, w2, b1, b2, wn):
    """A residual feed-forward block and its gradients through 8-bit checkpoints."""
    rows, k, n = x.shape[0], w1.shape[1], w1.shape[0]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    a, z, hk = gs.mx8_empty(rows, k), gs.mx8_empty(rows, n), gs.mx8_empty(rows, k)
    rstd, u, y = torch.empty(rows, device="cuda"), torch.empty(rows, n, **bf), torch.empty(rows, k, **bf)
    gs.gs_rmsnorm_fwd(x, wn, EPS, a, rstd, ckpt=hk)
    gs.gs_linear_fwd(a, w1, u, bias=b1, act="silu", z=z)
    gs.gs_linear_fwd(u, w2, y, bias=b2, residual=x)
    du, da, dx = torch.empty(rows, n, **bf), torch.empty(rows, k, **bf), torch.empty(rows, k, **bf)
    dw1, dw2 = torch.empty(n, k, device="cuda"), torch.empty(k, n, device="cuda")
    db1, db2, dwn = torch.empty(n, device="cuda"), torch.empty(k, device="cuda"), torch.empty(k, device="cuda")
    ws2, ws1 = gs.workspace(gs.GS_WS_LINEAR_BWD, n=rows, W=n, H=k), gs.workspace(gs.GS_WS_LINEAR_BWD, n=rows, W=k, H=n)
    gs.gs_linear_bwd(y, u, w2, du, dw2, db2, ws2)
    gs.gs_linear_bwd(du, a, w1, da, dw1, db1, ws1, act="silu", z=z)
    gs.gs_rmsnorm_bwd(da, hk, wn, rstd, dx, dwn, gs.workspace(gs.GS_WS_RMSNORM_BWD, n=rows, W=k), dres=y)
    return y, dx, dw1, dw2, db1, db2, dwn


def _block_inputs(rows, k, n):
    g = rng("block", rows, k, n)
    return (normal(g, rows, k).bfloat16().cuda(), normal(g, n, k, scale=k ** -0.5).bfloat16().cuda(),
            normal(g, k, n, scale=n ** -0.5).bfloat16().cuda(), normal(g, n).cuda(), normal(g, k).cuda(),
            1 + 0.1 * normal(g, k).cuda())


@pytest.mark.parametrize("rows,k,n", [(1000, 64, 128), (300, 320, 640), (1, 128, 256)])
def test_same_bits_on_another_stream_and_in_a_graph(gs, rows, k, n):
    args = _block_inputs(rows, k, n)
    want = _block(gs, *args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _block(gs, *args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = _block(gs, *args)
    for step in range(4):
        args[0].copy_(torch.roll(args[0], 1, 0))
        for t in rec:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        eager = _block(gs, *args)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(rec, eager)), step
