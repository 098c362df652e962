"""The network operators with more rows than the card takes at once, so that every wave or
block goes round its loop several times and the last turn is ragged.

References are the 64-bit forms, computed on the GPU; tolerances are those of
test_gpu_network.py, with a sum over the rows bounded by its longest chain of additions
(2048 rows in one block's share, 64 in the joins).  MX8 outputs are checked on the first and
last rows and a random sample.
"""
import pytest
import torch

from tests import network_ref as ref
from tests.test_gpu_network import EPS, SUM, check_mx8, output, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from differentiable_tile_gaussian_amd import gs as _gs
    return _gs


def normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def device_rng(*key):
    return torch.Generator(device="cuda").manual_seed(rng(*key).initial_seed())


def given(gs, v, kind):
    """Device matrix of the type and its float64 values (an MX8 one by the library's own
    packing, which has its own tests, read back in float32, exactly)."""
    if kind == "mx8":
        q, back = gs.mx8_empty(*v.shape), torch.empty_like(v)
        gs.gs_mx8_pack(v, q)
        gs.gs_mx8_unpack(q, back)
        return q, back.double()
    t = v.to(torch.bfloat16 if kind == "bf16" else torch.float32)
    return t, t.double()


def within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError((what, int(bad.sum()), bad.numel(), at, float(got[at]), float(want[at])))


def check(m, kind, v, tol, what):
    if kind != "mx8":
        within(m, v, tol * (1 + ref.UBF) + v.abs() * ref.rounding(m.dtype), what)
        return
    rows = v.shape[0]
    at = torch.cat([torch.arange(200), torch.arange(rows - 200, rows),
                    torch.randint(rows, (2000,), generator=rng("sample", rows))]).unique().cuda()

    class Sample:
        q, scales = m.q.view(torch.uint8)[at], m.scales.view(torch.uint8)[at]
    check_mx8(Sample, v[at].cpu(), tol[at].cpu(), what)


def matmul_t(a, b):
    return torch.matmul(a, b.t().contiguous())


# rows, in, out: whole pieces with one, two and four groups on either side; odd widths
FORWARD = [(200_003, 128, 128), (200_003, 64, 48), (200_003, 99, 113), (200_003, 35, 59), (100_003, 256, 256),
           (100_003, 144, 176), (100_003, 201, 130), (150_003, 7, 64)]


@pytest.mark.parametrize("rows,k,n", FORWARD)
@pytest.mark.parametrize("xk,act,rk,zk,yk", [("mx8", "silu", None, "mx8", "bf16"), ("bf16", "gelu", "bf16", None, "bf16"),
                                             ("bf16", "none", "f32", None, "f32")])
def test_linear_forward(gs, rows, k, n, xk, act, rk, zk, yk):
    print("linear_fwd", rows, k, n, xk, act, flush=True)
    g = device_rng("turns", rows, k, n)
    x, x64 = given(gs, normal(g, rows, k), xk)
    w, w64 = given(gs, normal(g, n, k, scale=k ** -0.5), "bf16")
    b = normal(g, n, scale=0.3)
    r, r64 = given(gs, normal(g, rows, n), rk) if rk else (None, None)
    y, z = output(gs, rows, n, yk), output(gs, rows, n, zk)
    gs.gs_linear_fwd(x, w, y, bias=b, act=act, residual=r, z=z)
    z64 = matmul_t(x64, w64) + b.double()
    y64 = ref.activation(z64, act)[0] + (0.0 if r64 is None else r64)
    ztol = (matmul_t(x64.abs(), w64.abs()) + b.abs().double()) * (k + 2) * SUM
    check(y, yk, y64, 1.2 * ztol + z64.abs() * (z64.abs() + 16) * ref.U24 + (0 if r64 is None else r64.abs() * 2 * ref.U24), "y")
    if z is not None:
        check(z, zk, z64, ztol, "z")


# one pass over the rows (both shares of a turn's rows, two and four groups) and in four launches
BACKWARD = [(40_003, 64, 48), (100_003, 64, 48), (200_003, 64, 64), (100_003, 128, 128), (100_003, 99, 113), (100_003, 256, 64),
            (100_003, 64, 200), (100_003, 7, 33), (40_003, 200, 200), (40_003, 144, 160), (40_003, 7, 200), (40_003, 300, 70)]


@pytest.mark.parametrize("rows,k,n", BACKWARD)
@pytest.mark.parametrize("dk,xk,zk,act,dxk", [("bf16", "mx8", "mx8", "silu", "bf16"), ("f32", "bf16", None, "none", "f32"),
                                              ("bf16", "bf16", "f32", "gelu", "bf16")])
def test_linear_backward(gs, rows, k, n, dk, xk, zk, act, dxk):
    print("linear_bwd", rows, k, n, dk, xk, zk, act, flush=True)
    g = device_rng("turnsgrad", rows, k, n)
    x, x64 = given(gs, normal(g, rows, k), xk)
    w, w64 = given(gs, normal(g, n, k, scale=k ** -0.5), "bf16")
    dy, dy64 = given(gs, normal(g, rows, n, scale=1e-6) * (torch.rand(rows, 1, generator=g, device="cuda") > 0.3), dk)
    z, z64 = given(gs, normal(g, rows, n, scale=2.0), zk) if zk else (None, None)
    dx, dw, db = output(gs, rows, k, dxk), output(gs, n, k, "f32"), torch.empty(n, device="cuda")
    ws = gs.workspace(gs.GS_WS_LINEAR_BWD, n=rows, W=k, H=n).fill_(0xff)
    gs.gs_linear_bwd(dy, x, w, dx, dw, db, ws, act=act, z=z)
    dz64 = dy64 if z64 is None else dy64 * ref.activation(z64, act)[1]
    rdz = ref.UBF                                          # dz's rounding
    dztol = torch.zeros_like(dy64) if z64 is None else dy64.abs() * (z64.abs() + 24) * ref.U24
    dz_abs, dz_t = dz64.abs(), dz64.t().contiguous()
    check(dx, dxk, torch.matmul(dz64, w64), torch.matmul(dz_abs, w64.abs()) * (rdz + (n + 2) * SUM) + torch.matmul(dztol, w64.abs()),
          "dx")
    within(dw, torch.matmul(dz_t, x64), torch.matmul(dz_t.abs(), x64.abs()) * (rdz + (2048 + 64) * SUM) +
           torch.matmul(dztol.t().contiguous(), x64.abs()), "dw")
    within(db, dz64.sum(0), dz_abs.sum(0) * (2048 + 64) * ref.U24 + dztol.sum(0), "db")
    # the same bits without the others, and from a workspace with other contents
    one = torch.full_like(dw, float("nan"))
    gs.gs_linear_bwd(dy, x, w, None, one, None, ws.fill_(0x7f), act=act, z=z)
    assert torch.equal(one, dw)


@pytest.mark.parametrize("rows,cols", [(60_001, 128), (200_003, 59), (200_003, 7), (15_001, 1000), (4001, 2047), (4001, 4096),
                                       (3001, 4100)])
@pytest.mark.parametrize("dk,hk,rk,ok", [("bf16", "mx8", "bf16", "bf16"), ("f32", "f32", None, "f32")])
def test_rmsnorm_backward(gs, rows, cols, dk, hk, rk, ok):
    print("rmsnorm_bwd", rows, cols, dk, hk, flush=True)
    g = device_rng("turnsnorm", rows, cols)
    h, h64 = given(gs, normal(g, rows, cols), hk)
    dy, dy64 = given(gs, normal(g, rows, cols, scale=1e-5), dk)
    dres, dres64 = given(gs, normal(g, rows, cols, scale=1e-5), rk) if rk else (None, None)
    w = 1 + normal(g, cols, scale=0.2)
    rstd = torch.rsqrt(h64.square().mean(1) + EPS).float()
    dh, dw = output(gs, rows, cols, ok), torch.empty(cols, device="cuda")
    ws = gs.workspace(gs.GS_WS_RMSNORM_BWD, n=rows, W=cols).fill_(0xff)
    gs.gs_rmsnorm_bwd(dy, h, w, rstd, dh, dw, ws, dres=dres)
    dh64, dw64 = ref.rmsnorm_grads(dy64, h64, w.double(), rstd.double(), dres64)
    xhat, u = h64 * rstd.double()[:, None], dy64 * w.double()
    scale = rstd.double()[:, None] * (u.abs() + xhat.abs() * (u * xhat).abs().mean(1, keepdim=True))
    if dres64 is not None:
        scale = scale + dres64.abs()
    check(dh, ok, dh64, scale * (cols / 64 + 32) * ref.U24, "dh")
    within(dw, dw64, (dy64 * xhat).abs().sum(0) * (512 + 64) * ref.U24, "dw")
    if rk:                                                 # in place of dres
        gs.gs_rmsnorm_bwd(dy, h, w, rstd, dres, None, ws, dres=dres)
        assert torch.equal(dres, dh)


@pytest.mark.parametrize("rows,cols", [(200_003, 128), (200_003, 59), (30_001, 1000), (9001, 2047), (5001, 4100)])
def test_rmsnorm_forward_and_packing(gs, rows, cols):
    print("rmsnorm_fwd", rows, cols, flush=True)
    g = device_rng("turnsfwd", rows, cols)
    x, x64 = given(gs, normal(g, rows, cols), "bf16")
    r, r64 = given(gs, normal(g, rows, cols), "bf16")
    w = 1 + normal(g, cols, scale=0.2)
    y, ckpt = gs.mx8_empty(rows, cols), gs.mx8_empty(rows, cols)
    h, rstd = output(gs, rows, cols, "bf16"), torch.empty(rows, device="cuda")
    gs.gs_rmsnorm_fwd(x, w, EPS, y, rstd, residual=r, h=h, ckpt=ckpt)
    h64, rstd64, y64 = ref.rmsnorm(x64, r64, w.double(), EPS)
    t = (cols / 64 + 24) * ref.U24
    within(rstd, rstd64, rstd64 * t, "rstd")
    check(h, "bf16", h64, x64.abs() * ref.U24 * 2, "h")
    check(ckpt, "mx8", h64, x64.abs() * ref.U24 * 2, "ckpt")
    check(y, "mx8", y64, y64.abs() * (t + 4 * ref.U24) + (h64.abs() + x64.abs()) * rstd64[:, None] * w.abs() * ref.U24, "y")
    # an 8-bit value is bfloat16's own: a second packing of it changes nothing
    back, again = torch.empty_like(x), gs.mx8_empty(rows, cols)
    gs.gs_mx8_unpack(ckpt, back)
    gs.gs_mx8_pack(back, again)
    b2 = torch.empty_like(back)
    gs.gs_mx8_unpack(again, b2)
    assert torch.equal(back, b2)


def test_rows_of_several_launches(gs):
    """The most rows there are, of one column: more than one launch takes, in place and not."""
    rows, step = (1 << 31) - 1, 1 << 28
    x = torch.empty((rows, 1), dtype=torch.bfloat16, device="cuda")
    for a in range(0, rows, step):
        x[a:a + step].normal_(generator=device_rng("launches", a))

    def eight(n):
        return gs.Mx8(torch.empty((n, 1), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                      torch.empty((n, 1), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu))
    q, w = eight(rows), torch.full((1,), 1.5, device="cuda")
    gs.gs_mx8_pack(x, q)
    back, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    gs.gs_mx8_unpack(q, back)
    y = torch.empty_like(x)
    gs.gs_rmsnorm_fwd(x, w, EPS, y, rstd, residual=back, h=h)
    for a in range(0, rows, step):
        n = min(step, rows - a)
        print("rows", a, n, flush=True)
        part, b, hh, yy, r = eight(n), *(torch.empty((n, 1), dtype=torch.bfloat16, device="cuda") for _ in range(3)), \
            torch.empty(n, device="cuda")
        gs.gs_mx8_pack(x[a:a + n], part)
        gs.gs_mx8_unpack(part, b)
        gs.gs_rmsnorm_fwd(x[a:a + n], w, EPS, yy, r, residual=b, h=hh)
        for whole, own in ((q.q.view(torch.uint8), part.q.view(torch.uint8)), (q.scales.view(torch.uint8), part.scales.view(torch.uint8)),
                           (back, b), (h, hh), (y, yy), (rstd, r)):
            assert torch.equal(whole[a:a + n], own), a
    gs.gs_rmsnorm_fwd(x, w, EPS, y, residual=back, h=back)
    assert torch.equal(back, h)


@pytest.mark.parametrize("rows,k,n", [(400_003, 128, 128), (400_003, 64, 48), (200_003, 99, 113), (100_003, 256, 256), (4000, 128, 128),
                                      (3000, 1024, 256), (8160, 1024, 1024), (16, 1024, 1024)])
def test_sums_are_those_of_32_bits(gs, rows, k, n):
    """z from exact operands is no farther from its value than a float32 product of them with the
    bias added, small z included, whose roundings to 8 bits show it first (1.25: the scatter of
    the two, from as few as 16384 values)."""
    print("sums", rows, k, n, flush=True)
    g = device_rng("sums", rows, k, n)
    x, x64 = given(gs, normal(g, rows, k) * torch.exp(0.5 * normal(g, 1, k)) + normal(g, 1, k, scale=0.2), "mx8")
    w, w64 = given(gs, normal(g, n, k, scale=k ** -0.5), "bf16")
    b = normal(g, n, scale=0.1)
    y, z = output(gs, rows, n, "bf16"), output(gs, rows, n, "f32")
    gs.gs_linear_fwd(x, w, y, bias=b, z=z)
    e = matmul_t(x64, w64) + b.double()
    p = matmul_t(x64.float(), w.float()) + b
    rms = e.square().mean().sqrt()
    for at in (e.abs() < 0.3 * rms, e.abs() >= 0.3 * rms):
        own, plain = ((v.double() - e)[at].square().mean().sqrt() / rms for v in (z, p))
        print("   error over the values' size: %.3g, a float32 product's %.3g" % (own, plain))
        assert own <= 1.25 * plain, (float(own), float(plain))
