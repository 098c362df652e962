"""Rows of the network operators keep to themselves: widths whose last columns end inside a
group of 64, with NaN in the padding between rows, behind the last row and in neighbouring rows.

Tolerances are those of test_gpu_network.py.
"""
import pytest
import torch

from tests import network_ref as ref
from tests.test_gpu_network import SUM, check_stored, given, normal, output, rng, untouched, within

pytestmark = pytest.mark.gpu

# widths in whole 16-column pieces: ending in the first, second and third piece of the third
# group of 64, in the fourth group, and in the first two
WIDTHS = [144, 160, 176, 208, 240, 80, 112, 16, 48]


@pytest.fixture(scope="module")
def gs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from differentiable_tile_gaussian_amd import gs as _gs
    return _gs


# what the kernel for whole pieces takes: x, act, residual, z, y
FORMS = [("bf16", "none", None, None, "f32"), ("mx8", "silu", None, "mx8", "bf16"), ("mx8", "gelu", "bf16", None, "bf16"),
         ("bf16", "relu", "f32", None, "f32"), ("mx8", "none", None, None, "bf16")]


# 8 more elements between rows keep them at multiples of 4 bytes.  33 rows: a block for every 64
# columns; 30,001 rows: all columns in one block.
@pytest.mark.parametrize("rows,k,n,pad", [(33, k, 64, pad) for k in WIDTHS for pad in (0, 8)] +
                         [(33, 64, n, 8) for n in WIDTHS] + [(30001, k, n, 8) for k, n in ((144, 48), (160, 160), (176, 240))])
@pytest.mark.parametrize("xk,act,rk,zk,yk", FORMS)
def test_forward_reads_its_row_alone(gs, rows, k, n, pad, xk, act, rk, zk, yk):
    print("linear_fwd", rows, k, n, pad, xk, act, rk, zk, yk, flush=True)
    g = rng("ownrow", rows, k, n)
    x, x64 = given(gs, normal(g, rows, k), xk, pad, 0)
    w, w64 = given(gs, normal(g, n, k, scale=k ** -0.5), "bf16", pad, 0)
    b = 0.3 * normal(g, n)
    r, r64 = given(gs, normal(g, rows, n), rk, pad, 0) if rk else (None, None)
    y, z = output(gs, rows, n, yk, pad, 0), output(gs, rows, n, zk, pad, 0)
    gs.gs_linear_fwd(x, w, y, bias=b.cuda(), act=act, residual=r, z=z)
    z64, y64 = ref.linear(x64, w64, b.double(), act, r64)
    ztol = (x64.abs() @ w64.abs().t() + b.abs().double()) * (k + 2) * SUM
    ytol = 1.2 * ztol + z64.abs() * (z64.abs() + 16) * ref.U24 + (0 if r64 is None else r64.abs() * 2 * ref.U24)
    check_stored(y, yk, y64, ytol, "y")
    assert untouched(y, rows, n)
    if z is not None:
        check_stored(z, zk, z64, ztol, "z")


@pytest.mark.parametrize("k,n", [(80, 144), (80, 160), (80, 176), (144, 208), (176, 240), (160, 80)])
@pytest.mark.parametrize("dk,xk,zk,act", [("bf16", "bf16", None, "none"), ("f32", "mx8", None, "none"), ("bf16", "mx8", "mx8", "silu")])
def test_backward_reads_its_row_alone(gs, k, n, dk, xk, zk, act):
    """dx contracts over n: the rows of dy, or of dz in a workspace full of NaN."""
    rows, pad = 61, 8
    print("linear_bwd", rows, k, n, dk, xk, zk, act, flush=True)
    g = rng("ownrowgrad", k, n)
    x, x64 = given(gs, normal(g, rows, k), xk, pad, 0)
    w, w64 = given(gs, normal(g, n, k, scale=k ** -0.5), "bf16", pad, 0)
    dy, dy64 = given(gs, normal(g, rows, n, scale=1e-6), dk, pad, 0)
    z, z64 = given(gs, normal(g, rows, n, scale=2.0), zk, pad, 0) if zk else (None, None)
    dx, dw, db = output(gs, rows, k, "bf16", pad, 0), output(gs, n, k, "f32"), torch.empty(n, device="cuda")
    ws = gs.workspace(gs.GS_WS_LINEAR_BWD, n=rows, W=k, H=n).fill_(0xff)
    gs.gs_linear_bwd(dy, x, w, dx, dw, db, ws, act=act, z=z)
    dz64, dx64, dw64, db64 = ref.linear_grads(dy64, z64, act, x64, w64)
    rdz = 0.0 if (dk == "bf16" and act == "none") else ref.UBF
    dztol = dy64.abs() * (0.0 if act == "none" else 1.0) * (0 if z64 is None else z64.abs() + 24) * ref.U24
    check_stored(dx, "bf16", dx64, (dz64.abs() @ w64.abs()) * (rdz + (n + 2) * SUM) + dztol @ w64.abs(), "dx")
    check_stored(dw, "f32", dw64, (dz64.abs().t() @ x64.abs()) * (rdz + (rows + 2) * SUM) + dztol.t() @ x64.abs(), "dw")
    within(db, db64, dz64.abs().sum(0) * (min(rows, 1024) + 64) * ref.U24 + dztol.sum(0), "db")


@pytest.mark.parametrize("k,n", [(144, 64), (160, 96), (176, 256), (208, 48), (80, 80)])
@pytest.mark.parametrize("kind", ["bf16", "mx8"])
def test_bad_rows_reach_no_other(gs, k, n, kind):
    """NaN and infinity in a row (in MX8: a NaN element and a NaN scale) leave all others' bits."""
    print("bad rows", k, n, kind, flush=True)
    g = rng("badrows", k, n)
    x, w = normal(g, 40, k), normal(g, n, k).bfloat16().cuda()
    bad = x.clone()
    bad[11], bad[30, 0], bad[39, k - 1] = float("nan"), float("inf"), float("nan")
    y = [torch.empty(40, n, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    z = [gs.mx8_empty(40, n) for _ in range(2)]
    for v, yy, zz in zip((x, bad), y, z):
        m = given(gs, v, kind)[0]
        if kind == "mx8" and v is bad:
            m.scales.view(torch.uint8)[11] = 255
        gs.gs_linear_fwd(m, w, yy, act="silu", z=zz)
    keep = torch.ones(40, dtype=torch.bool)
    keep[[11, 30, 39]] = False
    assert torch.isfinite(y[0]).all() and not torch.isfinite(y[1][[11, 30, 39]].float()).any()
    assert torch.equal(y[0][keep], y[1][keep])
    assert torch.equal(z[0].q.view(torch.uint8)[keep], z[1].q.view(torch.uint8)[keep])
    assert torch.equal(z[0].scales.view(torch.uint8)[keep], z[1].scales.view(torch.uint8)[keep])


@pytest.mark.parametrize("cols", [32, 59, 64, 200])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_bad_element_reaches_no_other(gs, cols, value, kind):
    """In 8 bits it becomes NaN; all other elements and all scales keep their bits, in its own
    block too (it is not the block's largest finite element, which sets the scale)."""
    g = rng("badelement", cols)
    x = normal(g, 24, cols)
    bad = x.clone()
    at = [(int(r), int(c)) for r, c in zip(torch.randperm(24, generator=g)[:8], torch.randint(cols, (8,), generator=g))]
    for r, c in at:
        b = c // 32 * 32
        top = int(x[r, b:b + 32].abs().argmax()) + b
        assert cols - b > 1
        bad[r, (c if c != top else b if top != b else b + 1)] = value
    q = [gs.mx8_empty(24, cols) for _ in range(2)]
    for v, m in zip((x, bad), q):
        gs.gs_mx8_pack(given(gs, v, kind)[0], m)
    hit = ~torch.isfinite(bad).cuda()
    a, b = (m.q.view(torch.uint8) for m in q)
    assert int(hit.sum()) == 8 and ((b[hit] & 0x7f) == 0x7f).all() and torch.equal(a[~hit], b[~hit])
    assert torch.equal(q[0].scales.view(torch.uint8), q[1].scales.view(torch.uint8))
