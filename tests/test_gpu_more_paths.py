"""The lookup's gradient and the MX4 layers along the ways that only large or rare sizes take: sorts of
more places than one launch's histogram or of more passes, tiles taken in turn with every type of
result, products of tiles with values that are not finite, and the narrowest contraction by tiles.

Tolerances as in test_gpu_more_network.py; sums of small whole numbers are exact."""
import pytest
import torch

from tests import network_ref as ref
from tests.test_gpu_more_network import check_stored, mx4_of, normal, operand, output, rng, untouched
from tests.test_gpu_network import SUM, given, gs  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------- lookup

def whole_sums(gs, rows, entries, index, dtype, cols=4, ws_rows=None):
    """The gradient of small whole numbers, which has one sum, exactly."""
    g = rng("whole", rows, entries)
    dy = torch.randint(-8, 9, (rows, cols), generator=g).float().cuda()
    out = torch.full((entries, cols), float("nan"), device="cuda")
    ws = gs.workspace(gs.GS_WS_LOOKUP_BWD, n=ws_rows or rows, W=cols, H=entries).fill_(0xff)
    gs.gs_lookup_bwd(dy, index.to(dtype).cuda(), out, ws)
    used = (index >= 0) & (index < entries)
    want = torch.zeros(entries, cols, dtype=torch.float64).index_add(0, index[used], dy.cpu()[used].double())
    assert float(want.abs().max()) < 2.0 ** 24
    assert torch.equal(out.cpu().double(), want), (rows, entries, dtype)


# on either side of 2048 and 4096 blocks of 1024 places, behind which a block takes 4096
@pytest.mark.parametrize("rows", [2_097_153, 4_194_304, 4_194_305, 5_000_011])
@pytest.mark.parametrize("entries", [3, 40_000, 300_007])
def test_lookup_gradient_of_many_rows(gs, rows, entries):
    print("many", rows, entries, flush=True)
    g = rng("many", rows, entries)
    index = (torch.rand(rows, generator=g) ** 3 * (entries + 1)).long() - 1       # -1: no entry
    for dtype in (torch.int32, torch.int64):
        whole_sums(gs, rows, entries, index, dtype)


def test_lookup_gradient_in_a_workspace_for_more_rows(gs):
    """Fewer rows are cut into more blocks by the sort than the most are."""
    index = torch.arange(4_194_304) % 1001 - 1
    whole_sums(gs, 4_194_304, 1000, index, torch.int32, ws_rows=4_194_305)


# 2^18 entries take a key of 19 bits with the one for no entry: three passes of digits
@pytest.mark.parametrize("rows", [3000, 9000, 131_072, 200_000, 1_500_000])
@pytest.mark.parametrize("entries", [262_143, 262_144, 1 << 21])
def test_lookup_gradient_in_three_passes(gs, rows, entries):
    print("passes", rows, entries, flush=True)
    g = rng("passes", rows, entries)
    index = torch.randint(-1, entries + 1, (rows,), generator=g)
    index[:7] = torch.tensor([0, entries - 1, entries, -1, entries - 1, 262_142, 511])
    for dtype in (torch.int32, torch.int64):
        whole_sums(gs, rows, entries, index, dtype, cols=3)


@pytest.mark.parametrize("cols", [5, 48, 512])
def test_lookup_gradient_of_rows_that_mostly_have_no_entry(gs, cols):
    """The run of no entry is the longest, whatever its rows hold."""
    rows, entries = 40_000, 50
    index = torch.full((rows,), -1)
    index[::997] = torch.arange(len(index[::997])) % entries
    dy = torch.full((rows, cols), float("nan"))
    dy[::997] = torch.randint(-8, 9, (len(index[::997]), cols), generator=rng("mostly", cols)).float()
    out = torch.full((entries, cols), float("nan"), device="cuda")
    gs.gs_lookup_bwd(dy.cuda(), index.cuda(), out, gs.workspace(gs.GS_WS_LOOKUP_BWD, n=rows, W=cols, H=entries).fill_(0xff))
    used = index >= 0
    assert torch.equal(out.cpu(), torch.zeros(entries, cols).index_add(0, index[used], dy[used]))


# ------------------------------------------------------------------------------- linear from MX4

def scale_bytes(v):
    """Scale bytes of a float64 device matrix in MX8."""
    rows, cols = v.shape
    top = torch.nn.functional.pad(v.abs(), (0, -cols % 32)).view(rows, -1, 32).amax(2) / 448.0
    frac, e = torch.frexp(top)
    e = torch.where(frac == 0.5, e - 1, e)
    return torch.where(top == 0, torch.full_like(e, -126), e).clamp(min=-126) + 127


def check_turns(y, kind, want, tol, what):
    """As check_stored, on the device (the matrices are large)."""
    if kind != "mx8":
        bad = ~((y.double() - want).abs() <= tol * (1 + ref.UBF) + want.abs() * ref.rounding(y.dtype))
    else:
        s = y.scales.view(torch.uint8).long()
        assert bool((s >= scale_bytes((want.abs() - tol).clamp(min=0))).all()) and bool((s <= scale_bytes(want.abs() + tol)).all()), what
        step = torch.exp2(s.double() - 127).repeat_interleave(32, dim=1)[:, :want.shape[1]]
        half = torch.maximum(want.abs() * 2.0 ** -4, step * 2.0 ** -10)
        bad = ~((y.q.double() * step - want).abs() <= half + tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("xk", ["mx8", "mx4"])
@pytest.mark.parametrize("yk", ["bf16", "mx8", "f32"])
@pytest.mark.parametrize("rk", [None, "bf16", "f32"])
def test_linear_mx4_tiles_take_turns_to_every_type(gs, xk, yk, rk):
    """More tiles than blocks, of one step (32, 128), of two and of several, whole and cut: the stores of
    one tile are on their way while the next one's operands arrive."""
    g = torch.Generator(device="cuda").manual_seed(12)
    rows, n = 20_000, 900
    for k in (32, 128, 160, 256, 544):
        print("turns", xk, yk, rk, k, flush=True)
        x, w = torch.randn(rows, k, generator=g, device="cuda"), torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
        b = torch.randn(n, generator=g, device="cuda") * 3
        w4, wv, xv = gs.mx4_empty(n, k), torch.empty_like(w), torch.empty_like(x)
        gs.gs_mx4_pack(w, w4)
        gs.gs_mx4_unpack(w4, wv)
        xq = gs.mx4_empty(rows, k) if xk == "mx4" else gs.mx8_empty(rows, k)
        (gs.gs_mx4_pack if xk == "mx4" else gs.gs_mx8_pack)(x, xq)
        (gs.gs_mx4_unpack if xk == "mx4" else gs.gs_mx8_unpack)(xq, xv)
        r = None if rk is None else torch.randn(rows, n, generator=g, device="cuda").to(torch.bfloat16 if rk == "bf16" else torch.float32)
        y = gs.mx8_empty(rows, n) if yk == "mx8" else torch.empty(rows, n, dtype=torch.bfloat16 if yk == "bf16" else torch.float32, device="cuda")
        gs.gs_linear_fwd(xq, w4, y, bias=b, act="silu", residual=r)
        z = xv.double() @ wv.double().t() + b.double()
        want = z * torch.sigmoid(z) + (0 if r is None else r.double())
        tol = 1.2 * (xv.double().abs() @ wv.double().abs().t() + b.double().abs()) * (k + 2) * SUM + z.abs() * (z.abs() + 16) * ref.U24
        tol += 0 if r is None else r.double().abs() * 2 * ref.U24
        check_turns(y, yk, want, tol, (xk, yk, rk, k))
        if rk == yk:                                           # y in place of the residual
            gs.gs_linear_fwd(xq, w4, r, bias=b, act="silu", residual=r)
            assert torch.equal(r, y)


@pytest.mark.parametrize("xk", ["bf16", "mx8", "mx4"])
@pytest.mark.parametrize("yk", ["f32", "mx8"])
@pytest.mark.parametrize("rows,k,n", [(1200, 640, 1000), (1200, 400, 1000), (1200, 389, 1000), (2500, 10, 700)])
def test_linear_mx4_tiles_keep_bad_values_to_their_rows(gs, xk, yk, rows, k, n):
    """A NaN or an infinity in a row of x, or in one of w, reaches that row, or that column, of y, and in
    8 bits leaves the scales to the others."""
    print("bad4", xk, yk, rows, k, n, flush=True)
    g = rng("bad4 tiles", xk, rows, k, n)
    xv, wv = normal(g, rows, k), normal(g, n, k)
    good = operand(gs, xv, xk)[0], mx4_of(gs, wv)[0]
    xv[1, 3], xv[700, k - 1], xv[rows - 1, k // 2] = float("nan"), float("inf"), float("-inf")
    wv[33, 2], wv[n - 1, k - 1] = float("nan"), float("inf")
    bad = operand(gs, xv, xk)[0], mx4_of(gs, wv)[0]
    ys = []
    for x, w in (good, bad):
        y = output(gs, rows, n, yk)
        gs.gs_linear_fwd(x, w, y)
        ys.append(y)
    rows_, cols_ = torch.zeros(rows, dtype=torch.bool, device="cuda"), torch.zeros(n, dtype=torch.bool, device="cuda")
    rows_[[1, 700, rows - 1]], cols_[[33, n - 1]] = True, True
    want = rows_[:, None] | cols_
    if yk == "f32":
        assert torch.equal(~torch.isfinite(ys[1]), want) and torch.equal(ys[1][~want], ys[0][~want])
    else:
        assert torch.equal((ys[1].q.view(torch.uint8) & 0x7f) == 0x7f, want)
        blocks = torch.nn.functional.pad(cols_, (0, -n % 32)).view(-1, 32).any(1)      # with a column that is not finite
        keep = ~(rows_[:, None] | blocks)
        assert torch.equal(ys[1].scales.view(torch.uint8)[keep], ys[0].scales.view(torch.uint8)[keep])
        keep = keep.repeat_interleave(32, dim=1)[:, :n]
        assert torch.equal(ys[1].q.view(torch.uint8)[keep], ys[0].q.view(torch.uint8)[keep])
        assert bool((ys[1].scales.view(torch.uint8) < 255).all())


# contractions of fewer than 16 by tiles
@pytest.mark.parametrize("rows,k,n", [(3000, 5, 1000), (1100, 15, 1100), (2049, 1, 700)])
@pytest.mark.parametrize("xk,act,rk,yk,pitch", [("bf16", "silu", "bf16", "bf16", 0), ("mx8", "gelu", None, "mx8", 1),
                                                ("mx4", "none", "f32", "f32", 0), ("bf16", "relu", "f32", "mx8", 1),
                                                ("mx8", "none", None, "f32", 0)])
def test_linear_mx4_of_few_columns_by_tiles(gs, rows, k, n, xk, act, rk, yk, pitch):
    print("few columns", rows, k, n, xk, act, rk, yk, flush=True)
    pad, off = [(0, 0), (3, 1)][pitch]
    g = rng("linear4 few", rows, k, n)
    x, x64 = operand(gs, normal(g, rows, k), xk, pad, off)
    w, w64 = mx4_of(gs, normal(g, n, k, scale=k ** -0.5), pad, behind=5)
    b = 0.3 * normal(g, n)
    r, r64 = given(gs, normal(g, rows, n), rk, pad, off) if rk else (None, None)
    y = output(gs, rows, n, yk, pad, off)
    gs.gs_linear_fwd(x, w, y, bias=b.cuda(), act=act, residual=r)
    z64, y64 = ref.linear(x64, w64, b.double(), act, r64)
    tol = 1.2 * (x64.abs() @ w64.abs().t() + b.abs().double()) * (k + 2) * SUM + z64.abs() * (z64.abs() + 16) * ref.U24
    check_stored(y, yk, y64, tol + (0 if r64 is None else r64.abs() * 2 * ref.U24), "y")
    assert untouched(y.q, rows, n) if yk == "mx8" else untouched(y, rows, n)
