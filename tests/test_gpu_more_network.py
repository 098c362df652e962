"""The lookup, the clipping and the MX4 operators on the GPU against plain 64-bit forms on the CPU.

Tolerances, per element, from the arithmetic, as for the other network operators: a float32 sum
of n terms is within n 2^-23 of the sum of their magnitudes, a store to bfloat16 within 2^-8 and to
float32 within 2^-24 of the value, each product by a scale within 2^-24.  MX4 encodings of given
values are compared bit for bit."""
import math

import numpy as np
import pytest
import torch

from tests import more_ref as more
from tests import network_ref as ref
from tests.test_gpu_network import SUM, check_stored, given, gs, normal, output, rng, strided, untouched, within  # noqa: F401

pytestmark = pytest.mark.gpu

SPECIAL = [0.0, -0.0, 6.0, 6.01, 5.0, -5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.2500001, 1e-45, 1e-38, 2.0 ** -126, 2.0 ** -127,
           3.4028234e38, -3.4028234e38, float("inf"), float("nan"), float("-inf"), 7.0, 100.0]


def mx4_of(gs, v, pad=0, behind=0):
    """Device Mx4 and its float64 values of a float32 host matrix; pad: blocks between rows."""
    codes, s = more.mx4_encode(v.double().numpy())
    q = torch.from_numpy(more.mx4_bytes(codes, behind)).cuda()
    return gs.Mx4(strided(q, 16 * pad, 0), strided(torch.from_numpy(s).view(torch.float8_e8m0fnu).cuda(), pad, pad), v.shape[1]), \
        torch.from_numpy(more.mx4_decode(codes, s))


def operand(gs, v, kind, pad=0, offset=0):
    return mx4_of(gs, v, pad, behind=7) if kind == "mx4" else given(gs, v, kind, pad, offset)


# ------------------------------------------------------------------------------- MX4

@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (3, 5, 0, 0), (2, 8, 0, 0), (3, 31, 0, 0), (5, 32, 0, 0), (7, 33, 1, 1),
                                                  (64, 59, 0, 0), (33, 128, 8, 0), (9, 257, 3, 3), (4, 513, 0, 0),
                                                  (2, 4100, 0, 1), (1025, 64, 0, 0), (70, 7, 2, 0)])
def test_mx4_pack_and_unpack_bit_for_bit(gs, kind, rows, cols, pad, offset):
    print("mx4", kind, rows, cols, pad, offset, flush=True)
    g = rng("mx4", rows, cols)
    v = normal(g, rows, cols) * torch.exp2(torch.randint(-40, 40, (rows, 1), generator=g).float())
    flat = v.view(-1)
    at = torch.randperm(flat.numel(), generator=g)[:min(len(SPECIAL), max(flat.numel() // 40, 1))]
    flat[at] = torch.tensor(SPECIAL[:len(at)])
    if rows > 2:
        v[1] = 0.0
    x, x64 = given(gs, v, kind, pad, offset)
    blocks = (cols + 31) // 32
    q = gs.Mx4(strided(torch.zeros(rows, 16 * blocks, dtype=torch.uint8, device="cuda"), 16 * pad, 0),
               strided(torch.zeros(rows, blocks, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu), pad, offset), cols)
    gs.gs_mx4_pack(x, q)
    codes, s = more.mx4_encode(x64.numpy())
    assert np.array_equal(q.scales.view(torch.uint8).cpu().numpy(), s)
    assert np.array_equal(q.q.cpu().numpy(), more.mx4_bytes(codes))              # zeros behind the last column
    assert untouched(q.q, rows, 16 * blocks) and untouched(q.scales, rows, blocks)
    for out_kind in ("f32", "bf16"):
        back = output(gs, rows, cols, out_kind, pad, offset)
        gs.gs_mx4_unpack(q, back)
        want = torch.from_numpy(more.mx4_decode(codes, s))
        want = want.float() if out_kind == "f32" else want.float().bfloat16()
        assert torch.equal(torch.nan_to_num(back.cpu().float(), 1.0, 2.0, 3.0), torch.nan_to_num(want.float(), 1.0, 2.0, 3.0))
        assert untouched(back, rows, cols)


def test_mx4_unpack_reads_every_code_and_scale(gs):
    codes = torch.arange(16, dtype=torch.uint8).repeat(2, 16).numpy()
    for bytes_ in ([0, 1, 127, 250, 3, 130, 64, 251], [255, 0, 254, 100, 2, 200, 1, 255]):
        s = np.array([bytes_, bytes_], np.uint8)
        q = gs.Mx4(torch.from_numpy(more.mx4_bytes(codes)).cuda(), torch.from_numpy(s).view(torch.float8_e8m0fnu).cuda(), 256)
        out = torch.empty(2, 256, device="cuda")
        gs.gs_mx4_unpack(q, out)
        want = torch.from_numpy(more.mx4_decode(codes, s)).float()
        assert torch.equal(torch.nan_to_num(out.cpu(), 1.0, 2.0, 3.0), torch.nan_to_num(want, 1.0, 2.0, 3.0))


# rows, in, out: single values, single rows, widths around the blocks, steps and tiles, narrow and wide
MX4_SHAPES = [(1, 1, 1), (1, 1024, 1024), (2, 64, 48), (17, 35, 59), (64, 32, 64), (1000, 128, 128), (513, 64, 48), (5, 16, 7),
              (300, 257, 130), (129, 1024, 384), (4097, 96, 200), (64, 300, 2000), (33, 256, 256), (2050, 3, 3), (70, 31, 33),
              (5, 4096, 40), (700, 512, 640), (257, 129, 65), (1, 5000, 7), (1100, 80, 1000), (1030, 83, 1001), (2100, 48, 1104),
              (300, 160, 144), (16, 2048, 512), (3, 33, 300), (130, 640, 272)]


@pytest.mark.parametrize("rows,k,n", MX4_SHAPES + [(3200, 2048, 2048)])
@pytest.mark.parametrize("xk,act,rk,yk,pitch", [("bf16", "silu", "bf16", "bf16", 0), ("mx8", "gelu", None, "mx8", 0),
                                                ("mx4", "none", "f32", "f32", 0), ("mx4", "relu", None, "mx8", 1),
                                                ("mx8", "none", "bf16", "f32", 1), ("bf16", "relu", None, "f32", 1),
                                                ("mx4", "silu", "bf16", "bf16", 0), ("bf16", "gelu", "f32", "mx8", 2)])
def test_linear_mx4(gs, rows, k, n, xk, act, rk, yk, pitch):
    print("linear_mx4", rows, k, n, xk, act, rk, yk, pitch, flush=True)
    pad, off = [(0, 0), (3, 1), (8, 0)][pitch]
    g = rng("linear4", rows, k, n)
    x, x64 = operand(gs, normal(g, rows, k), xk, pad, off)
    w, w64 = mx4_of(gs, normal(g, n, k, scale=k ** -0.5), pad, behind=5)
    b = 0.3 * normal(g, n)
    r, r64 = given(gs, normal(g, rows, n), rk, pad, off) if rk else (None, None)
    y = output(gs, rows, n, yk, pad, off)
    gs.gs_linear_fwd(x, w, y, bias=b.cuda(), act=act, residual=r)
    z64, y64 = ref.linear(x64, w64, b.double(), act, r64)
    ztol = (x64.abs() @ w64.abs().t() + b.abs().double()) * (k + 2) * SUM
    ytol = 1.2 * ztol + z64.abs() * (z64.abs() + 16) * ref.U24 + (0 if r64 is None else r64.abs() * 2 * ref.U24)
    check_stored(y, yk, y64, ytol, "y")
    if yk == "mx8":
        assert untouched(y.q, rows, n) and untouched(y.scales, rows, (n + 31) // 32)
    else:
        assert untouched(y, rows, n)
    if rk == yk:                                          # y in place of the residual
        gs.gs_linear_fwd(x, w, r, bias=b.cuda(), act=act, residual=r)
        assert torch.equal(r, y)


@pytest.mark.parametrize("xk", ["bf16", "mx8", "mx4"])
@pytest.mark.parametrize("rows,k,n", [(3, 96, 40), (200, 128, 64), (300, 640, 300)])
def test_linear_mx4_keeps_bad_values_to_their_rows(gs, xk, rows, k, n):
    """A NaN or an infinity in a row of x, or in one of w, reaches that row, or that column, of y."""
    g = rng("bad4", xk, rows, k, n)
    xv, wv = normal(g, rows, k), normal(g, n, k)
    xv[1, 37], xv[2, 5] = float("nan"), float("inf")
    wv[33, 64] = float("nan")
    (x, _), (w, _) = operand(gs, xv, xk), mx4_of(gs, wv)
    y = torch.empty(rows, n, device="cuda")
    gs.gs_linear_fwd(x, w, y)
    bad = ~torch.isfinite(y.cpu())
    want = torch.zeros(rows, n, dtype=torch.bool)
    want[1], want[2], want[:, 33] = True, True, True
    assert torch.equal(bad, want)


def test_linear_mx4_without_bias_and_large_values(gs):
    """Scales at the ends of their range: sums that fit float32 come out."""
    g = rng("range4")
    for ex, ew in ((60, -60), (-60, 50), (100, -30), (-100, -10)):
        xv, wv = normal(g, 40, 160) * 2.0 ** ex, normal(g, 50, 160) * 2.0 ** ew
        for xk in ("bf16", "mx8", "mx4"):
            (x, x64), (w, w64) = operand(gs, xv, xk), mx4_of(gs, wv)
            y = torch.empty(40, 50, device="cuda")
            gs.gs_linear_fwd(x, w, y)
            within(y, x64 @ w64.t(), (x64.abs() @ w64.abs().t()) * 162 * SUM, (ex, ew, xk))


@pytest.mark.parametrize("rows,k,n", [(1200, 272, 1000), (3000, 1040, 700), (1100, 128, 1024), (4200, 512, 400)])
@pytest.mark.parametrize("pad,offset", [(4, 0), (0, 4), (12, 8), (1, 0)])
def test_linear_mx4_by_tiles_from_rows_of_any_alignment(gs, rows, k, n, pad, offset):
    """Rows of x in MX8 that start at multiples of 4, 8 or 1 bytes, and scales of any pitch."""
    g = rng("align4", rows, k, n)
    (x, x64), (w, w64) = given(gs, normal(g, rows, k), "mx8", pad, offset), mx4_of(gs, normal(g, n, k, scale=k ** -0.5), pad % 3, behind=3)
    y = output(gs, rows, n, "f32", pad, offset)
    gs.gs_linear_fwd(x, w, y)
    within(y, x64 @ w64.t(), (x64.abs() @ w64.abs().t()) * (k + 2) * SUM, "y")
    assert untouched(y, rows, n)


@pytest.mark.parametrize("xk", ["mx8", "mx4"])
@pytest.mark.parametrize("rows,k,n", [(1200, 272, 1007), (300, 640, 33), (20, 96, 7), (4000, 128, 113)])
def test_absent_columns_do_not_reach_a_block(gs, xk, rows, k, n):
    """y in MX8 of zero weights is zero with the smallest scale, whatever was computed before."""
    g = rng("absent4", rows, k, n)
    x, _ = operand(gs, normal(g, rows, k) * 1e30, xk)
    y = output(gs, rows, n, "mx8")
    gs.gs_linear_fwd(x, mx4_of(gs, normal(g, n, k))[0], y)
    gs.gs_linear_fwd(x, mx4_of(gs, torch.zeros(n, k))[0], y)
    assert bool((y.scales.view(torch.uint8) == 1).all()) and bool(((y.q.view(torch.uint8) & 0x7f) == 0).all())


@pytest.mark.parametrize("xk", ["bf16", "mx8", "mx4"])
@pytest.mark.parametrize("rows,k,n", [(1, 5, 40), (5, 300, 40), (300, 270, 130), (100, 40, 48), (90, 48, 64), (90, 37, 35),
                                      (1200, 400, 1000), (1200, 392, 1000), (1200, 389, 1000), (4000, 333, 300)])
def test_linear_mx4_takes_nothing_from_behind_a_row(gs, xk, rows, k, n):
    """The last block's columns that exist are zeros, those behind them are codes that its scale makes
    infinite in bfloat16: y is what the blocks in front of it give."""
    print("behind4", xk, rows, k, n, flush=True)
    g = rng("behind4", xk, rows, k, n)
    x, x64 = operand(gs, normal(g, rows, k), xk)
    wv, last = normal(g, n, k), k // 32 * 32
    wv[:, last:] = 0
    w, w64 = mx4_of(gs, wv)
    w.q[:, (k + 1) // 2:] = 0xff
    if k % 2:
        w.q[:, k // 2] = 0xf0
    w.scales.view(torch.uint8)[:, -1] = 254
    y = torch.empty(rows, n, device="cuda")
    gs.gs_linear_fwd(x, w, y)
    want, mag = x64 @ w64.t(), x64.abs() @ w64.abs().t()
    assert bool(((y.cpu().double() - want).abs() <= mag * (k + 2) * SUM).all())


def test_linear_mx4_tiles_take_turns(gs):
    """More tiles than blocks, and tiles of a single step, of which the loads of several are under way
    at once: every tile has its own bias, scales and rows."""
    g = torch.Generator(device="cuda").manual_seed(11)
    for k in (32, 128, 160, 256, 300, 544):
        x, w = torch.randn(20_000, k, generator=g, device="cuda"), torch.randn(900, k, generator=g, device="cuda")
        b = torch.randn(900, generator=g, device="cuda") * 10
        w4, x4 = gs.mx4_empty(900, k), gs.mx4_empty(20_000, k)
        gs.gs_mx4_pack(w, w4)
        gs.gs_mx4_pack(x, x4)
        x8 = gs.mx8_empty(20_000, k)
        gs.gs_mx8_pack(x, x8)
        wv = torch.empty_like(w)
        gs.gs_mx4_unpack(w4, wv)
        for q, unpack in ((x4, gs.gs_mx4_unpack), (x8, gs.gs_mx8_unpack)):
            xv, y = torch.empty_like(x), torch.empty(20_000, 900, device="cuda")
            unpack(q, xv)
            gs.gs_linear_fwd(q, w4, y, bias=b)
            want, mag = xv.double() @ wv.double().t() + b.double(), xv.double().abs() @ wv.double().abs().t() + b.double().abs()
            assert bool(((y.double() - want).abs() <= mag * (k + 2) * SUM).all()), k
            again = torch.empty_like(y)
            gs.gs_linear_fwd(q, w4, again, bias=b)
            assert torch.equal(again, y)


# ------------------------------------------------------------------------------- lookup

LOOKUP_SHAPES = [(1, 1, 1), (1, 7, 32), (5, 3, 7), (64, 10, 8), (65, 1, 64), (63, 200, 59), (1000, 64, 128), (4097, 33, 3),
                 (300, 5000, 48), (2050, 17, 257), (129, 130, 600), (20_000, 300, 33), (9000, 100_000, 16)]


def indices(g, rows, entries, how, dtype):
    if how == "one":
        i = torch.full((rows,), entries // 2)
    elif how == "skewed":
        i = (torch.rand(rows, generator=g) ** 4 * entries).long().clamp(max=entries - 1)
        i[torch.rand(rows, generator=g) < 0.1] = -1
    elif how == "outside":
        i = torch.randint(-3, entries + 3, (rows,), generator=g)
        i[::3] = torch.iinfo(dtype).min
        i[1::3] = torch.iinfo(dtype).max
    else:
        i = torch.arange(rows) % entries
    return i.to(dtype)


@pytest.mark.parametrize("rows,entries,cols", LOOKUP_SHAPES)
@pytest.mark.parametrize("tk,yk,how,dtype,pad,offset", [("f32", "bf16", "skewed", torch.int64, 0, 0), ("bf16", "f32", "outside", torch.int32, 3, 1),
                                                        ("f32", "f32", "ordered", torch.int32, 8, 0), ("bf16", "bf16", "outside", torch.int64, 0, 3)])
def test_lookup(gs, rows, entries, cols, tk, yk, how, dtype, pad, offset):
    print("lookup", rows, entries, cols, tk, yk, how, flush=True)
    g = rng("lookup", rows, entries, cols, how)
    table, t64 = given(gs, normal(g, entries, cols), tk, pad, offset)
    index, y = indices(g, rows, entries, how, dtype), output(gs, rows, cols, yk, pad, offset)
    gs.gs_lookup_fwd(table, index.cuda(), y, scale=1.7)
    want, _ = more.lookup(t64, index.long(), float(np.float32(1.7)))
    within(y, want, want.abs() * (ref.U24 + ref.rounding(y.dtype)), "y")
    assert untouched(y, rows, cols)


@pytest.mark.parametrize("rows,entries,cols", LOOKUP_SHAPES + [(150_000, 3, 16), (70_000, 20_000, 24)])
@pytest.mark.parametrize("dk,tk,how,dtype,pad,offset", [("bf16", "f32", "skewed", torch.int64, 0, 0), ("f32", "bf16", "outside", torch.int32, 3, 1),
                                                        ("f32", "f32", "one", torch.int32, 8, 0), ("bf16", "bf16", "ordered", torch.int64, 0, 3)])
def test_lookup_gradient(gs, rows, entries, cols, dk, tk, how, dtype, pad, offset):
    print("lookup_bwd", rows, entries, cols, dk, tk, how, flush=True)
    g = rng("lookupgrad", rows, entries, cols, how)
    dy, d64 = given(gs, normal(g, rows, cols, scale=1e-5) * (torch.rand(rows, 1, generator=g) > 0.3), dk, pad, offset)
    index = indices(g, rows, entries, how, dtype)
    out = output(gs, entries, cols, tk, pad, offset)
    ws = gs.workspace(gs.GS_WS_LOOKUP_BWD, n=rows + 100, W=cols, H=entries).fill_(0xff)
    gs.gs_lookup_bwd(dy, index.cuda(), out, ws, scale=-0.3)
    want, mag, count = more.lookup_grad(d64, index.long(), entries, float(np.float32(-0.3)))
    tol = mag * (count[:, None] + 1).double() * SUM
    within(out, want, tol * (1 + ref.UBF) + want.abs() * ref.rounding(out.dtype), "dtable")
    assert untouched(out, entries, cols)
    assert bool((out[(count == 0).cuda()] == 0).all())
    again = output(gs, entries, cols, tk, pad, offset)
    gs.gs_lookup_bwd(dy, index.cuda(), again, ws, scale=-0.3)
    assert torch.equal(again, out)                                     # the same bits


@pytest.mark.parametrize("rows", [2, 255, 256, 257, 4095, 4096, 4097, 131_072, 131_073])
@pytest.mark.parametrize("entries", [1, 2, 255, 256, 65_535, 70_000])
def test_lookup_gradient_sorted_in_few_launches(gs, rows, entries):
    """Around the most places that are sorted in one block, and in two launches a pass: small whole numbers
    have one sum, exactly."""
    g = rng("lookupsmall", rows, entries)
    index = torch.randint(-1, entries + 1, (rows,), generator=g)
    dy = torch.randint(-8, 9, (rows, 8), generator=g).float()        # sums exact in float32
    out = torch.empty(entries, 8, device="cuda")
    ws = gs.workspace(gs.GS_WS_LOOKUP_BWD, n=rows, W=8, H=entries).fill_(0xff)
    for dtype in (torch.int32, torch.int64):
        gs.gs_lookup_bwd(dy.cuda(), index.to(dtype).cuda(), out.fill_(7.0), ws)
        used = (index >= 0) & (index < entries)
        assert torch.equal(out.cpu(), torch.zeros(entries, 8).index_add(0, index[used], dy[used]))


def test_lookup_keeps_bad_values_to_their_entries(gs):
    """Rows of no entry may hold anything; a NaN reaches its own entry alone."""
    g = rng("badlookup")
    dy, index = normal(g, 500, 40), torch.randint(0, 20, (500,), generator=g)
    index[::7] = -1
    dy[::7] = float("nan")
    dy[index == 3] = float("inf")
    out = torch.empty(20, 40, device="cuda")
    gs.gs_lookup_bwd(dy.cuda(), index.int().cuda(), out, gs.workspace(gs.GS_WS_LOOKUP_BWD, n=500, W=40, H=20))
    finite = torch.isfinite(out.cpu()).all(1)
    assert not finite[3] and finite.sum() == 19
    table = normal(g, 20, 40)
    table[0] = float("nan")                              # what an index outside reads nothing of
    y = torch.empty(500, 40, device="cuda")
    gs.gs_lookup_fwd(table.cuda(), torch.where(index == 0, -1, index).cuda(), y)
    assert bool(torch.isfinite(y).all())


def test_lookup_without_rows(gs):
    out = torch.full((5, 9), float("nan"), device="cuda")
    empty, none = torch.empty(0, 9, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    gs.gs_lookup_bwd(empty, none, out, gs.workspace(gs.GS_WS_LOOKUP_BWD, n=0, W=9, H=5))
    assert bool((out == 0).all())
    gs.gs_lookup_fwd(out, none, empty)


def test_lookup_gradient_against_differences(gs):
    g = rng("lookupdiff")
    table, index, dy = normal(g, 6, 5), torch.tensor([0, 5, 2, 2, -1, 0, 2]), normal(g, 7, 5)
    out = torch.empty(6, 5, device="cuda")
    gs.gs_lookup_bwd(dy.cuda(), index.cuda(), out, gs.workspace(gs.GS_WS_LOOKUP_BWD, n=7, W=5, H=6), scale=0.5)

    def loss(t):
        return float((more.lookup(t, index, 0.5)[0] * dy.double()).sum())
    for i in range(6):
        for j in range(5):
            e = torch.zeros(6, 5, dtype=torch.float64)
            e[i, j] = 1e-5
            assert abs((loss(table.double() + e) - loss(table.double() - e)) / 2e-5 - float(out[i, j])) < 1e-6


# ------------------------------------------------------------------------------- clipping

def clip_check(gs, grads, out, got_norm, max_norm):
    norm, want = more.clip([t.cpu() for t in grads], max_norm)
    assert abs(float(got_norm) - norm) <= norm * 2.0 ** -22, (float(got_norm), norm)     # the sums are float64's; one rounding
    for i, (o, w) in enumerate(zip(out, want)):
        within(o, w, w.abs() * (2 * ref.U24 + ref.rounding(o.dtype)) + 2.0 ** -149, i)


@pytest.mark.parametrize("shapes", [[(1,)], [(5, 3), (7,), (1, 1)], [(128, 64), (64,), (48, 128), (48,)] * 5, [(3,)] * 70, [(0, 4), (9,), (0,)],
                                    [(1000, 59)], [(16384,), (16385,), (8191, 2)], [(7, 1001), (300, 513)], [(3, 4, 5, 7)]])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("part", [0.3, 3.0])
def test_clip(gs, shapes, kind, part):
    print("clip", shapes[:3], len(shapes), kind, part, flush=True)
    g = rng("clip", shapes, part)
    grads = [(normal(g, *s) * 1e-6).to(kind).cuda() for s in shapes]
    max_norm = part * 1e-6 * math.sqrt(sum(t.numel() for t in grads))
    ws = gs.workspace(gs.GS_WS_CLIP_GRADS).fill_(0xff)
    norm, out = torch.full((1,), float("nan"), device="cuda"), [torch.full_like(t, float("nan"), dtype=torch.float32) for t in grads]
    gs.gs_clip_grads(grads, max_norm, norm, ws, out=out)
    clip_check(gs, grads, out, norm, max_norm)
    only = torch.full((1,), float("nan"), device="cuda")
    before = [t.clone() for t in grads]
    gs.gs_clip_grads(grads, float("inf"), only, ws)
    assert torch.equal(only, norm) and all(torch.equal(a, b) for a, b in zip(grads, before))
    lists = gs.Matrices(grads)
    gs.gs_clip_grads(lists, max_norm, norm, ws)                          # in place
    assert torch.equal(only, norm)
    clip_check(gs, before, grads, norm, max_norm)


def test_clip_strided_and_blocked(gs):
    g = rng("clipstrided")
    for n, degree in ((1, 0), (63, 1), (64, 1), (200, 3), (70_001, 2)):
        P = 11 + 3 * (degree + 1) ** 2
        planar = normal(g, P, n).cuda()
        blocked = gs.to_blocked(planar, degree)
        if n % 64:
            blocked[-1, :, n % 64:] = float("nan")       # the padding is neither read nor written
        wide = strided(normal(g, 37, 29).cuda(), 6, 1)
        rest = wide.clone()
        parts = gs.blocked_matrices(blocked, n, degree) + [wide]
        norm = torch.empty(1, device="cuda")
        gs.gs_clip_grads(parts, 2.5, norm, gs.workspace(gs.GS_WS_CLIP_GRADS))
        clip_check(gs, [planar, rest], [gs.from_blocked(blocked, n, degree), wide], norm, 2.5)
        assert untouched(wide, 37, 29)
        if n % 64:
            assert bool(torch.isnan(blocked[-1, :, n % 64:]).all())


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_clip_beyond_the_squares_of_float32(gs, scale):
    grads = [normal(rng("cliprange", scale), 1000, 33).cuda() * scale]
    norm = torch.empty(1, device="cuda")
    out = [torch.empty_like(grads[0])]
    gs.gs_clip_grads(grads, 3.0 * scale, norm, gs.workspace(gs.GS_WS_CLIP_GRADS), out=out)
    clip_check(gs, grads, out, norm, 3.0 * scale)


def test_clip_of_what_is_not_finite(gs):
    ws, norm = gs.workspace(gs.GS_WS_CLIP_GRADS), torch.empty(1, device="cuda")
    for bad in (float("nan"), float("inf")):
        grads = [torch.ones(40, 9, device="cuda"), torch.ones(5, device="cuda")]
        grads[0][3, 4] = bad
        gs.gs_clip_grads(grads, 1.0, norm, ws)
        if math.isnan(bad):
            assert bool(torch.isnan(norm)) and all(bool(torch.isnan(t).all()) for t in grads)
        else:
            assert float(norm) == bad and bool((grads[1] == 0).all())
            assert bool(torch.isnan(grads[0][3, 4])) and int((grads[0] == 0).sum()) == 40 * 9 - 1
    zeros = [torch.zeros(7, 7, device="cuda")]
    gs.gs_clip_grads(zeros, 1.0, norm, ws)
    assert float(norm) == 0.0 and bool((zeros[0] == 0).all())
    gs.gs_clip_grads([], 1.0, norm.fill_(5.0), ws)
    assert float(norm) == 0.0


def test_clip_of_more_pieces_than_blocks(gs):
    g = torch.Generator(device="cuda").manual_seed(5)
    t = torch.randn(36_000_007, generator=g, device="cuda")
    norm, ws = torch.empty(1, device="cuda"), gs.workspace(gs.GS_WS_CLIP_GRADS)
    out = torch.empty_like(t)
    gs.gs_clip_grads([t], 10.0, norm, ws, out=[out])
    want = t.double().square().sum().sqrt()
    assert abs(float(norm) - float(want)) <= float(want) * 2.0 ** -22
    exact = t.double() * (10.0 / want)
    assert bool(((out.double() - exact).abs() <= exact.abs() * 3 * ref.U24).all())


# ------------------------------------------------------------------------------- together

def served(gs, t):
    """The calls of one step over shared features: lookup, a layer from 4-bit weights, its rows'
    gradient into the table, and the clipping of that with others."""
    gs.gs_lookup_fwd(t["table"], t["index"], t["x"], scale=0.5)
    gs.gs_mx4_pack(t["x"], t["x4"])
    gs.gs_linear_fwd(t["x4"], t["w4"], t["y8"], act="silu")
    gs.gs_linear_fwd(t["x"], t["w4"], t["y"], act="silu")
    gs.gs_lookup_bwd(t["x"], t["index"], t["dtable"], t["ws"])
    gs.gs_clip_grads([t["dtable"], t["y"]], 1.0, t["norm"], t["clip_ws"], out=t["out"])
    return [t[k].clone() for k in ("x", "y", "dtable", "norm")] + [t["x4"].q.clone(), t["x4"].scales.clone().view(torch.uint8),
                                                                    t["y8"].q.clone().view(torch.uint8)] + [o.clone() for o in t["out"]]


def step_buffers(gs, seed, rows=3000, entries=200, width=96, outer=160):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = {"table": torch.randn(entries, width, generator=g, device="cuda"),
         "index": torch.randint(-1, entries, (rows,), generator=g, device="cuda"),
         "x": torch.empty(rows, width, dtype=torch.bfloat16, device="cuda"), "x4": gs.mx4_empty(rows, width),
         "w4": gs.mx4_empty(outer, width), "y": torch.empty(rows, outer, device="cuda"), "y8": gs.mx8_empty(rows, outer),
         "dtable": torch.empty(entries, width, device="cuda"), "ws": gs.workspace(gs.GS_WS_LOOKUP_BWD, n=rows, W=width, H=entries),
         "clip_ws": gs.workspace(gs.GS_WS_CLIP_GRADS), "norm": torch.empty(1, device="cuda")}
    t["out"] = [torch.empty_like(t["dtable"]), torch.empty_like(t["y"])]
    gs.gs_mx4_pack(torch.randn(outer, width, generator=g, device="cuda") * 0.1, t["w4"])
    return t


def test_captured_and_replayed(gs):
    t = step_buffers(gs, 1)
    want = served(gs, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        served_only = (gs.gs_lookup_fwd(t["table"], t["index"], t["x"], scale=0.5), gs.gs_mx4_pack(t["x"], t["x4"]),
                       gs.gs_linear_fwd(t["x4"], t["w4"], t["y8"], act="silu"), gs.gs_linear_fwd(t["x"], t["w4"], t["y"], act="silu"),
                       gs.gs_lookup_bwd(t["x"], t["index"], t["dtable"], t["ws"]),
                       gs.gs_clip_grads([t["dtable"], t["y"]], 1.0, t["norm"], t["clip_ws"], out=t["out"]))
        assert all(r is None for r in served_only)
    for k in range(4):
        for key in ("x", "y", "dtable", "norm"):
            t[key].fill_(float("nan"))
        t["ws"].fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        got = [t[key] for key in ("x", "y", "dtable", "norm")] + [t["x4"].q, t["x4"].scales.view(torch.uint8), t["y8"].q.view(torch.uint8)] + t["out"]
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
        # the program's own work between replays: other values, and back
        table = t["table"].clone()
        t["table"].mul_(2.0)
        served(gs, t)
        t["table"].copy_(table)


def test_on_other_streams(gs):
    """Two steps with buffers of their own on two streams at once give each its own results."""
    steps = [step_buffers(gs, s) for s in (2, 3)]
    want = [served(gs, t) for t in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        got = []
        for t, s in zip(steps, streams):
            with torch.cuda.stream(s):
                got.append(served(gs, t))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
