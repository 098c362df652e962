"""Launches of the lookup, the clipping and the MX4 operators at the ends of their ranges, by the
stand-in for the HIP runtime that test_network_launches.py uses: no GPU is touched."""
from tests.test_network_launches import recorder  # noqa: F401

MORE = '''
MX4 = 4
gs.gs_lookup_fwd.argtypes = [C.c_void_p, C.c_void_p, C.c_int32, C.c_float, C.c_void_p, C.c_void_p]
gs.gs_lookup_bwd.argtypes = [C.c_void_p, C.c_void_p, C.c_int32, C.c_float, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
gs.gs_clip_grads.argtypes = [C.c_void_p, C.c_void_p, C.c_int32, C.c_double, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]

def m4(rows, cols):
    at[0] += 1 << 44
    return C.byref(Matrix(at[0], at[0] + (1 << 43), rows, cols, (cols + 31) // 32 * 32, (cols + 31) // 32, MX4))

def fwd4(rows, k, n, x=None, y=BF16):
    return gs.gs_linear_fwd(x or m4(rows, k), m4(n, k), None, 2, None, None, m(rows, n, y), None)
'''


def test_grids_for_the_most_rows(recorder):  # noqa: F811
    recorder(MORE + '''
ROWS = (1 << 31) - 1
for cols, per in ((1, 128), (32, 128), (64, 64), (256, 16), (512, 8), (4097, 8)):
    for call in (lambda: gs.gs_mx4_pack(m(ROWS, cols), m4(ROWS, cols), None), lambda: gs.gs_mx4_unpack(m4(ROWS, cols), m(ROWS, cols), None)):
        assert sum(b for _, b, _ in ok(call())) * per >= ROWS, cols
for k, n in ((1, 1), (16, 16), (128, 128), (256, 256), (5, 200), (300, 64)):
    for x in (None, m(ROWS, k), m(ROWS, k, MX8)):
        ok(fwd4(ROWS, k, n, x, MX8))
for cols in (1, 8, 64, 256):
    ok(gs.gs_lookup_fwd(m(1000, cols, F32), 1 << 50, 8, 1.0, m(ROWS, cols), None))
    ok(gs.gs_lookup_bwd(m(ROWS, cols), 1 << 50, 4, 1.0, m(ROWS, cols, F32), 1 << 51, 1 << 45, None))
    ok(gs.gs_lookup_bwd(m(1, cols), 1 << 50, 4, 1.0, m(ROWS, cols, F32), 1 << 51, 1 << 45, None))
''')


def test_clip_in_as_many_launches_as_the_list_takes(recorder):  # noqa: F811
    recorder(MORE + '''
for count in (0, 1, 32, 33, 1000, 1024):
    many = (Matrix * max(count, 1))(*[Matrix((1 << 40) + (i << 20), None, 3, 5, 7, 0, F32) for i in range(count)])
    names = [name for name, _, _ in ok(gs.gs_clip_grads(many, None, count, 1.0, 16, 64, 1 << 20, None))]
    assert sum("squares_kernel" in n for n in names) == (count + 31) // 32 and sum("clip_kernel" in n for n in names) == 1
    names = [name for name, _, _ in ok(gs.gs_clip_grads(many, many, count, 1.0, 16, 64, 1 << 20, None))]
    assert sum("clip_kernel" in n for n in names) == max((count + 31) // 32, 1)
# the sums fit the workspace: at most 2048 blocks together
big = (Matrix * 1024)(*[Matrix((1 << 40) + (i << 30), None, 1 << 14, 1 << 10, 1 << 10, 0, F32) for i in range(1024)])
blocks = [b for n, b, _ in ok(gs.gs_clip_grads(big, None, 1024, 1.0, 16, 64, 1 << 20, None)) if "squares_kernel" in n]
assert sum(blocks) <= 2048 and len(blocks) == 32
''')


def test_every_device_is_allowed_the_lds(recorder):  # noqa: F811
    recorder(MORE + '''
for call, name in ((lambda: fwd4(8160, 1024, 4096), "tile_mx4_kernel"), (lambda: fwd4(8160, 1024, 4096, m(8160, 1024, MX8)), "tile_mx4_kernel"),
                   (lambda: fwd4(8160, 1024, 4096, m(8160, 1024)), "tile_nt_kernel"), (lambda: fwd4(100000, 256, 256), "rows_fwd_kernel"),
                   (lambda: fwd4(100000, 255, 255), "rows_fwd_any_kernel")):
    for device in (0, 1, 7):
        rec.recorder_device(device)
        launched = ok(call())
        assert any(name in k for k, _, _ in launched) and all(d == device for _, _, d in launched), (name, launched)
    rec.recorder_device(3)
    rec.recorder_refuse_attributes(1)
    assert call() == -4 and gs.gs_last_error(), name
    kernels()
    ok(call())
for rows, k, n in ((1, 1024, 1024), (16, 128, 128), (64, 4096, 1024), (700, 1024, 1024)):
    for x in (None, m(rows, k), m(rows, k, MX8)):
        assert [("linear_mx4_kernel" in name) for name, _, _ in ok(fwd4(rows, k, n, x))] == [True], (rows, k, n)
''')
