"""Which kernels the network operators launch, on which device and with which grids, by a
stand-in for the HIP runtime (recording_runtime.cpp) in a process of its own: no GPU is used."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(os.path.dirname(HERE), "differentiable_tile_gaussian_amd", "libgs.so")

PRELUDE = '''
import ctypes as C, sys
rec = C.CDLL(sys.argv[1], mode=C.RTLD_GLOBAL)
gs = C.CDLL(sys.argv[2])
rec.recorder_name.restype = C.c_char_p
gs.gs_last_error.restype = C.c_char_p
gs.gs_workspace_bytes.argtypes = [C.c_int32, C.c_int64, C.c_uint32, C.c_int32, C.c_int32, C.c_void_p]
gs.gs_workspace_bytes.restype = C.c_size_t
F32, BF16, MX8 = 0, 1, 2

class Matrix(C.Structure):
    _fields_ = [("data", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64), ("ld", C.c_int64),
                ("scales_ld", C.c_int64), ("type", C.c_int32)]

at = [1 << 40]
def m(rows, cols, kind=BF16):
    at[0] += 1 << 44
    return C.byref(Matrix(at[0], at[0] + (1 << 43) if kind == MX8 else None, rows, cols, (cols + 15) // 16 * 16, (cols + 31) // 32, kind))

def kernels(status=0):
    """The launches since the last look: (mangled name, blocks along x, device)."""
    out = [(rec.recorder_name(i).decode(), rec.recorder_blocks(i) & 0xffffffff, rec.recorder_launch_device(i))
           for i in range(rec.recorder_launches())]
    rec.recorder_clear()
    return out

def fwd(rows, k, n, xk=BF16, z=None, y=BF16):
    return gs.gs_linear_fwd(m(rows, k, xk), m(n, k), None, 2, None, z and m(rows, n, z), m(rows, n, y), None)

def bwd(rows, k, n, z=None, act=0, xk=BF16):
    need = gs.gs_workspace_bytes(9, rows, 0, k, n, None)
    return gs.gs_linear_bwd(m(rows, n), m(rows, n, z) if z is not None else None, act, m(rows, k, xk), m(n, k), m(rows, k), m(n, k, F32), C.c_void_p(1 << 50),
                            C.c_void_p(1 << 51), C.c_size_t(need), None)

def ok(status):
    assert status == 0, gs.gs_last_error()
    return kernels()
'''


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    if not os.path.exists(LIB):
        pytest.skip("libgs.so is not built")
    out = str(tmp_path_factory.mktemp("recorder") / "recorder.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", os.path.join(HERE, "recording_runtime.cpp"), "-o", out], check=True)

    def run(script):
        r = subprocess.run([sys.executable, "-c", PRELUDE + script, out, LIB], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout
    return run


def test_every_device_is_allowed_the_lds(recorder):
    """Each kernel that takes more than 64 KiB of LDS is allowed it on every device that calls,
    once, and a refusal is an error of that call alone."""
    recorder('''
calls = {"rows_fwd_kernel": lambda: fwd(100000, 256, 256), "rows_fwd_any_kernel": lambda: fwd(100000, 255, 255),
         "rows_bwd_kernel": lambda: bwd(1000, 128, 128), "tile_nt_kernel": lambda: fwd(8160, 1024, 4096),
         "tile_tn_kernel": lambda: bwd(8160, 1024, 4096)}
for name, call in calls.items():
    for device in (0, 1, 7):
        rec.recorder_device(device)
        launched = ok(call())
        assert any(name in k for k, _, _ in launched) and all(d == device for _, _, d in launched), (name, launched)
        before = rec.recorder_attributes()
        ok(call())
        assert rec.recorder_attributes() == before, name
    rec.recorder_device(3)
    rec.recorder_refuse_attributes(1)
    assert call() == -4 and gs.gs_last_error(), name
    kernels()
    ok(call())
''')


def test_grids_for_the_most_rows(recorder):
    """Rows up to 2^31 - 1, the range that the header gives: no launch of 2^32 threads, and as
    many blocks as the rows take."""
    recorder('''
ROWS = (1 << 31) - 1
def norm(rows, cols, yk, ckpt, residual):
    return gs.gs_rmsnorm_fwd(m(rows, cols), m(rows, cols) if residual else None, C.c_void_p(1 << 50), C.c_float(1e-6), None,
                             m(rows, cols, MX8) if ckpt else None, m(rows, cols, yk), C.c_void_p(1 << 51), None)
# columns and rows a block: 4 to 64 lanes a row and the whole block, one and two chunks a lane
for cols, pack_rows, norm_rows in ((1, 128, 128), (7, 128, 128), (32, 128, 128), (64, 64, 64), (128, 32, 32), (256, 16, 16),
                                   (512, 8, 8), (1024, 8, 4), (2048, 8, 2), (4096, 8, 1), (4097, 8, 4)):
    for call, per in ((lambda: gs.gs_mx8_pack(m(ROWS, cols), m(ROWS, cols, MX8), None), pack_rows),
                      (lambda: gs.gs_mx8_unpack(m(ROWS, cols, MX8), m(ROWS, cols), None), pack_rows),
                      (lambda: norm(ROWS, cols, BF16, False, False), norm_rows),
                      (lambda: norm(ROWS, cols, MX8, True, True), norm_rows)):
        launched = ok(call())
        assert sum(b for _, b, _ in launched) * per >= ROWS, (cols, launched)
    norm_bwd = gs.gs_rmsnorm_bwd(m(ROWS, cols), m(ROWS, cols, MX8), C.c_void_p(1 << 50), C.c_void_p(1 << 51), None, m(ROWS, cols), C.c_void_p(1 << 52),
                                 C.c_void_p(1 << 53), C.c_size_t(1 << 40), None)
    ok(norm_bwd)
for k, n in ((1, 1), (16, 16), (64, 64), (128, 128), (256, 256), (5, 200)):
    ok(fwd(ROWS, k, n))
    ok(bwd(ROWS, k, n))
''')


def test_many_outputs_with_an_activation(recorder):
    """129 outputs on against 16 to 64 inputs go in one pass over the rows, but with an activation
    only in whole 16-column pieces and with z in 8 or 16 bits: other kernels would not hold their
    values in registers.  The workspace is enough for either way."""
    recorder('''
for k, n in ((16, 144), (64, 256), (45, 201), (33, 129), (48, 130)):
    for rows in (1, 300, 20000, 100000):
        dz = (rows * ((n + 7) // 8 * 8) * 2 + 255) // 256 * 256
        assert gs.gs_workspace_bytes(9, rows, 0, k, n, None) >= dz + k * ((n + 7) // 8 * 8) * 2, (k, n, rows)
        for z, act in ((F32, 2), (F32, 1), (F32, 0), (BF16, 2), (MX8, 3), (MX8, 0), (None, 0)):
            one_pass = act == 0 or z != F32 and k % 16 == 0 and n % 16 == 0
            names = [name for name, _, _ in ok(bwd(rows, k, n, z, act))]
            assert any("rows_bwd_kernel" in name for name in names) == one_pass, (k, n, rows, z, act, names)
            assert any("transpose_kernel" in name for name in names) != one_pass, (k, n, rows, z, act, names)
for k, n in ((64, 128), (128, 128), (256, 64), (5, 5), (99, 113)):
    assert any("rows_bwd_kernel" in name for name, _, _ in ok(bwd(1000, k, n, F32, 2)))
''')


def test_the_kernel_for_any_type_is_for_narrow_widths(recorder):
    """From 16 columns on both sides the types are compiled in, a float32 z among them."""
    recorder('''
def any_type(rows, k, n, z, act):
    name, = {name for name, _, _ in ok(bwd(rows, k, n, z, act)) if "rows_bwd_kernel" in name}
    return "ELin1ELin1ELin1E" in name       # the three types are the argument -1
for k, n in ((16, 16), (64, 48), (128, 128), (99, 113), (256, 64), (64, 128)):
    for z, act in ((F32, 2), (BF16, 1), (MX8, 3), (None, 0)):
        assert not any_type(1000, k, n, z, act), (k, n, z, act)
assert any_type(1000, 15, 64, BF16, 2) and any_type(1000, 64, 15, F32, 2)
''')
