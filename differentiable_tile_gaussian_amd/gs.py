"""ctypes binding of libgs.so (include/gs.h).

The functions below have the names of the C entry points and do argument
marshalling only: torch tensors supply device memory and the current HIP stream,
every step of the rasteriser runs in the library's HIP kernels.  There is no CPU
fallback: if libgs.so is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np
import torch  # noqa: F401  (loads the HIP runtime the library then binds to)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgs.so")

GS_OK, GS_ERR_INVALID_ARG, GS_ERR_CAPACITY, GS_ERR_UNSUPPORTED, GS_ERR_HIP = 0, -1, -2, -3, -4
GS_WS_PREPROCESS, GS_WS_BIN_SORT, GS_WS_LOSS, GS_WS_RENDER, GS_WS_DENSIFY, GS_WS_LOSS_CHARBONNIER = 0, 1, 2, 3, 4, 5
GS_WS_CAMERA_GRAD, GS_WS_RELOCATE, GS_WS_RMSNORM_BWD, GS_WS_LINEAR_BWD, GS_WS_LOOKUP_BWD, GS_WS_CLIP_GRADS = 6, 7, 8, 9, 10, 11
GS_GRAD_SUMS_FLOAT, GS_GRAD_SUMS_FIXED = 0, 1
GS_MAT_F32, GS_MAT_BF16, GS_MAT_MX8, GS_MAT_MX4 = 0, 1, 2, 4
GS_CLIP_MAX = 1024
GS_ACT_NONE, GS_ACT_RELU, GS_ACT_SILU, GS_ACT_GELU = 0, 1, 2, 3
ACTIVATIONS = {"none": GS_ACT_NONE, "relu": GS_ACT_RELU, "silu": GS_ACT_SILU, "gelu": GS_ACT_GELU}

EXPORTED = ("gs_preprocess", "gs_bin_sort", "gs_render_fwd", "gs_loss_l1_dssim", "gs_render_bwd",
            "gs_adam_step", "gs_render_bwd_adam", "gs_render_bwd_adam_project", "gs_render_bwd_weighted",
            "gs_camera_grad", "gs_densify_accumulate", "gs_densify", "gs_relocate", "gs_loss_charbonnier",
            "gs_workspace_bytes", "gs_loss_l1_dssim_noalloc", "gs_profile_enable", "gs_profile_query", "gs_param_floats", "gs_params_to_blocked",
            "gs_params_from_blocked", "gs_mx8_pack", "gs_mx8_unpack", "gs_rmsnorm_fwd", "gs_rmsnorm_bwd",
            "gs_linear_fwd", "gs_linear_bwd", "gs_mx4_pack", "gs_mx4_unpack", "gs_lookup_fwd", "gs_lookup_bwd",
            "gs_clip_grads", "gs_last_error")


class GsError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"gs status {status}: {message}")
        self.status = status


class GsCamera(C.Structure):
    _fields_ = [("R", C.c_float * 9), ("t", C.c_float * 3), ("campos", C.c_float * 3),
                ("fx", C.c_float), ("fy", C.c_float), ("cx", C.c_float), ("cy", C.c_float),
                ("width", C.c_int32), ("height", C.c_int32), ("znear", C.c_float), ("bg", C.c_float * 3)]


class GsScene(C.Structure):
    _fields_ = [("n", C.c_int64), ("sh_degree", C.c_int32), ("params", C.c_void_p)]


class GsConfig(C.Structure):
    """gs_config: the per-call settings (defaults: float sums, every SH band, no Mip
    compensation, the default split sizes)."""
    _fields_ = [("grad_sums", C.c_int32), ("active_sh_degree", C.c_int32), ("mip_compensation", C.c_int32),
                ("split_first", C.c_int32), ("split_chunk", C.c_int32)]

    def __init__(self, grad_sums=GS_GRAD_SUMS_FLOAT, active_sh_degree=-1, mip_compensation=False, split_first=0,
                 split_chunk=0):
        super().__init__(int(grad_sums), int(active_sh_degree), int(bool(mip_compensation)), int(split_first),
                         int(split_chunk))


def _cfg(cfg):
    return None if cfg is None else C.byref(cfg)


class GsProj(C.Structure):
    _fields_ = [("splat", C.c_void_p), ("depth", C.c_void_p), ("rect", C.c_void_p), ("tiles", C.c_void_p),
                ("order", C.c_void_p), ("n_visible", C.c_void_p), ("offs", C.c_void_p), ("rect_order", C.c_void_p)]


class GsMatrix(C.Structure):
    _fields_ = [("data", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64),
                ("ld", C.c_int64), ("scales_ld", C.c_int64), ("type", C.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950)")
    lib = C.CDLL(LIB_PATH)
    P, I64, I32, U32 = C.c_void_p, C.c_int64, C.c_int32, C.c_uint32
    lib.gs_preprocess.argtypes = [P, P, P, P, P, C.c_size_t, P, P]
    lib.gs_bin_sort.argtypes = [P, I64, P, U32, P, P, U32, P, P, C.c_size_t, P]
    lib.gs_render_fwd.argtypes = [P, I64, P, P, U32, P, P, P, P, P, C.c_size_t, P, P]
    lib.gs_loss_l1_dssim.argtypes = [P, P, I32, I32, C.c_float, P, P, P, C.c_size_t, P]
    lib.gs_render_bwd.argtypes = [P, P, P, P, U32, P, P, P, P, P, P, P, C.c_size_t, P, P]
    lib.gs_render_bwd_adam.argtypes = [P, I64, I32, P, P, P, U32, P, P, P, P, P, P, P, P, C.c_double, C.c_double,
                                       C.c_double, I32, P, C.c_size_t, P, P]
    lib.gs_render_bwd_adam.restype = I32
    lib.gs_render_bwd_adam_project.argtypes = [P, I64, I32, P, P, P, U32, P, P, P, P, P, P, P, P, C.c_double,
                                               C.c_double, C.c_double, I32, P, C.c_size_t, P, P, P, P, C.c_size_t,
                                               P, P, P]
    lib.gs_render_bwd_adam_project.restype = I32
    lib.gs_loss_l1_dssim_noalloc.argtypes = [P, P, I32, I32, C.c_float, P, P, P]
    lib.gs_loss_l1_dssim_noalloc.restype = I32
    lib.gs_loss_charbonnier.argtypes = [P, P, I32, I32, C.c_float, P, P, P, P, P, C.c_size_t, P]
    lib.gs_loss_charbonnier.restype = I32
    lib.gs_render_bwd_weighted.argtypes = [P, P, P, P, U32, P, P, P, P, P, P, C.c_float, I32, P, C.c_size_t, P, P]
    lib.gs_render_bwd_weighted.restype = I32
    lib.gs_camera_grad.argtypes = [P, P, P, P, I32, P, P, C.c_size_t, P, P]
    lib.gs_relocate.argtypes = [P, P, P, I64, I32, P, C.c_double, C.c_double, I64, P, P, C.c_size_t, P]
    lib.gs_relocate.restype = I32
    lib.gs_camera_grad.restype = I32
    lib.gs_densify_accumulate.argtypes = [P, I64, P, P, P]
    lib.gs_densify_accumulate.restype = I32
    D = C.c_double
    lib.gs_densify.argtypes = [P, P, P, P, P, I64, I32, D, D, D, D, I32, D, P, P, P, P, I64, P, P, P, C.c_size_t, P]
    lib.gs_densify.restype = I32
    lib.gs_adam_step.argtypes = [P, P, P, P, I64, I32, P, C.c_double, C.c_double, C.c_double, I32, P]
    lib.gs_profile_enable.argtypes = [I32, C.c_char_p]
    lib.gs_profile_enable.restype = I32
    lib.gs_profile_query.argtypes = [I32, P, P, P]
    lib.gs_profile_query.restype = I32
    lib.gs_param_floats.argtypes = [I64, I32]
    lib.gs_param_floats.restype = C.c_size_t
    lib.gs_params_to_blocked.argtypes = [P, P, I64, I32, P]
    lib.gs_params_to_blocked.restype = I32
    lib.gs_params_from_blocked.argtypes = [P, P, I64, I32, P]
    lib.gs_params_from_blocked.restype = I32
    lib.gs_workspace_bytes.argtypes = [I32, I64, U32, I32, I32, P]
    lib.gs_workspace_bytes.restype = C.c_size_t
    lib.gs_mx8_pack.argtypes = [P, P, P]
    lib.gs_mx8_unpack.argtypes = [P, P, P]
    lib.gs_rmsnorm_fwd.argtypes = [P, P, P, C.c_float, P, P, P, P, P]
    lib.gs_rmsnorm_bwd.argtypes = [P, P, P, P, P, P, P, P, C.c_size_t, P]
    lib.gs_linear_fwd.argtypes = [P, P, P, I32, P, P, P, P]
    lib.gs_linear_bwd.argtypes = [P, P, I32, P, P, P, P, P, P, C.c_size_t, P]
    lib.gs_mx4_pack.argtypes = [P, P, P]
    lib.gs_mx4_unpack.argtypes = [P, P, P]
    lib.gs_lookup_fwd.argtypes = [P, P, I32, C.c_float, P, P]
    lib.gs_lookup_bwd.argtypes = [P, P, I32, C.c_float, P, P, C.c_size_t, P]
    lib.gs_clip_grads.argtypes = [P, P, I32, C.c_double, P, P, C.c_size_t, P]
    for name in ("gs_mx8_pack", "gs_mx8_unpack", "gs_rmsnorm_fwd", "gs_rmsnorm_bwd", "gs_linear_fwd",
                 "gs_linear_bwd", "gs_mx4_pack", "gs_mx4_unpack", "gs_lookup_fwd", "gs_lookup_bwd", "gs_clip_grads"):
        getattr(lib, name).restype = I32
    lib.gs_last_error.restype = C.c_char_p
    for name in ("gs_preprocess", "gs_bin_sort", "gs_render_fwd", "gs_loss_l1_dssim", "gs_render_bwd",
                 "gs_adam_step"):
        getattr(lib, name).restype = I32
    return lib


_lib = _load()


def lib():
    return _lib


def _check(status):
    if status != GS_OK:
        raise GsError(status, _lib.gs_last_error().decode())


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


# The current stream's handle without building a torch.cuda.Stream (3 us of a small call's
# 12); absent from a torch that does not offer it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return C.c_void_p(_raw_stream(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def make_camera(cam) -> GsCamera:
    c = GsCamera()
    c.R[:] = [float(x) for x in np.asarray(cam.R, np.float32).reshape(9)]
    c.t[:] = [float(x) for x in np.asarray(cam.t, np.float32)]
    c.campos[:] = [float(x) for x in np.asarray(cam.campos, np.float32)]
    c.fx, c.fy, c.cx, c.cy = cam.fx, cam.fy, cam.cx, cam.cy
    c.width, c.height = cam.width, cam.height
    c.znear = cam.znear
    c.bg[:] = [float(x) for x in cam.bg]
    return c


class Proj:
    """Device buffers of the projected state (gs_proj) for n Gaussians."""

    def __init__(self, n, device="cuda"):
        self.n = n
        self.splat = torch.empty((max(n, 1), 12), dtype=torch.float32, device=device)
        self.depth = torch.empty(max(n, 1), dtype=torch.float32, device=device)
        self.rect = torch.empty((max(n, 1), 2), dtype=torch.int32, device=device)
        self.tiles = torch.empty(max(n, 1), dtype=torch.int32, device=device)
        self.order = torch.empty(max(n, 1), dtype=torch.int32, device=device)
        self.n_visible = torch.empty(1, dtype=torch.int32, device=device)
        self.offs = torch.empty(n + 1, dtype=torch.int32, device=device)
        self.rect_order = torch.empty((max(n, 1), 2), dtype=torch.int32, device=device)
        self.struct = GsProj(self.splat.data_ptr(), self.depth.data_ptr(), self.rect.data_ptr(),
                             self.tiles.data_ptr(), self.order.data_ptr(), self.n_visible.data_ptr(),
                             self.offs.data_ptr(), self.rect_order.data_ptr())


def workspace(which, n=0, pairs=0, W=0, H=0, device="cuda", cfg=None):
    nbytes = int(_lib.gs_workspace_bytes(which, n, pairs, W, H, _cfg(cfg)))
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def gs_workspace_bytes(which, n=0, pairs=0, W=0, H=0, cfg=None):
    return int(_lib.gs_workspace_bytes(which, n, pairs, W, H, _cfg(cfg)))


def gs_param_floats(n, sh_degree):
    return int(_lib.gs_param_floats(n, sh_degree))


def _blocked(t, n, sh_degree):
    """Check that a tensor can hold a blocked parameter array for n Gaussians."""
    need = gs_param_floats(n, sh_degree)
    if t is None or t.dtype != torch.float32 or not t.is_contiguous() or t.numel() < need:
        raise ValueError(f"expected a contiguous float32 tensor of at least {need} floats (blocked layout)")
    return t


def empty_blocked(n, sh_degree, device="cuda", zero=False):
    """A device tensor of gs_param_floats(n, sh_degree) floats, shaped [groups][P][64]."""
    P = 11 + 3 * (sh_degree + 1) ** 2
    groups = max((n + 63) // 64, 1)
    f = torch.zeros if zero else torch.empty
    return f((groups, P, 64), dtype=torch.float32, device=device)


def to_blocked(planar, sh_degree, out=None, stream=None):
    """[P][n] device tensor -> blocked layout (gs_params_to_blocked)."""
    assert planar.dim() == 2 and planar.is_contiguous() and planar.dtype == torch.float32
    n = planar.shape[1]
    out = empty_blocked(n, sh_degree, planar.device) if out is None else _blocked(out, n, sh_degree)
    _check(_lib.gs_params_to_blocked(_ptr(planar), _ptr(out), n, sh_degree, _stream(stream)))
    return out


def from_blocked(blocked, n, sh_degree, out=None, stream=None):
    """Blocked layout -> [P][n] device tensor (gs_params_from_blocked)."""
    _blocked(blocked, n, sh_degree)
    P = 11 + 3 * (sh_degree + 1) ** 2
    out = torch.empty((P, n), dtype=torch.float32, device=blocked.device) if out is None else out
    assert out.shape == (P, n) and out.is_contiguous()
    _check(_lib.gs_params_from_blocked(_ptr(blocked), _ptr(out), n, sh_degree, _stream(stream)))
    return out


def gs_preprocess(params, sh_degree, cam: GsCamera, proj: Proj, ws, cfg=None, stream=None) -> int:
    """Projection + tile-count scan; returns the pair count (synchronises the stream once).
    params: blocked layout for proj.n Gaussians."""
    n = proj.n
    _blocked(params, n, sh_degree)
    scene = GsScene(n, sh_degree, params.data_ptr() if n else None)
    total = C.c_uint32(0)
    _check(_lib.gs_preprocess(C.byref(scene), C.byref(cam), C.byref(proj.struct), C.byref(total), _ptr(ws),
                              ws.numel(), _cfg(cfg), _stream(stream)))
    return int(total.value)


def gs_bin_sort(proj: Proj, cam: GsCamera, total_pairs, keys, vals, ranges, ws, stream=None):
    cap = keys.numel() if keys is not None else 0
    _check(_lib.gs_bin_sort(C.byref(proj.struct), proj.n, C.byref(cam), total_pairs, _ptr(keys), _ptr(vals), cap,
                            _ptr(ranges), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)))


def gs_render_fwd(proj: Proj, vals, ranges, total_pairs, cam: GsCamera, rgb, T_final, n_contrib, ws, cfg=None,
                  stream=None):
    _check(_lib.gs_render_fwd(C.byref(proj.struct), proj.n, _ptr(vals), _ptr(ranges), total_pairs, C.byref(cam),
                              _ptr(rgb), _ptr(T_final), _ptr(n_contrib), _ptr(ws), ws.numel(), _cfg(cfg),
                              _stream(stream)))


def gs_loss_l1_dssim(img, target, lambda_dssim, loss_out, dL_dimg, ws, stream=None):
    _, H, W = img.shape
    _check(_lib.gs_loss_l1_dssim(_ptr(img), _ptr(target), H, W, float(lambda_dssim), _ptr(loss_out),
                                 _ptr(dL_dimg), _ptr(ws), ws.numel(), _stream(stream)))


def gs_loss_l1_dssim_noalloc(img, target, lambda_dssim, loss_out, dL_dimg, stream=None):
    """gs_loss_l1_dssim without a workspace: the library's static scratch (no allocation)."""
    _, H, W = img.shape
    _check(_lib.gs_loss_l1_dssim_noalloc(_ptr(img), _ptr(target), H, W, float(lambda_dssim), _ptr(loss_out),
                                         _ptr(dL_dimg), _stream(stream)))


def gs_render_bwd(params, sh_degree, proj: Proj, vals, ranges, total_pairs, cam: GsCamera, T_final, n_contrib, dL_dimg,
                  gscreen, gparams, ws, cfg=None, stream=None):
    n = proj.n
    _blocked(params, n, sh_degree)
    _blocked(gparams, n, sh_degree)
    scene = GsScene(n, sh_degree, params.data_ptr() if n else None)
    _check(_lib.gs_render_bwd(C.byref(scene), C.byref(proj.struct), _ptr(vals), _ptr(ranges), total_pairs,
                              C.byref(cam),
                              _ptr(T_final), _ptr(n_contrib), _ptr(dL_dimg), _ptr(gscreen), _ptr(gparams),
                              _ptr(ws), ws.numel(), _cfg(cfg), _stream(stream)))


def gs_render_bwd_weighted(params, sh_degree, proj: Proj, vals, ranges, total_pairs, cam: GsCamera, T_final,
                           n_contrib, dL_dimg, gscreen, gparams, ws, weight, accumulate, cfg=None, stream=None):
    n = proj.n
    _blocked(params, n, sh_degree)
    _blocked(gparams, n, sh_degree)
    scene = GsScene(n, sh_degree, params.data_ptr() if n else None)
    _check(_lib.gs_render_bwd_weighted(C.byref(scene), C.byref(proj.struct), _ptr(vals), _ptr(ranges), total_pairs,
                                       C.byref(cam), _ptr(T_final), _ptr(n_contrib), _ptr(dL_dimg), _ptr(gscreen),
                                       _ptr(gparams), float(weight), int(bool(accumulate)), _ptr(ws), ws.numel(),
                                       _cfg(cfg), _stream(stream)))


def gs_relocate(params, m, v, n, sh_degree, rand, ws, dead_opacity=0.02, donor_opacity=0.4, max_moves=-1,
                stream=None):
    """Moves the dead Gaussians to the largest donors in place; returns the number of moves."""
    for t in (params, m, v):
        _blocked(t, n, sh_degree)
    moves = C.c_int64(0)
    _check(_lib.gs_relocate(_ptr(params), _ptr(m), _ptr(v), n, sh_degree, _ptr(rand), float(dead_opacity),
                            float(donor_opacity), int(max_moves), C.byref(moves), _ptr(ws), ws.numel(),
                            _stream(stream)))
    return int(moves.value)


def gs_camera_grad(params, sh_degree, proj: Proj, cam: GsCamera, gscreen, grad_out, ws, position_only=False,
                   cfg=None, stream=None):
    """grad_out: device float64[6] = (rotation, translation) gradient of the camera pose
    (with position_only, the trainer's position-path terms alone)."""
    n = proj.n
    _blocked(params, n, sh_degree)
    if grad_out.dtype != torch.float64 or grad_out.numel() < 6:
        raise ValueError("grad_out must hold 6 float64 values")
    scene = GsScene(n, sh_degree, params.data_ptr() if n else None)
    _check(_lib.gs_camera_grad(C.byref(scene), C.byref(proj.struct), C.byref(cam), _ptr(gscreen),
                               int(bool(position_only)), _ptr(grad_out), _ptr(ws), ws.numel(), _cfg(cfg),
                               _stream(stream)))


def gs_adam_step(params, grads, m, v, n, sh_degree, lr, beta1, beta2, eps, step, stream=None):
    for t in (params, grads, m, v):
        _blocked(t, n, sh_degree)
    lr_arr = (C.c_float * 5)(*[float(x) for x in lr])
    _check(_lib.gs_adam_step(_ptr(params), _ptr(grads), _ptr(m), _ptr(v), n, sh_degree, lr_arr, float(beta1),
                             float(beta2), float(eps), int(step), _stream(stream)))


def gs_render_bwd_adam(params, sh_degree, proj: Proj, vals, ranges, total_pairs, cam: GsCamera, T_final,
                       n_contrib, dL_dimg, gscreen, m, v, lr, beta1, beta2, eps, step, ws, cfg=None, stream=None):
    for t in (params, m, v):
        _blocked(t, proj.n, sh_degree)
    lr_arr = (C.c_float * 5)(*[float(x) for x in lr])
    _check(_lib.gs_render_bwd_adam(_ptr(params), proj.n, sh_degree, C.byref(proj.struct), _ptr(vals), _ptr(ranges),
                                   total_pairs, C.byref(cam), _ptr(T_final), _ptr(n_contrib), _ptr(dL_dimg),
                                   _ptr(gscreen), _ptr(m), _ptr(v), lr_arr, float(beta1), float(beta2),
                                   float(eps), int(step), _ptr(ws), ws.numel(), _cfg(cfg), _stream(stream)))


def gs_render_bwd_adam_project(params, sh_degree, proj: Proj, vals, ranges, total_pairs, cam: GsCamera, T_final,
                               n_contrib, dL_dimg, gscreen, m, v, lr, beta1, beta2, eps, step, ws,
                               next_cam: GsCamera, next_proj: Proj, pre_ws, densify_stats=None, cfg=None,
                               stream=None) -> int:
    """gs_render_bwd_adam, then the projection of the updated scene for next_cam into
    next_proj (may be proj); returns the next pair count (synchronises once).  With
    densify_stats ([n][2]), this step's observations are added to it."""
    for t in (params, m, v):
        _blocked(t, proj.n, sh_degree)
    assert next_proj.n == proj.n
    lr_arr = (C.c_float * 5)(*[float(x) for x in lr])
    total = C.c_uint32(0)
    _check(_lib.gs_render_bwd_adam_project(
        _ptr(params), proj.n, sh_degree, C.byref(proj.struct), _ptr(vals), _ptr(ranges), total_pairs, C.byref(cam),
        _ptr(T_final), _ptr(n_contrib), _ptr(dL_dimg), _ptr(gscreen), _ptr(m), _ptr(v), lr_arr, float(beta1),
        float(beta2), float(eps), int(step), _ptr(ws), ws.numel(), C.byref(next_cam), C.byref(next_proj.struct),
        C.byref(total), _ptr(pre_ws), pre_ws.numel(), _ptr(densify_stats), _cfg(cfg), _stream(stream)))
    return int(total.value)


def gs_densify_accumulate(proj: Proj, gscreen, stats, stream=None):
    """Adds one step's screen-position gradient lengths and observation counts to stats [n][2]."""
    _check(_lib.gs_densify_accumulate(C.byref(proj.struct), proj.n, _ptr(gscreen), _ptr(stats), _stream(stream)))


def gs_densify(params, m, v, stats, rand, n, sh_degree, grad_threshold, prune_opacity, prune_scale, split_scale,
               ws, reset_opacity=False, opacity_cap=0.01, params_out=None, m_out=None, v_out=None, stats_out=None,
               capacity=0, stream=None):
    """One densification; returns (new count, (kept, cloned, split)).  Without params_out
    only the counts are computed."""
    n_out = C.c_int64(0)
    counts = (C.c_int64 * 3)()
    _check(_lib.gs_densify(_ptr(params), _ptr(m), _ptr(v), _ptr(stats), _ptr(rand), n, sh_degree,
                           float(grad_threshold), float(prune_opacity), float(prune_scale), float(split_scale),
                           1 if reset_opacity else 0, float(opacity_cap), _ptr(params_out), _ptr(m_out),
                           _ptr(v_out), _ptr(stats_out), int(capacity), C.byref(n_out), counts, _ptr(ws),
                           ws.numel() if ws is not None else 0, _stream(stream)))
    return int(n_out.value), tuple(int(c) for c in counts)


def gs_loss_charbonnier(img, target, exposure, loss_out, dL_dimg, ws, delta=0.03, dL_dexposure=None, stream=None):
    """Charbonnier loss with exposure (log gain, bias): mean of sqrt(err^2 + delta^2) - delta."""
    _, H, W = img.shape
    _check(_lib.gs_loss_charbonnier(_ptr(img), _ptr(target), H, W, float(delta), _ptr(exposure), _ptr(loss_out),
                                    _ptr(dL_dimg), _ptr(dL_dexposure), _ptr(ws), ws.numel(), _stream(stream)))


# ---- the operators of a network over Gaussians

class Mx8:
    """An MX8 matrix: q [rows][cols] (torch.float8_e4m3fn) and scales [rows][ceil(cols / 32)]
    (torch.float8_e8m0fnu), both with adjacent columns; the value of a column is q times its
    32-column block's scale."""

    __slots__ = ("q", "scales")

    def __init__(self, q, scales):
        self.q, self.scales = q, scales

    @property
    def shape(self):
        return self.q.shape


def mx8_empty(rows, cols, device="cuda"):
    """An uninitialised MX8 matrix whose rows start at multiples of 16 bytes."""
    pitch = (cols + 15) // 16 * 16
    q = torch.empty((rows, pitch), dtype=torch.float8_e4m3fn, device=device)
    scales = torch.empty((rows, (cols + 31) // 32), dtype=torch.float8_e8m0fnu, device=device)
    return Mx8(q if pitch == cols else q[:, :cols], scales)


class Mx4:
    """An MX4 matrix of `cols` columns: q [rows][16 ceil(cols / 32)] (torch.uint8, two columns to a
    byte, the even one in the low half) and scales [rows][ceil(cols / 32)] (torch.float8_e8m0fnu); the
    rows of q start at multiples of 16 bytes."""

    __slots__ = ("q", "scales", "cols")

    def __init__(self, q, scales, cols):
        self.q, self.scales, self.cols = q, scales, cols

    @property
    def shape(self):
        return torch.Size((self.q.shape[0], self.cols))


def mx4_empty(rows, cols, device="cuda"):
    """An uninitialised MX4 matrix."""
    blocks = (cols + 31) // 32
    return Mx4(torch.empty((rows, 16 * blocks), dtype=torch.uint8, device=device),
               torch.empty((rows, blocks), dtype=torch.float8_e8m0fnu, device=device), cols)


_KINDS = {torch.float32: GS_MAT_F32, torch.bfloat16: GS_MAT_BF16}


def _matrix(t, name):
    """gs_matrix of a two-dimensional tensor (float32, bfloat16), Mx8 or Mx4 with adjacent columns."""
    return None if t is None else C.byref(_struct(t, name))


def _struct(t, name):
    if isinstance(t, Mx4):
        if t.q.dtype != torch.uint8 or t.scales.dtype != torch.float8_e8m0fnu:
            raise ValueError(f"{name}: an Mx4 is a uint8 matrix with float8_e8m0fnu scales")
        rows, blocks = t.q.shape[0], (t.cols + 31) // 32
        if t.cols < 1 or t.q.shape != (rows, 16 * blocks) or t.scales.shape != (rows, blocks):
            raise ValueError(f"{name}: an Mx4 of {t.cols} columns has rows of whole blocks: 16 bytes and a scale for 32 columns")
        _, scales, scales_ld = _rows(t.scales, f"{name} (scales)")
        _, data, pitch = _rows(t.q, name)
        return GsMatrix(data, scales, rows, t.cols, 2 * pitch, scales_ld, GS_MAT_MX4)
    if isinstance(t, Mx8):
        q, kind = t.q, GS_MAT_MX8
        if q.dtype != torch.float8_e4m3fn or t.scales.dtype != torch.float8_e8m0fnu:
            raise ValueError(f"{name}: an Mx8 is a float8_e4m3fn matrix with float8_e8m0fnu scales")
        blocks, scales, scales_ld = _rows(t.scales, f"{name} (scales)")
    else:
        q, kind, blocks, scales, scales_ld = t, _KINDS.get(t.dtype), None, None, 0
        if kind is None:
            raise ValueError(f"{name}: expected float32, bfloat16, an Mx8 or an Mx4, got {t.dtype}")
    (rows, cols), data, ld = _rows(q, name)
    if blocks is not None and blocks != (rows, (cols + 31) // 32):
        raise ValueError(f"{name}: scales must be [rows][ceil(cols / 32)]")
    return GsMatrix(data, scales, rows, cols, ld, scales_ld, kind)


def _rows(t, name):
    """(shape, address, elements between rows) of a device matrix with adjacent columns; a
    single row's (or an empty matrix's) stride says nothing."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name}: expected a matrix with adjacent columns")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected device memory")
    return shape, t.data_ptr(), stride[0] if shape[0] > 1 else shape[1]


def _floats(t, n, name):
    """A contiguous float32 vector of n values (None passes)."""
    if t is None:
        return None
    if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != n or not t.is_cuda:
        raise ValueError(f"{name}: expected {n} contiguous float32 values in device memory")
    return t.data_ptr()


def _activation(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act: expected one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def gs_mx8_pack(x, q, stream=None):
    """x (float32 or bfloat16) to the Mx8 q of the same size."""
    _check(_lib.gs_mx8_pack(_matrix(x, "x"), _matrix(q, "q"), _stream(stream)))


def gs_mx8_unpack(q, x, stream=None):
    """The Mx8 q's values to x (float32 or bfloat16)."""
    _check(_lib.gs_mx8_unpack(_matrix(q, "q"), _matrix(x, "x"), _stream(stream)))


def gs_mx4_pack(x, q, stream=None):
    """x (float32 or bfloat16) to the Mx4 q of the same size."""
    _check(_lib.gs_mx4_pack(_matrix(x, "x"), _matrix(q, "q"), _stream(stream)))


def gs_mx4_unpack(q, x, stream=None):
    """The Mx4 q's values to x (float32 or bfloat16)."""
    _check(_lib.gs_mx4_unpack(_matrix(q, "q"), _matrix(x, "x"), _stream(stream)))


def _index(t, rows):
    """(address, bytes an element) of a contiguous int32 or int64 vector."""
    if t.dtype not in (torch.int32, torch.int64) or t.dim() != 1 or not t.is_contiguous() or t.numel() != rows or not t.is_cuda:
        raise ValueError(f"index: expected {rows} contiguous int32 or int64 values in device memory")
    return t.data_ptr(), t.element_size()


def gs_lookup_fwd(table, index, y, scale=1.0, stream=None):
    """y[i] = scale table[index[i]], zeros where index[i] is outside the table (int32 or int64)."""
    _check(_lib.gs_lookup_fwd(_matrix(table, "table"), *_index(index, y.shape[0]), float(scale), _matrix(y, "y"),
                              _stream(stream)))


def gs_lookup_bwd(dy, index, dtable, ws, scale=1.0, stream=None):
    """dtable[t] = scale times the sum of dy[i] over the rows i with index[i] = t."""
    _check(_lib.gs_lookup_bwd(_matrix(dy, "dy"), *_index(index, dy.shape[0]), float(scale), _matrix(dtable, "dtable"),
                              _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)))


class Matrices:
    """A list of float32 or bfloat16 tensors as the array of gs_matrix that gs_clip_grads takes, for
    buffers that stay where they are from step to step (it keeps them alive).  Matrices need adjacent
    columns, tensors of other dimensions have to be contiguous."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        parts = []
        for i, t in enumerate(self.tensors):
            parts += [_struct(v, f"[{i}]") for v in _as_matrices(t, f"[{i}]")]
        self.count = len(parts)
        self.array = (GsMatrix * max(self.count, 1))(*parts)


def _as_matrices(t, name):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor")
    if t.dim() == 2 and t.shape[1] <= 1 << 20:
        return [t] if t.shape[1] else []
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a matrix with adjacent columns, or a contiguous tensor")
    t, n = t.view(-1), t.numel()
    whole = n >> 20 << 20
    return ([t[:whole].view(-1, 1 << 20)] if whole else []) + ([t[whole:].view(1, -1)] if n > whole else [])


def blocked_matrices(t, n, sh_degree):
    """The parameters of n Gaussians in a blocked array as matrices (without the padding)."""
    _blocked(t, n, sh_degree)
    P, full = 11 + 3 * (sh_degree + 1) ** 2, n // 64
    t = t.view(-1)
    out = [t[:full * P * 64].view(-1, 64)] if full else []
    if n % 64:
        out.append(t[full * P * 64:(full + 1) * P * 64].view(P, 64)[:, :n % 64])
    return out


def gs_clip_grads(grads, max_norm, norm, ws, out=None, stream=None):
    """norm (float32 [1]) = the norm of all grads together, and out = grads min(1, max_norm / norm).
    grads, out: lists of tensors, or Matrices; out None: in place; max_norm inf: only the norm (with
    out None)."""
    grads = grads if isinstance(grads, Matrices) else Matrices(grads)
    if out is None:
        to = None if max_norm == float("inf") else grads.array
    else:
        out = out if isinstance(out, Matrices) else Matrices(out)
        if out.count != grads.count:
            raise ValueError(f"out: expected {grads.count} matrices, got {out.count}")
        to = out.array
    _check(_lib.gs_clip_grads(grads.array, to, grads.count, float(max_norm), _floats(norm, 1, "norm"), _ptr(ws),
                              ws.numel() if ws is not None else 0, _stream(stream)))


def gs_rmsnorm_fwd(x, weight, eps, y, rstd=None, residual=None, h=None, ckpt=None, stream=None):
    """h = x + residual, y = h (mean(h^2) + eps)^-1/2 weight by rows; ckpt: an Mx8 for h."""
    rows, cols = x.shape
    _check(_lib.gs_rmsnorm_fwd(_matrix(x, "x"), _matrix(residual, "residual"), _floats(weight, cols, "weight"),
                               float(eps), _matrix(h, "h"), _matrix(ckpt, "ckpt"), _matrix(y, "y"),
                               _floats(rstd, rows, "rstd"), _stream(stream)))


def gs_rmsnorm_bwd(dy, h, weight, rstd, dh, dweight, ws, dres=None, stream=None):
    """The gradients of h (plus dres) and of the weight; h: float32, bfloat16 or the Mx8 checkpoint."""
    rows, cols = dy.shape
    _check(_lib.gs_rmsnorm_bwd(_matrix(dy, "dy"), _matrix(h, "h"), _floats(weight, cols, "weight"),
                               _floats(rstd, rows, "rstd"), _matrix(dres, "dres"), _matrix(dh, "dh"),
                               _floats(dweight, cols, "dweight"), _ptr(ws), ws.numel() if ws is not None else 0,
                               _stream(stream)))


def gs_linear_fwd(x, w, y, bias=None, act="none", residual=None, z=None, stream=None):
    """y = act(x w^T + bias) + residual; z (float32, bfloat16 or Mx8) receives x w^T + bias.  With w an
    Mx4, x may be one too, y an Mx8, and z is None."""
    _check(_lib.gs_linear_fwd(_matrix(x, "x"), _matrix(w, "w"), _floats(bias, w.shape[0], "bias"), _activation(act),
                              _matrix(residual, "residual"), _matrix(z, "z"), _matrix(y, "y"), _stream(stream)))


def gs_linear_bwd(dy, x, w, dx, dw, dbias, ws, act="none", z=None, stream=None):
    """The gradients of x, w and the bias (each output may be None) from x and z as kept."""
    _check(_lib.gs_linear_bwd(_matrix(dy, "dy"), _matrix(z, "z"), _activation(act), _matrix(x, "x"), _matrix(w, "w"),
                              _matrix(dx, "dx"), _matrix(dw, "dw"), _floats(dbias, w.shape[0], "dbias"), _ptr(ws),
                              ws.numel() if ws is not None else 0, _stream(stream)))


def gs_profile_enable(on, only=None):
    """Start (on=True) or stop per-kernel event timing; `only` restricts it to one kernel name."""
    _check(_lib.gs_profile_enable(1 if on else 0, only.encode() if only else None))


def gs_profile_query(max_names=64):
    """{kernel name: (launches, summed milliseconds)} for the launches recorded since enabling."""
    names = C.create_string_buffer(64 * max_names)
    launches = (C.c_int64 * max_names)()
    total_ms = (C.c_double * max_names)()
    k = _lib.gs_profile_query(max_names, C.cast(names, C.c_void_p), C.cast(launches, C.c_void_p),
                              C.cast(total_ms, C.c_void_p))
    _check(min(k, 0))
    return {names.raw[64 * i:64 * (i + 1)].split(b"\0", 1)[0].decode(): (int(launches[i]), float(total_ms[i]))
            for i in range(k)}


def gs_last_error():
    return _lib.gs_last_error().decode()
