"""Thin ctypes binding of libgsraster.so.

The functions below carry the names of the C entry points declared in
``include/gsraster.h`` and do argument marshalling only: every stage runs in
the library's HIP kernels.  PyTorch supplies device memory and the stream
(``torch.cuda.current_stream()``); no compute happens in torch.  There is no
fallback: if the library is missing or the device is not a GPU, calls raise.

Array layout is the library's: per-Gaussian structure-of-arrays planes
``[P, ld]`` (float32/int32/uint32, contiguous), images ``[H, W, 3]`` and
``[H, W]``.  :class:`Frame` strings the five calls together with caller-owned
buffers (growing the instance capacity when ``gs_bin_and_sort`` asks for it).
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgsraster.so")

GS_OK, GS_ERR_INVALID_ARGUMENT, GS_ERR_CAPACITY, GS_ERR_HIP = 0, 1, 2, 3
EXPORTED = ("gs_default_settings", "gs_status_string", "gs_last_error", "gs_num_tiles",
            "gs_project_fwd", "gs_bin_and_sort_workspace_size", "gs_bin_and_sort",
            "gs_rasterize_fwd", "gs_rasterize_bwd", "gs_project_bwd", "gs_image_loss_grad",
            "gs_densify_prune_workspace_size", "gs_densify_prune", "gs_bin_and_sort_packed",
            "gs_rasterize_bwd_packed", "gs_project_bwd_packed", "gs_l1_dssim_workspace_size",
            "gs_l1_dssim_loss_grad", "gs_default_adam_config", "gs_adam_step",
            "gs_adam_step_packed", "gs_project_fwd_batched",
            "gs_bin_and_sort_batched_workspace_size", "gs_bin_and_sort_batched",
            "gs_rasterize_fwd_batched", "gs_rasterize_bwd_batched", "gs_project_bwd_batched",
            "gs_bin_and_sort_device", "gs_rasterize_fwd_loss", "gs_tile_order",
            "gs_rasterize_fwd_loss_batched", "gs_bin_and_sort_noalloc",
            "gs_rasterize_workspace_size", "gs_qk_norm_rope_fwd",
            "gs_qk_norm_rope_bwd_workspace_size", "gs_qk_norm_rope_bwd",
            "gs_attention_fwd_workspace_size", "gs_attention_fwd",
            "gs_attention_bwd_workspace_size", "gs_attention_bwd", "gs_gated_scan_saved_size",
            "gs_gated_scan_fwd_workspace_size", "gs_gated_scan_fwd",
            "gs_gated_scan_bwd_workspace_size", "gs_gated_scan_bwd")
GS_F32, GS_BF16, GS_F16 = 0, 1, 2


class GsError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s: %s" % (status, msg))
        self.status = status


class gs_camera(C.Structure):
    _fields_ = [("R", C.c_float * 9), ("t", C.c_float * 3), ("fx", C.c_float),
                ("fy", C.c_float), ("cx", C.c_float), ("cy", C.c_float),
                ("width", C.c_int32), ("height", C.c_int32),
                ("near_plane", C.c_float), ("far_plane", C.c_float)]


class gs_settings(C.Structure):
    _fields_ = [(k, C.c_float) for k in
                ("eps2d", "alpha_min", "alpha_max", "T_min", "fov_clamp", "sh_offset")]


_lib = None


class gs_adam_config(C.Structure):
    _fields_ = [(n, C.c_float) for n in ("lr_means", "lr_scales", "lr_quats", "lr_opacities",
                                         "lr_sh", "beta1", "beta2", "eps")]


class gs_heads(C.Structure):
    """[rows][heads][dim] view (element strides); keeps its tensor alive."""
    _fields_ = [("data", C.c_void_p), ("row", C.c_int64), ("head", C.c_int64)]


class gs_rows(C.Structure):
    """[rows][channels] view (element stride); keeps its tensor alive."""
    _fields_ = [("data", C.c_void_p), ("row", C.c_int64)]


class gs_documents(C.Structure):
    _fields_ = [("count", C.c_int32), ("max_q_len", C.c_int32), ("max_k_len", C.c_int32)] + \
        [(n, C.c_void_p) for n in ("q_start", "q_len", "k_start", "k_len", "prefix")]


class gs_qk_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("dtype", "heads_q", "heads_k", "head_dim",
                                         "rotary_dim", "interleaved", "norm")] + \
        [("eps", C.c_float), ("amplitude", C.c_float)]


class gs_attention_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("dtype", "heads_q", "heads_k", "head_dim", "causal")] + \
        [("scale", C.c_float), ("softcap", C.c_float), ("slopes", C.c_void_p)]


class gs_scan_config(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("coupled", C.c_int32), ("channels", C.c_int64)]


def load():
    """Load libgsraster.so (built in-tree by ``build.py``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libgsraster.so is not built: run differentiable_rasterization_amd/build.py")
    from . import build
    try:
        built = open(build.HASH_FILE).read().strip()
    except OSError:
        built = None
    if built != build.source_hash():
        raise RuntimeError("libgsraster.so was not built from the current csrc/ and include/ "
                           "sources: run differentiable_rasterization_amd/build.py")
    lib = C.CDLL(LIB_PATH)
    P, i64, i32, u64 = C.c_void_p, C.c_int64, C.c_int32, C.c_uint64
    lib.gs_default_settings.restype = gs_settings
    lib.gs_default_settings.argtypes = []
    lib.gs_status_string.restype = C.c_char_p
    lib.gs_status_string.argtypes = [C.c_int]
    lib.gs_last_error.restype = C.c_char_p
    lib.gs_last_error.argtypes = []
    lib.gs_num_tiles.restype = i32
    lib.gs_num_tiles.argtypes = [i32, i32]
    lib.gs_project_fwd.restype = C.c_int
    lib.gs_project_fwd.argtypes = [i64, i64, i32] + [P] * 4 + [P, P] + [P] * 7 + [P]
    lib.gs_rasterize_workspace_size.restype = C.c_size_t
    lib.gs_rasterize_workspace_size.argtypes = [i64]
    lib.gs_bin_and_sort_workspace_size.restype = C.c_size_t
    lib.gs_bin_and_sort_workspace_size.argtypes = [i64, u64, i32, i32]
    lib.gs_bin_and_sort.restype = C.c_int
    lib.gs_bin_and_sort.argtypes = [i64, i64, P, P, P, P, i32, i32, P, u64, P, P, P, P, P,
                                    C.c_size_t, P]
    lib.gs_rasterize_fwd.restype = C.c_int
    SZ = C.c_size_t
    lib.gs_rasterize_fwd.argtypes = [i64, i64, i32, i32] + [P] * 3 + [P] * 7 + [P, P] + \
        [P] * 5 + [P, SZ, P, P]
    lib.gs_rasterize_bwd.restype = C.c_int
    lib.gs_rasterize_bwd.argtypes = [i64, i64, i32, i32] + [P] * 3 + [P] * 6 + [P, P, u64] + \
        [P, P] + [P] * 3 + [P, SZ, i32, P, u64] + [P] * 5 + [i32, P, P]
    lib.gs_project_bwd.restype = C.c_int
    lib.gs_project_bwd.argtypes = [i64, i64, i32] + [P] * 4 + [P, P, P] + [P] * 3 + [P] * 4 + \
        [i32, P]
    lib.gs_bin_and_sort_packed.restype = C.c_int
    lib.gs_bin_and_sort_packed.argtypes = [i64, i64, P, P, P, P, i32, i32, P, u64, P, P, P, P,
                                           P, P, C.c_size_t, P]
    lib.gs_rasterize_bwd_packed.restype = C.c_int
    lib.gs_rasterize_bwd_packed.argtypes = [i64, i64, i32, i32] + [P] * 3 + [P] * 6 + \
        [P, P, u64, P, i64, i64] + [P, P] + [P] * 3 + [P, SZ, i32, P, u64] + [P] * 5 + \
        [i32, P, P]
    lib.gs_project_bwd_packed.restype = C.c_int
    lib.gs_project_bwd_packed.argtypes = [i64, P, i64, i64, i64, i32] + [P] * 4 + [P, P, P] + \
        [P] * 3 + [P] * 4 + [i32, P]
    lib.gs_l1_dssim_workspace_size.restype = C.c_size_t
    lib.gs_l1_dssim_workspace_size.argtypes = [i32, i32]
    lib.gs_l1_dssim_loss_grad.restype = C.c_int
    lib.gs_l1_dssim_loss_grad.argtypes = [i32, i32, P, P, C.c_float, P, P, P, C.c_size_t, P]
    lib.gs_default_adam_config.restype = gs_adam_config
    lib.gs_default_adam_config.argtypes = []
    lib.gs_adam_step.restype = C.c_int
    lib.gs_adam_step.argtypes = [i64, i64, i32, i64, P] + [P] * 7 + [P] * 5 + [P, P, P]
    lib.gs_adam_step_packed.restype = C.c_int
    lib.gs_adam_step_packed.argtypes = [i64, P, i64, i64, i64, i32, i64, P] + [P] * 7 + \
        [P] * 5 + [P, P, P]
    lib.gs_project_fwd_batched.restype = C.c_int
    lib.gs_project_fwd_batched.argtypes = [i32, P, i64, i64, i32] + [P] * 4 + [P] + [P] * 7 + [P]
    lib.gs_bin_and_sort_batched_workspace_size.restype = C.c_size_t
    lib.gs_bin_and_sort_batched_workspace_size.argtypes = [i32, i64, u64, i32, i32]
    lib.gs_bin_and_sort_batched.restype = C.c_int
    lib.gs_bin_and_sort_batched.argtypes = [i32, i64, P, P, P, P, i32, i32, P, u64, P, P, P, P,
                                            P, C.c_size_t, P]
    lib.gs_rasterize_fwd_batched.restype = C.c_int
    lib.gs_rasterize_fwd_batched.argtypes = [i32, i64, i32, i32] + [P] * 3 + [P] * 7 + [P, P] + \
        [P] * 5 + [P, SZ, P, P]
    lib.gs_rasterize_bwd_batched.restype = C.c_int
    lib.gs_rasterize_bwd_batched.argtypes = [i32, i64, i32, i32] + [P] * 3 + [P] * 6 + \
        [P, P, u64] + [P, P] + [P] * 3 + [P, SZ, i32, P, u64] + [P] * 5 + [i32, P, P]
    lib.gs_project_bwd_batched.restype = C.c_int
    lib.gs_project_bwd_batched.argtypes = [i32, P, i64, i64, i32] + [P] * 4 + [P, P] + \
        [P] * 3 + [P] + [P] * 5 + [i32, P]
    lib.gs_bin_and_sort_noalloc.restype = C.c_int
    lib.gs_bin_and_sort_noalloc.argtypes = [i64, i64, P, P, P, P, i32, i32, P, u64, P, P, P, P,
                                            P]
    lib.gs_bin_and_sort_device.restype = C.c_int
    lib.gs_bin_and_sort_device.argtypes = [i64, i64, P, P, P, P, i32, i32, P, u64, P, P, P, P, P,
                                           C.c_size_t, P]
    lib.gs_rasterize_fwd_loss.restype = C.c_int
    lib.gs_rasterize_fwd_loss.argtypes = [i64, i64, i32, i32] + [P] * 3 + [P] * 7 + [P, P] + \
        [i32, P] + [P] * 5 + [P, P] + [P, SZ, P, P]
    lib.gs_tile_order.restype = C.c_int
    lib.gs_tile_order.argtypes = [i32, i32, i32, P, P, P]
    lib.gs_rasterize_fwd_loss_batched.restype = C.c_int
    lib.gs_rasterize_fwd_loss_batched.argtypes = [i32, i64, i32, i32] + [P] * 3 + [P] * 7 + \
        [P, P] + [i32, P] + [P] * 5 + [P, P] + [P, SZ, P, P]
    lib.gs_image_loss_grad.restype = C.c_int
    lib.gs_image_loss_grad.argtypes = [i32, i64, P, P, P, P, P]
    lib.gs_densify_prune_workspace_size.restype = C.c_size_t
    lib.gs_densify_prune_workspace_size.argtypes = [i64, C.c_float]
    lib.gs_densify_prune.restype = C.c_int
    lib.gs_densify_prune.argtypes = [i64, i64, i32] + [P] * 6 + [C.c_float, C.c_float, i64] + \
        [P] * 5 + [P, P, C.c_size_t, P]
    lib.gs_qk_norm_rope_fwd.restype = C.c_int
    lib.gs_qk_norm_rope_fwd.argtypes = [P, i64] + [P] * 4 + [P] * 4 + [P]
    lib.gs_qk_norm_rope_bwd_workspace_size.restype = SZ
    lib.gs_qk_norm_rope_bwd_workspace_size.argtypes = [P, i64]
    lib.gs_qk_norm_rope_bwd.restype = C.c_int
    lib.gs_qk_norm_rope_bwd.argtypes = [P, i64] + [P] * 4 + [P] * 6 + [P, P] + [P, SZ, P]
    for name in ("fwd", "bwd"):
        fn = getattr(lib, "gs_attention_%s_workspace_size" % name)
        fn.restype, fn.argtypes = SZ, [P, P, i64, i64]
        fn = getattr(lib, "gs_gated_scan_%s_workspace_size" % name)
        fn.restype, fn.argtypes = SZ, [P, P, i64]
    lib.gs_attention_fwd.restype = C.c_int
    lib.gs_attention_fwd.argtypes = [P, P, i64, i64] + [P] * 5 + [P, SZ, P]
    lib.gs_attention_bwd.restype = C.c_int
    lib.gs_attention_bwd.argtypes = [P, P, i64, i64] + [P] * 9 + [P, SZ, P]
    lib.gs_gated_scan_saved_size.restype = SZ
    lib.gs_gated_scan_saved_size.argtypes = [P, P, i64]
    lib.gs_gated_scan_fwd.restype = C.c_int
    lib.gs_gated_scan_fwd.argtypes = [P, P, i64] + [P] * 6 + [P, SZ, P]
    lib.gs_gated_scan_bwd.restype = C.c_int
    lib.gs_gated_scan_bwd.argtypes = [P, P, i64] + [P] * 8 + [P, SZ, P]
    _name_types()
    _lib = lib
    return lib


def _check(status):
    if status != GS_OK:
        lib = load()
        raise GsError(lib.gs_status_string(status).decode(), lib.gs_last_error().decode())


def _p(t):
    """Device (or host) pointer of a tensor/array, None for None."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data_as(C.c_void_p)
    return C.c_void_p(t.data_ptr())


_raw_stream = None


def _stream(stream):
    """hipStream_t of a torch stream, or of the current one (by its raw handle
    where torch offers it: making a Stream object costs 2.5 us a call, as much
    as a kernel launch)."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        if raw is not None and device is not None:
            torch.cuda.current_stream()  # initialises the device
            _raw_stream = lambda: raw(device())
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream
    return _raw_stream()


def make_camera(cam) -> gs_camera:
    """gs_camera from any object with R, t, fx, fy, cx, cy, width, height, near, far."""
    c = gs_camera()
    R = np.asarray(cam.R, np.float32).reshape(9)
    t = np.asarray(cam.t, np.float32).reshape(3)
    for i in range(9):
        c.R[i] = float(R[i])
    for i in range(3):
        c.t[i] = float(t[i])
    c.fx, c.fy, c.cx, c.cy = float(cam.fx), float(cam.fy), float(cam.cx), float(cam.cy)
    c.width, c.height = int(cam.width), int(cam.height)
    c.near_plane = float(getattr(cam, "near", 0.01))
    c.far_plane = float(getattr(cam, "far", 1e10))
    return c


def default_settings(**overrides) -> gs_settings:
    s = load().gs_default_settings()
    for k, v in overrides.items():
        setattr(s, k, float(v))
    return s


def num_tiles(width, height) -> int:
    return int(load().gs_num_tiles(int(width), int(height)))


# ---------------------------------------------------------------------------
# The entry points
# ---------------------------------------------------------------------------
def gs_project_fwd(N, ld, sh_degree, means, scales, quats, sh, cam, settings, means2d, conics,
                   chol, depths, radii, colors, tiles_touched, stream=None):
    lib = load()
    _check(lib.gs_project_fwd(N, ld, sh_degree, _p(means), _p(scales), _p(quats), _p(sh),
                              C.byref(cam), C.byref(settings), _p(means2d), _p(conics),
                              _p(chol), _p(depths), _p(radii), _p(colors), _p(tiles_touched),
                              _stream(stream)))


def gs_bin_and_sort_workspace_size(N, capacity, width, height) -> int:
    return int(load().gs_bin_and_sort_workspace_size(N, capacity, width, height))


def gs_bin_and_sort(N, ld, means2d, radii, depths, tiles_touched, width, height, offsets,
                    capacity, keys, ids, tile_ranges, workspace, workspace_bytes, stream=None,
                    num_instances=None):
    """Returns (status, M); GS_ERR_CAPACITY is returned, not raised.
    ``num_instances``: optional page-locked one-element int64 host tensor that
    receives M (saves the runtime a staging copy)."""
    lib = load()
    M = C.c_uint64(0)
    out = C.byref(M) if num_instances is None else _p(num_instances)
    st = lib.gs_bin_and_sort(N, ld, _p(means2d), _p(radii), _p(depths), _p(tiles_touched),
                             width, height, _p(offsets), capacity, out, _p(keys), _p(ids),
                             _p(tile_ranges), _p(workspace), workspace_bytes, _stream(stream))
    if st not in (GS_OK, GS_ERR_CAPACITY):
        _check(st)
    return st, int(M.value) if num_instances is None else int(num_instances[0])


def gs_bin_and_sort_noalloc(N, ld, means2d, radii, depths, tiles_touched, width, height,
                            offsets, capacity, keys, ids, tile_ranges, stream=None,
                            num_instances=None):
    """gs_bin_and_sort with the library's own scratch (no workspace, no
    allocation).  Returns (status, M); GS_ERR_CAPACITY is returned, not
    raised."""
    lib = load()
    M = C.c_uint64(0)
    out = C.byref(M) if num_instances is None else _p(num_instances)
    st = lib.gs_bin_and_sort_noalloc(N, ld, _p(means2d), _p(radii), _p(depths),
                                     _p(tiles_touched), width, height, _p(offsets), capacity, out,
                                     _p(keys), _p(ids), _p(tile_ranges), _stream(stream))
    if st not in (GS_OK, GS_ERR_CAPACITY):
        _check(st)
    return st, int(M.value) if num_instances is None else int(num_instances[0])


@dataclasses.dataclass
class SplatPlanes:
    """The projection's planes that the compositing calls read (device
    tensors): means2d [2][ld], conics [3][ld], chol [3][ld], the caller's
    opacities [ld], colors [3][ld], radii [ld] and (for a depth output)
    depths [ld]; a batch's per-camera planes are blocks [c][P][ld]."""
    means2d: "object"
    conics: "object"
    chol: "object"
    opacities: "object"
    colors: "object"
    radii: "object"
    depths: "object" = None

    def args(self):
        return [_p(self.means2d), _p(self.conics), _p(self.chol), _p(self.opacities),
                _p(self.colors), _p(self.radii)]


@dataclasses.dataclass
class Grad2D:
    """2D gradient planes of the compositing backward: means2d [2][ld],
    conics [3][ld], opacities [ld], colors [3][ld] and, optionally, the
    absolute-gradient sums abs [2][ld]."""
    means2d: "object"
    conics: "object"
    opacities: "object"
    colors: "object"
    abs: "object" = None

    def args(self):
        return [_p(self.means2d), _p(self.conics), _p(self.opacities), _p(self.colors),
                _p(self.abs)]


def gs_rasterize_workspace_size(rows) -> int:
    return int(load().gs_rasterize_workspace_size(int(rows)))


def _bg(background):
    return (C.c_float * 3)(*[float(x) for x in background])


def gs_rasterize_fwd(N, ld, width, height, tile_ranges, ids, sp: SplatPlanes, background,
                     settings, image, final_T, last_idx, workspace, workspace_bytes,
                     out_depth=None, out_alpha=None, counters=None, stream=None,
                     tile_order=None):
    lib = load()
    _check(lib.gs_rasterize_fwd(N, ld, width, height, _p(tile_ranges), _p(tile_order), _p(ids),
                                *sp.args(), _p(sp.depths), _bg(background), C.byref(settings),
                                _p(image), _p(final_T), _p(last_idx), _p(out_depth),
                                _p(out_alpha), _p(workspace), int(workspace_bytes),
                                _p(counters), _stream(stream)))


def gs_rasterize_bwd(N, ld, width, height, tile_ranges, ids, sp: SplatPlanes, offsets,
                     tiles_touched, num_instances, background, settings, final_T, last_idx,
                     dL_dimage, workspace, workspace_bytes, staged, partials,
                     partials_capacity, g2: Grad2D, accumulate=0, counters=None, stream=None,
                     tile_order=None):
    lib = load()
    _check(lib.gs_rasterize_bwd(N, ld, width, height, _p(tile_ranges), _p(tile_order), _p(ids),
                                *sp.args(), _p(offsets), _p(tiles_touched),
                                int(num_instances), _bg(background), C.byref(settings),
                                _p(final_T), _p(last_idx), _p(dL_dimage), _p(workspace),
                                int(workspace_bytes), int(staged), _p(partials),
                                int(partials_capacity), *g2.args(), int(accumulate),
                                _p(counters), _stream(stream)))


def gs_project_bwd(N, ld, sh_degree, means, scales, quats, sh, cam, settings, radii,
                   dL_dmeans2d, dL_dconics, dL_dcolors, dL_dmeans, dL_dscales, dL_dquats,
                   dL_dsh, accumulate=0, stream=None):
    lib = load()
    _check(lib.gs_project_bwd(N, ld, sh_degree, _p(means), _p(scales), _p(quats), _p(sh),
                              C.byref(cam), C.byref(settings), _p(radii), _p(dL_dmeans2d),
                              _p(dL_dconics), _p(dL_dcolors), _p(dL_dmeans), _p(dL_dscales),
                              _p(dL_dquats), _p(dL_dsh), int(accumulate), _stream(stream)))


def gs_bin_and_sort_packed(N, ld, means2d, radii, depths, tiles_touched, width, height, offsets,
                           capacity, keys, ids, tile_ranges, vis_ids, workspace, workspace_bytes,
                           counts, stream=None):
    """Returns (status, M, V); GS_ERR_CAPACITY is returned, not raised.
    ``counts``: two-element int64 host tensor (page-locked saves a staging
    copy) that receives M and V."""
    lib = load()
    st = lib.gs_bin_and_sort_packed(N, ld, _p(means2d), _p(radii), _p(depths),
                                    _p(tiles_touched), width, height, _p(offsets), capacity,
                                    _p(counts), _p(keys), _p(ids), _p(tile_ranges),
                                    _p(vis_ids), _p(workspace), workspace_bytes,
                                    _stream(stream))
    if st not in (GS_OK, GS_ERR_CAPACITY):
        _check(st)
    return st, int(counts[0]), int(counts[1])


def gs_rasterize_bwd_packed(N, ld, width, height, tile_ranges, ids, sp: SplatPlanes, offsets,
                            tiles_touched, num_instances, vis_ids, num_visible, ldv, background,
                            settings, final_T, last_idx, dL_dimage, workspace, workspace_bytes,
                            staged, partials, partials_capacity, g2: Grad2D, accumulate=0,
                            counters=None, stream=None, tile_order=None):
    lib = load()
    _check(lib.gs_rasterize_bwd_packed(N, ld, width, height, _p(tile_ranges), _p(tile_order),
                                       _p(ids), *sp.args(), _p(offsets), _p(tiles_touched),
                                       int(num_instances), _p(vis_ids), int(num_visible),
                                       int(ldv), _bg(background), C.byref(settings),
                                       _p(final_T), _p(last_idx), _p(dL_dimage), _p(workspace),
                                       int(workspace_bytes), int(staged), _p(partials),
                                       int(partials_capacity), *g2.args(), int(accumulate),
                                       _p(counters), _stream(stream)))


def gs_project_bwd_packed(num_visible, vis_ids, N, ld, ldv, sh_degree, means, scales, quats, sh,
                          cam, settings, radii, dL_dmeans2d, dL_dconics, dL_dcolors, dL_dmeans,
                          dL_dscales, dL_dquats, dL_dsh, accumulate=0, stream=None):
    lib = load()
    _check(lib.gs_project_bwd_packed(int(num_visible), _p(vis_ids), N, ld, ldv, sh_degree,
                                     _p(means), _p(scales), _p(quats), _p(sh), C.byref(cam),
                                     C.byref(settings), _p(radii), _p(dL_dmeans2d),
                                     _p(dL_dconics), _p(dL_dcolors), _p(dL_dmeans),
                                     _p(dL_dscales), _p(dL_dquats), _p(dL_dsh),
                                     int(accumulate), _stream(stream)))


def gs_project_fwd_batched(cams, N, ld, sh_degree, means, scales, quats, sh, settings, means2d,
                           conics, chol, depths, radii, colors, tiles_touched, stream=None):
    lib = load()
    arr = (gs_camera * len(cams))(*cams)
    _check(lib.gs_project_fwd_batched(len(cams), arr, N, ld, sh_degree, _p(means), _p(scales),
                                      _p(quats), _p(sh), C.byref(settings), _p(means2d),
                                      _p(conics), _p(chol), _p(depths), _p(radii), _p(colors),
                                      _p(tiles_touched), _stream(stream)))


def gs_bin_and_sort_batched_workspace_size(num_cams, ld, capacity, width, height) -> int:
    return int(load().gs_bin_and_sort_batched_workspace_size(num_cams, ld, capacity, width,
                                                             height))


def gs_bin_and_sort_batched(num_cams, ld, means2d, radii, depths, tiles_touched, width, height,
                            offsets, capacity, keys, ids, tile_ranges, workspace,
                            workspace_bytes, num_instances, stream=None):
    """Returns (status, M); GS_ERR_CAPACITY is returned, not raised."""
    lib = load()
    st = lib.gs_bin_and_sort_batched(num_cams, ld, _p(means2d), _p(radii), _p(depths),
                                     _p(tiles_touched), width, height, _p(offsets), capacity,
                                     _p(num_instances), _p(keys), _p(ids), _p(tile_ranges),
                                     _p(workspace), workspace_bytes, _stream(stream))
    if st not in (GS_OK, GS_ERR_CAPACITY):
        _check(st)
    return st, int(num_instances[0])


def gs_rasterize_fwd_batched(num_cams, ld, width, height, tile_ranges, ids, sp: SplatPlanes,
                             background, settings, image, final_T, last_idx, workspace,
                             workspace_bytes, out_depth=None, out_alpha=None, counters=None,
                             stream=None, tile_order=None):
    lib = load()
    _check(lib.gs_rasterize_fwd_batched(num_cams, ld, width, height, _p(tile_ranges),
                                        _p(tile_order), _p(ids), *sp.args(), _p(sp.depths),
                                        _bg(background), C.byref(settings), _p(image),
                                        _p(final_T), _p(last_idx), _p(out_depth),
                                        _p(out_alpha), _p(workspace), int(workspace_bytes),
                                        _p(counters), _stream(stream)))


def gs_rasterize_bwd_batched(num_cams, ld, width, height, tile_ranges, ids, sp: SplatPlanes,
                             offsets, tiles_touched, num_instances, background, settings,
                             final_T, last_idx, dL_dimage, workspace, workspace_bytes, staged,
                             partials, partials_capacity, g2: Grad2D, accumulate=0,
                             counters=None, stream=None, tile_order=None):
    lib = load()
    _check(lib.gs_rasterize_bwd_batched(num_cams, ld, width, height, _p(tile_ranges),
                                        _p(tile_order), _p(ids), *sp.args(), _p(offsets),
                                        _p(tiles_touched), int(num_instances), _bg(background),
                                        C.byref(settings), _p(final_T), _p(last_idx),
                                        _p(dL_dimage), _p(workspace), int(workspace_bytes),
                                        int(staged), _p(partials), int(partials_capacity),
                                        *g2.args(), int(accumulate), _p(counters),
                                        _stream(stream)))


def gs_project_bwd_batched(cams, N, ld, sh_degree, means, scales, quats, sh, settings, radii,
                           dL_dmeans2d, dL_dconics, dL_dcolors, dL_dopacities_cams, dL_dmeans,
                           dL_dscales, dL_dquats, dL_dopacities, dL_dsh, accumulate=0,
                           stream=None):
    lib = load()
    arr = (gs_camera * len(cams))(*cams)
    _check(lib.gs_project_bwd_batched(len(cams), arr, N, ld, sh_degree, _p(means), _p(scales),
                                      _p(quats), _p(sh), C.byref(settings), _p(radii),
                                      _p(dL_dmeans2d), _p(dL_dconics), _p(dL_dcolors),
                                      _p(dL_dopacities_cams), _p(dL_dmeans), _p(dL_dscales),
                                      _p(dL_dquats), _p(dL_dopacities), _p(dL_dsh),
                                      int(accumulate), _stream(stream)))


def gs_bin_and_sort_device(N, ld, means2d, radii, depths, tiles_touched, width, height, offsets,
                           capacity, counts, keys, ids, tile_ranges, workspace, workspace_bytes,
                           stream=None):
    """No read-back: ``counts`` (device int64[2]) receives M and the overflow
    flag."""
    lib = load()
    _check(lib.gs_bin_and_sort_device(N, ld, _p(means2d), _p(radii), _p(depths),
                                      _p(tiles_touched), width, height, _p(offsets), capacity,
                                      _p(counts), _p(keys), _p(ids), _p(tile_ranges),
                                      _p(workspace), workspace_bytes, _stream(stream)))


def gs_rasterize_fwd_loss(N, ld, width, height, tile_ranges, ids, sp: SplatPlanes, background,
                          settings, kind, target, image, final_T, last_idx, dL_dimage,
                          workspace, workspace_bytes, out_depth=None, out_alpha=None,
                          loss=None, counters=None, stream=None, tile_order=None):
    lib = load()
    _check(lib.gs_rasterize_fwd_loss(N, ld, width, height, _p(tile_ranges), _p(tile_order),
                                     _p(ids), *sp.args(), _p(sp.depths), _bg(background),
                                     C.byref(settings), int(kind), _p(target), _p(image),
                                     _p(final_T), _p(last_idx), _p(out_depth), _p(out_alpha),
                                     _p(dL_dimage), _p(loss), _p(workspace),
                                     int(workspace_bytes), _p(counters), _stream(stream)))


def gs_rasterize_fwd_loss_batched(num_cams, ld, width, height, tile_ranges, ids,
                                  sp: SplatPlanes, background, settings, kind, target, image,
                                  final_T, last_idx, dL_dimage, workspace, workspace_bytes,
                                  out_depth=None, out_alpha=None, loss=None, counters=None,
                                  stream=None, tile_order=None):
    lib = load()
    _check(lib.gs_rasterize_fwd_loss_batched(num_cams, ld, width, height, _p(tile_ranges),
                                             _p(tile_order), _p(ids), *sp.args(),
                                             _p(sp.depths), _bg(background),
                                             C.byref(settings), int(kind), _p(target),
                                             _p(image), _p(final_T), _p(last_idx),
                                             _p(out_depth), _p(out_alpha), _p(dL_dimage),
                                             _p(loss), _p(workspace), int(workspace_bytes),
                                             _p(counters), _stream(stream)))


def gs_tile_order(num_cams, width, height, tile_ranges, tile_order, stream=None):
    """Longest-list-first schedule of each camera's tiles into tile_order
    (device uint32 [num_cams * T]), for the gs_rasterize_* calls."""
    _check(load().gs_tile_order(num_cams, width, height, _p(tile_ranges), _p(tile_order),
                                _stream(stream)))


def gs_image_loss_grad(kind, count, image, target, dL_dimage, loss=None, stream=None):
    lib = load()
    _check(lib.gs_image_loss_grad(int(kind), int(count), _p(image), _p(target), _p(dL_dimage),
                                  _p(loss), _stream(stream)))


def gs_l1_dssim_workspace_size(width, height) -> int:
    return int(load().gs_l1_dssim_workspace_size(int(width), int(height)))


def gs_l1_dssim_loss_grad(width, height, image, target, lam, dL_dimage, loss, workspace,
                          workspace_bytes, stream=None):
    lib = load()
    _check(lib.gs_l1_dssim_loss_grad(int(width), int(height), _p(image), _p(target),
                                     float(lam), _p(dL_dimage), _p(loss), _p(workspace),
                                     int(workspace_bytes), _stream(stream)))


def default_adam_config(**overrides) -> gs_adam_config:
    c = load().gs_default_adam_config()
    for k, v in overrides.items():
        setattr(c, k, float(v))
    return c


def gs_adam_step(N, ld, sh_degree, step, cfg, means, log_scales, quats, logits, sh, scales,
                 opacities, g_means, g_scales, g_quats, g_opacities, g_sh, exp_avg, exp_avg_sq,
                 stream=None):
    lib = load()
    _check(lib.gs_adam_step(N, ld, sh_degree, int(step), C.byref(cfg), _p(means),
                            _p(log_scales), _p(quats), _p(logits), _p(sh), _p(scales),
                            _p(opacities), _p(g_means), _p(g_scales), _p(g_quats),
                            _p(g_opacities), _p(g_sh), _p(exp_avg), _p(exp_avg_sq),
                            _stream(stream)))


def gs_adam_step_packed(num_visible, vis_ids, ldv, N, ld, sh_degree, step, cfg, means,
                        log_scales, quats, logits, sh, scales, opacities, g_means, g_scales,
                        g_quats, g_opacities, g_sh, exp_avg, exp_avg_sq, stream=None):
    lib = load()
    _check(lib.gs_adam_step_packed(int(num_visible), _p(vis_ids), int(ldv), N, ld, sh_degree,
                                   int(step), C.byref(cfg), _p(means), _p(log_scales),
                                   _p(quats), _p(logits), _p(sh), _p(scales), _p(opacities),
                                   _p(g_means), _p(g_scales), _p(g_quats), _p(g_opacities),
                                   _p(g_sh), _p(exp_avg), _p(exp_avg_sq), _stream(stream)))


def gs_densify_prune_workspace_size(N, clone_fraction) -> int:
    return int(load().gs_densify_prune_workspace_size(int(N), float(clone_fraction)))


def gs_densify_prune(N, ld, sh_degree, means, scales, quats, opacities, sh, dL_dmeans,
                     clone_fraction, min_opacity, ld_out, means_out, scales_out, quats_out,
                     opacities_out, sh_out, workspace, workspace_bytes, stream=None) -> int:
    """Returns the new Gaussian count."""
    lib = load()
    n_out = C.c_int64(0)
    _check(lib.gs_densify_prune(N, ld, sh_degree, _p(means), _p(scales), _p(quats),
                                _p(opacities), _p(sh), _p(dL_dmeans), float(clone_fraction),
                                float(min_opacity), ld_out, _p(means_out), _p(scales_out),
                                _p(quats_out), _p(opacities_out), _p(sh_out), C.byref(n_out),
                                _p(workspace), workspace_bytes, _stream(stream)))
    return int(n_out.value)

# ---------------------------------------------------------------------------
# Token operators
# ---------------------------------------------------------------------------
_kinds = {}            # torch dtype: gs_dtype
_F32 = _I32 = None     # torch.float32, torch.int32 (torch is imported on first use)


def _name_types():
    global _F32, _I32
    if not _kinds:
        import torch
        _F32, _I32 = torch.float32, torch.int32
        _kinds.update({torch.float32: GS_F32, torch.bfloat16: GS_BF16, torch.float16: GS_F16})


def _dtype(dtype) -> int:
    _name_types()
    if dtype not in _kinds:
        raise ValueError("dtype must be torch.float32, bfloat16 or float16, not %s" % dtype)
    return _kinds[dtype]


def _on_device(t) -> bool:
    """Whether kernels may read the tensor: device memory, or page-locked."""
    return t.is_cuda or t.is_pinned()


def _extent(t):
    """What calls hold against their configuration: type, then sizes."""
    _name_types()
    return (_kinds.get(t.dtype) if _on_device(t) else None,) + tuple(t.shape)


def heads(t) -> gs_heads:
    """The view of a [rows, heads, dim] device tensor (last dimension
    contiguous).  Calls take the tensor or its view; a view made once saves
    the calls their making it."""
    if type(t) is gs_rows or t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError("need a [rows, heads, dim] tensor with contiguous elements")
    h = gs_heads(t.data_ptr(), t.stride(0), t.stride(1))
    h.tensor, h.extent, h.address = t, _extent(t), C.addressof(h)
    return h


def rows(t) -> gs_rows:
    """The view of a [rows, channels] device tensor (last dimension
    contiguous)."""
    if type(t) is gs_heads or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("need a [rows, channels] tensor with contiguous elements")
    r = gs_rows(t.data_ptr(), t.stride(0))
    r.tensor, r.extent, r.address = t, _extent(t), C.addressof(r)
    return r


def _view(kind, make, t, want):
    """The view of a tensor, or a view that a call was given, if it has the
    type and at least the sizes ``want``: another one would be read past its
    end."""
    if t is None:
        return None
    v = t if type(t) is kind else make(t)
    e = getattr(v, "extent", None)
    if e is None:  # filled in by the caller
        v.address = C.addressof(v)
    elif e[0] != want[0] or any(x < y for x, y in zip(e[1:], want[1:])):
        raise ValueError("need a device tensor %s of the configuration's dtype, not %s of %s" %
                         (list(want[1:]), list(e[1:]), v.tensor.dtype))
    return v


def _heads(t, want):
    """want: (gs_dtype, rows, heads, dim)."""
    return t if type(t) is gs_heads and getattr(t, "extent", None) == want else \
        _view(gs_heads, heads, t, want)


def _rows(t, want):
    """want: (gs_dtype, rows, channels)."""
    return t if type(t) is gs_rows and getattr(t, "extent", None) == want else \
        _view(gs_rows, rows, t, want)


def _where(view):
    return None if view is None else view.address


def _at(t, dtype, n):
    """Device address of n contiguous elements of a dtype; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous() or \
            not (t.is_cuda or _on_device(t)):
        raise ValueError("need a contiguous %s device tensor of %d elements, not %s of %s" %
                         (dtype, n, list(t.shape), t.dtype))
    return t.data_ptr()


def _bytes(t, n):
    """Device address of n bytes of a tensor of any type; None for None."""
    if t is None:
        return None
    if t.nbytes < n or not t.is_contiguous() or not (t.is_cuda or _on_device(t)):
        raise ValueError("need a contiguous device tensor of %d bytes, not %s of %s" %
                         (n, list(t.shape), t.dtype))
    return t.data_ptr()


def documents(q_start, q_len, k_start=None, k_len=None, prefix=None, max_q_len=0,
              max_k_len=0) -> gs_documents:
    """gs_documents of int32 device tensors (kept alive with it)."""
    import torch
    arrays = (q_start, q_len, k_start, k_len, prefix)
    for t in arrays:
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous() or
                              t.numel() != q_start.numel()):
            raise ValueError("documents need contiguous int32 arrays of one length")
        if t is not None and t.numel() and not _on_device(t):
            raise ValueError("documents need device arrays")
    d = gs_documents(q_start.numel(), int(max_q_len), int(max_k_len),
                     *[None if t is None else t.data_ptr() for t in arrays])
    d.tensors = arrays
    return d


def qk_config(dtype, heads_q, heads_k, head_dim, rotary_dim=None, interleaved=False, norm=True,
              eps=1e-6, amplitude=1.0) -> gs_qk_config:
    """dtype: a torch dtype; rotary_dim: None for the whole head."""
    return gs_qk_config(_dtype(dtype), int(heads_q), int(heads_k), int(head_dim),
                        int(head_dim if rotary_dim is None else rotary_dim), int(interleaved),
                        int(norm), float(eps), float(amplitude))


def attention_config(dtype, heads_q, heads_k, head_dim, scale, causal=False, softcap=0.0,
                     slopes=None) -> gs_attention_config:
    """dtype: torch.bfloat16 or float16; slopes: fp32 device tensor [heads_q]."""
    if slopes is not None and (slopes.numel() != heads_q or not slopes.is_contiguous() or
                               _dtype(slopes.dtype) != GS_F32):
        raise ValueError("slopes must be a contiguous float32 tensor [heads_q]")
    if slopes is not None and not _on_device(slopes):
        raise ValueError("slopes must be a device tensor")
    c = gs_attention_config(_dtype(dtype), int(heads_q), int(heads_k), int(head_dim),
                            int(causal), float(scale), float(softcap),
                            None if slopes is None else slopes.data_ptr())
    c.tensor = slopes
    return c


def scan_config(dtype, channels, coupled=True) -> gs_scan_config:
    return gs_scan_config(_dtype(dtype), int(coupled), int(channels))


def _qk_arrays(cfg, n, dim, positions, inv_freq, wq, wk):
    """Addresses of a call's arrays; what the configuration leaves out is not
    looked at."""
    turned, norm = cfg.rotary_dim, cfg.norm
    return (_at(positions, _I32, n) if turned else None,
            _at(inv_freq, _F32, turned // 2) if turned else None,
            _at(wq, _F32, dim) if norm else None, _at(wk, _F32, dim) if norm else None)


def gs_qk_norm_rope_fwd(cfg, rows, positions, inv_freq, wq, wk, q, k, q_out, k_out, stream=None):
    kind, dim = cfg.dtype, cfg.head_dim
    for_q, for_k = (kind, rows, cfg.heads_q, dim), (kind, rows, cfg.heads_k, dim)
    # views made here live until the call is made
    q, k, q_out, k_out = (_heads(q, for_q), _heads(k, for_k), _heads(q_out, for_q),
                          _heads(k_out, for_k))
    _check(load().gs_qk_norm_rope_fwd(
        C.byref(cfg), rows, *_qk_arrays(cfg, rows, dim, positions, inv_freq, wq, wk), _where(q),
        _where(k), _where(q_out), _where(k_out), _stream(stream)))


def gs_qk_norm_rope_bwd_workspace_size(cfg, rows) -> int:
    return int(load().gs_qk_norm_rope_bwd_workspace_size(C.byref(cfg), rows))


def gs_qk_norm_rope_bwd(cfg, rows, positions, inv_freq, wq, wk, q, k, dL_dq_out, dL_dk_out,
                        dL_dq, dL_dk, dL_dwq, dL_dwk, workspace, workspace_bytes, stream=None):
    kind, dim, norm = cfg.dtype, cfg.head_dim, cfg.norm
    for_q, for_k = (kind, rows, cfg.heads_q, dim), (kind, rows, cfg.heads_k, dim)
    v = (_heads(q, for_q), _heads(k, for_k), _heads(dL_dq_out, for_q), _heads(dL_dk_out, for_k),
         _heads(dL_dq, for_q), _heads(dL_dk, for_k))
    _check(load().gs_qk_norm_rope_bwd(
        C.byref(cfg), rows, *_qk_arrays(cfg, rows, dim, positions, inv_freq, wq, wk),
        *map(_where, v), _at(dL_dwq, _F32, dim) if norm else None,
        _at(dL_dwk, _F32, dim) if norm else None, _bytes(workspace, workspace_bytes),
        int(workspace_bytes), _stream(stream)))


def gs_attention_fwd_workspace_size(cfg, docs, rows_q, rows_k) -> int:
    return int(load().gs_attention_fwd_workspace_size(C.byref(cfg), C.byref(docs), rows_q,
                                                      rows_k))


def gs_attention_fwd(cfg, docs, rows_q, rows_k, q, k, v, out, lse, workspace, workspace_bytes,
                     stream=None):
    """lse: fp32 [heads_q, rows_q], or None where no gradient follows."""
    kind, hq, dim = cfg.dtype, cfg.heads_q, cfg.head_dim
    for_q, for_k = (kind, rows_q, hq, dim), (kind, rows_k, cfg.heads_k, dim)
    q, k, v, out = _heads(q, for_q), _heads(k, for_k), _heads(v, for_k), _heads(out, for_q)
    _check(load().gs_attention_fwd(
        C.byref(cfg), C.byref(docs), rows_q, rows_k, _where(q), _where(k), _where(v), _where(out),
        _at(lse, _F32, hq * rows_q), _bytes(workspace, workspace_bytes), int(workspace_bytes),
        _stream(stream)))


def gs_attention_bwd_workspace_size(cfg, docs, rows_q, rows_k) -> int:
    return int(load().gs_attention_bwd_workspace_size(C.byref(cfg), C.byref(docs), rows_q,
                                                      rows_k))


def gs_attention_bwd(cfg, docs, rows_q, rows_k, q, k, v, out, lse, dL_dout, dL_dq, dL_dk, dL_dv,
                     workspace, workspace_bytes, stream=None):
    kind, hq, dim = cfg.dtype, cfg.heads_q, cfg.head_dim
    for_q, for_k = (kind, rows_q, hq, dim), (kind, rows_k, cfg.heads_k, dim)
    inputs = _heads(q, for_q), _heads(k, for_k), _heads(v, for_k), _heads(out, for_q)
    grads = (_heads(dL_dout, for_q), _heads(dL_dq, for_q), _heads(dL_dk, for_k),
             _heads(dL_dv, for_k))
    _check(load().gs_attention_bwd(
        C.byref(cfg), C.byref(docs), rows_q, rows_k, *map(_where, inputs),
        _at(lse, _F32, hq * rows_q), *map(_where, grads), _bytes(workspace, workspace_bytes),
        int(workspace_bytes), _stream(stream)))


def gs_gated_scan_saved_size(cfg, docs, rows) -> int:
    return int(load().gs_gated_scan_saved_size(C.byref(cfg), C.byref(docs), rows))


def gs_gated_scan_fwd_workspace_size(cfg, docs, rows) -> int:
    return int(load().gs_gated_scan_fwd_workspace_size(C.byref(cfg), C.byref(docs), rows))


def _saved(cfg, docs, n, saved):
    return None if saved is None else _bytes(saved, gs_gated_scan_saved_size(cfg, docs, n))


def gs_gated_scan_fwd(cfg, docs, rows, gate, x, state_in, y, state_out, saved, workspace,
                      workspace_bytes, stream=None):
    """saved: None, or gs_gated_scan_saved_size() bytes for the gradient."""
    want, states = (cfg.dtype, rows, cfg.channels), docs.count * cfg.channels
    gate, x, y = _rows(gate, want), _rows(x, want), _rows(y, want)
    _check(load().gs_gated_scan_fwd(
        C.byref(cfg), C.byref(docs), rows, _where(gate), _where(x), _at(state_in, _F32, states),
        _where(y), _at(state_out, _F32, states), _saved(cfg, docs, rows, saved),
        _bytes(workspace, workspace_bytes), int(workspace_bytes), _stream(stream)))


def gs_gated_scan_bwd_workspace_size(cfg, docs, rows) -> int:
    return int(load().gs_gated_scan_bwd_workspace_size(C.byref(cfg), C.byref(docs), rows))


def gs_gated_scan_bwd(cfg, docs, rows, gate, x, saved, dL_dy, dL_dstate_out, dL_dgate, dL_dx,
                      dL_dstate_in, workspace, workspace_bytes, stream=None):
    want, states = (cfg.dtype, rows, cfg.channels), docs.count * cfg.channels
    gate, x, dL_dy = _rows(gate, want), _rows(x, want), _rows(dL_dy, want)
    dL_dgate, dL_dx = _rows(dL_dgate, want), _rows(dL_dx, want)
    _check(load().gs_gated_scan_bwd(
        C.byref(cfg), C.byref(docs), rows, _where(gate), _where(x),
        _saved(cfg, docs, rows, saved), _where(dL_dy), _at(dL_dstate_out, _F32, states),
        _where(dL_dgate), _where(dL_dx), _at(dL_dstate_in, _F32, states),
        _bytes(workspace, workspace_bytes), int(workspace_bytes), _stream(stream)))


# ---------------------------------------------------------------------------
# Device-resident Gaussians and a frame orchestrator
# ---------------------------------------------------------------------------
@dataclasses.dataclass
class Gaussians:
    """Parameters as SoA planes [P, ld] on the GPU (first N columns used)."""
    means: "object"
    scales: "object"
    quats: "object"
    opacities: "object"
    sh: "object"
    sh_degree: int
    N: int

    @property
    def ld(self) -> int:
        return int(self.means.shape[1])

    @staticmethod
    def from_scene(scene, device="cuda", ld=None) -> "Gaussians":
        """Upload a scene with [N, ...] arrays as [P, ld] planes."""
        import torch
        N = scene.means.shape[0]
        ld = N if ld is None else ld
        K = (scene.sh_degree + 1) ** 2

        def planes(a, P):
            out = torch.zeros((P, ld), dtype=torch.float32, device=device)
            if N:
                out[:, :N] = torch.from_numpy(np.ascontiguousarray(
                    np.asarray(a, np.float32).reshape(N, P).T)).to(device)
            return out
        return Gaussians(planes(scene.means, 3), planes(scene.scales, 3), planes(scene.quats, 4),
                         planes(scene.opacities, 1), planes(scene.sh, 3 * K), scene.sh_degree, N)


def densify_prune(g: "Gaussians", dL_dmeans, clone_fraction=0.02, min_opacity=0.005,
                  ld_out=None) -> "Gaussians":
    """gs_densify_prune into freshly allocated planes (leading dimension
    ``ld_out``, default N plus the clones); returns the new Gaussians."""
    import torch
    K = (g.sh_degree + 1) ** 2
    n_clone = int(np.floor(float(np.float32(clone_fraction)) * g.N + 0.5))
    ld_out = g.N + n_clone if ld_out is None else int(ld_out)
    dev = g.means.device
    z = lambda P: torch.zeros((P, max(ld_out, 1)), dtype=torch.float32, device=dev)
    out = Gaussians(z(3), z(3), z(4), z(1), z(3 * K), g.sh_degree, 0)
    ws_bytes = gs_densify_prune_workspace_size(g.N, clone_fraction)
    ws = torch.empty((ws_bytes + 256,), dtype=torch.uint8, device=dev)
    off = (-ws.data_ptr()) % 256
    out.N = gs_densify_prune(g.N, g.ld, g.sh_degree, g.means, g.scales, g.quats, g.opacities,
                             g.sh, dL_dmeans, clone_fraction, min_opacity, max(ld_out, 1),
                             out.means, out.scales, out.quats, out.opacities, out.sh,
                             ws[off:off + ws_bytes], ws_bytes)
    return out


class Frame:
    """Buffers and calls for one camera: projection, binning + sort,
    compositing, and the two backward stages.  All buffers are torch tensors
    on the current device; only ``gs_bin_and_sort`` synchronises (to read
    the instance count).

    The stages exchange the documented planes: means2d, conics, chol,
    depths, radii, colors, tiles from the projection; g_means2d, g_conics,
    g_opacities, g_colors (and g_abs with absgrad) from the compositing
    backward; g_means, g_scales, g_quats, g_sh from the projection backward.
    ``records`` is the compositing calls' staging workspace; the backward
    reuses what the forward staged there.

    ``packed=True`` runs the packed calls: ``vis_ids[:V]`` lists the visible
    Gaussians, and columns ``[:, :V]`` of the 2D and 3D gradient planes hold
    their rows in that order (leading dimension ``ld``); nothing is written
    for the others.

    ``device_count=True`` bins without the read-back (gs_bin_and_sort_device):
    nothing in a frame waits for the GPU, so a frame can be captured into a
    HIP graph; ``check_counts()`` reads M and the overflow flag afterwards.

    ``schedule=True`` (the default) runs gs_tile_order after the binning and
    hands the schedule to the compositing calls (longest tiles first);
    ``False`` keeps their fixed order.  The outputs are the same."""

    def __init__(self, ld, sh_degree, width, height, capacity=None, settings=None,
                 background=(0.0, 0.0, 0.0), with_depth_alpha=False, device="cuda",
                 packed=False, device_count=False, schedule=True):
        import torch
        self.torch = torch
        self.device = device
        self.ld, self.sh_degree, self.W, self.H = int(ld), int(sh_degree), int(width), int(height)
        self.K = (sh_degree + 1) ** 2
        self.settings = settings if settings is not None else default_settings()
        self.background = tuple(float(x) for x in background)
        self.T = num_tiles(width, height)
        # index buffers use signed torch dtypes of the same width: the library
        # reads them as uint32/uint64 and torch only supplies the storage
        f32, i32, u32 = torch.float32, torch.int32, torch.int32
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
        self.means2d, self.conics, self.chol = z((2, ld), f32), z((3, ld), f32), z((3, ld), f32)
        self.depths, self.radii = z((ld,), f32), z((ld,), i32)
        self.colors, self.tiles = z((3, ld), f32), z((ld,), u32)
        self.offsets = z((max(ld, 1),), u32)
        self.ranges = z((self.T, 2), u32)
        self.order = z((self.T,), u32) if schedule else None
        self.image = z((height, width, 3), f32)
        self.final_T = z((height, width), f32)
        self.last_idx = z((height, width), u32)
        self.out_depth = z((height, width), f32) if with_depth_alpha else None
        self.out_alpha = z((height, width), f32) if with_depth_alpha else None
        # staged 64-byte records (torch allocations are 256-byte aligned)
        self.rec_bytes = gs_rasterize_workspace_size(ld)
        self.records = z((self.rec_bytes // 4,), f32)
        self.g_means2d, self.g_conics = z((2, ld), f32), z((3, ld), f32)
        self.g_opacities, self.g_colors = z((ld,), f32), z((3, ld), f32)
        self.g_abs = z((2, ld), f32)
        self.g_means, self.g_scales = z((3, ld), f32), z((3, ld), f32)
        self.g_quats, self.g_sh = z((4, ld), f32), z((3 * self.K, ld), f32)
        self.dL_dimage = z((height, width, 3), f32)
        self.loss = z((1,), f32)
        # page-locked host word for the instance count (allocated pinned)
        self.m_host = torch.zeros((2,), dtype=torch.int64, pin_memory=True)
        self.M = 0
        self.packed = bool(packed)
        self.device_count = bool(device_count)
        assert not (self.packed and self.device_count)
        self.counts = z((2,), torch.int64)
        self.vis_ids = z((max(ld, 1),), u32) if packed else None
        self.V = 0
        self.staged = False
        self._alloc_sort(capacity if capacity else max(1024, 4 * ld))

    def _alloc_sort(self, capacity):
        torch = self.torch
        self.capacity = int(capacity)
        self.keys = torch.zeros((self.capacity,), dtype=torch.int64, device=self.device)
        self.ids = torch.zeros((self.capacity,), dtype=torch.int32, device=self.device)
        # per-instance 48-byte gradient slots of the compositing backward
        self.partials = torch.empty((self.capacity, 12), dtype=torch.float32, device=self.device)
        self.ws_bytes = gs_bin_and_sort_workspace_size(self.ld, self.capacity, self.W, self.H)
        self.workspace = torch.zeros((self.ws_bytes + 256,), dtype=torch.uint8, device=self.device)
        # 256-byte alignment of the workspace start
        off = (-self.workspace.data_ptr()) % 256
        self.ws = self.workspace[off:off + self.ws_bytes]

    def planes(self, g: "Gaussians") -> SplatPlanes:
        return SplatPlanes(self.means2d, self.conics, self.chol, g.opacities, self.colors,
                           self.radii, self.depths)

    def grads2d(self, absgrad=False) -> Grad2D:
        return Grad2D(self.g_means2d, self.g_conics, self.g_opacities, self.g_colors,
                      self.g_abs if absgrad else None)

    def project(self, g: Gaussians, cam):
        self.cam = cam if isinstance(cam, gs_camera) else make_camera(cam)
        self.staged = False
        gs_project_fwd(g.N, g.ld, g.sh_degree, g.means, g.scales, g.quats, g.sh, self.cam,
                       self.settings, self.means2d, self.conics, self.chol, self.depths,
                       self.radii, self.colors, self.tiles)

    def _bin_and_sort_packed(self, g: Gaussians):
        args = lambda: (g.N, g.ld, self.means2d, self.radii, self.depths, self.tiles, self.W,
                        self.H, self.offsets, self.capacity, self.keys, self.ids, self.ranges,
                        self.vis_ids, self.ws, self.ws_bytes, self.m_host)
        st, M, V = gs_bin_and_sort_packed(*args())
        if st == GS_ERR_CAPACITY:
            self._alloc_sort(int(M * 1.25) + 1024)
            st, M, V = gs_bin_and_sort_packed(*args())
            _check(st)
        self.M, self.V = M, V
        self._schedule()
        return M

    def _schedule(self):
        if self.order is not None:
            gs_tile_order(1, self.W, self.H, self.ranges, self.order)

    def check_counts(self):
        """(M, overflowed) of the last device-count binning (synchronises)."""
        c = self.counts.cpu().numpy()
        return int(c[0]), bool(c[1])

    def bin_and_sort(self, g: Gaussians):
        if self.packed:
            return self._bin_and_sort_packed(g)
        if self.device_count:
            gs_bin_and_sort_device(g.N, g.ld, self.means2d, self.radii, self.depths, self.tiles,
                                   self.W, self.H, self.offsets, self.capacity, self.counts,
                                   self.keys, self.ids, self.ranges, self.ws, self.ws_bytes)
            # the instance count stays on the device; the backward bounds its
            # slots by the capacity
            self.M = self.capacity
            self._schedule()
            return None
        st, M = gs_bin_and_sort(g.N, g.ld, self.means2d, self.radii, self.depths, self.tiles,
                                self.W, self.H, self.offsets, self.capacity, self.keys, self.ids,
                                self.ranges, self.ws, self.ws_bytes, num_instances=self.m_host)
        if st == GS_ERR_CAPACITY:
            self._alloc_sort(int(M * 1.25) + 1024)
            st, M = gs_bin_and_sort(g.N, g.ld, self.means2d, self.radii, self.depths, self.tiles,
                                    self.W, self.H, self.offsets, self.capacity, self.keys,
                                    self.ids, self.ranges, self.ws, self.ws_bytes,
                                    num_instances=self.m_host)
            _check(st)
        self.M = M
        self._schedule()
        return M

    def rasterize_loss(self, g: Gaussians, target, kind, with_loss=False, counters=None):
        """Compositing with the loss gradient fused in: dL_dimage (and the
        loss value when with_loss) against target."""
        gs_rasterize_fwd_loss(g.N, g.ld, self.W, self.H, self.ranges, self.ids, self.planes(g),
                              self.background, self.settings, kind, target, self.image,
                              self.final_T, self.last_idx, self.dL_dimage, self.records,
                              self.rec_bytes, self.out_depth, self.out_alpha,
                              self.loss if with_loss else None, counters,
                              tile_order=self.order)
        self.staged = True

    def rasterize(self, g: Gaussians, counters=None):
        gs_rasterize_fwd(g.N, g.ld, self.W, self.H, self.ranges, self.ids, self.planes(g),
                         self.background, self.settings, self.image, self.final_T,
                         self.last_idx, self.records, self.rec_bytes, self.out_depth,
                         self.out_alpha, counters, tile_order=self.order)
        self.staged = True

    def forward(self, g: Gaussians, cam):
        self.project(g, cam)
        self.bin_and_sort(g)
        self.rasterize(g)
        return self.image

    def loss_grad(self, target, kind, with_loss=True):
        gs_image_loss_grad(kind, self.W * self.H * 3, self.image, target, self.dL_dimage,
                           self.loss if with_loss else None)

    def rasterize_backward(self, g: Gaussians, dL_dimage=None, counters=None, absgrad=False,
                           accumulate=0):
        dl = self.dL_dimage if dL_dimage is None else dL_dimage
        common = (g.N, g.ld, self.W, self.H, self.ranges, self.ids, self.planes(g), self.offsets,
                  self.tiles, self.M)
        if self.packed:
            gs_rasterize_bwd_packed(*common, self.vis_ids, self.V, self.ld, self.background,
                                    self.settings, self.final_T, self.last_idx, dl, self.records,
                                    self.rec_bytes, int(self.staged), self.partials,
                                    self.capacity, self.grads2d(absgrad), accumulate,
                                    counters=counters, tile_order=self.order)
        else:
            gs_rasterize_bwd(*common, self.background, self.settings, self.final_T,
                             self.last_idx, dl, self.records, self.rec_bytes, int(self.staged),
                             self.partials, self.capacity, self.grads2d(absgrad), accumulate,
                             counters=counters, tile_order=self.order)
        self.staged = True

    def project_backward(self, g: Gaussians, accumulate=0):
        if self.packed:
            gs_project_bwd_packed(self.V, self.vis_ids, g.N, g.ld, self.ld, g.sh_degree, g.means,
                                  g.scales, g.quats, g.sh, self.cam, self.settings, self.radii,
                                  self.g_means2d, self.g_conics, self.g_colors, self.g_means,
                                  self.g_scales, self.g_quats, self.g_sh, accumulate)
            return
        gs_project_bwd(g.N, g.ld, g.sh_degree, g.means, g.scales, g.quats, g.sh, self.cam,
                       self.settings, self.radii, self.g_means2d, self.g_conics, self.g_colors,
                       self.g_means, self.g_scales, self.g_quats, self.g_sh, accumulate)

    def backward(self, g: Gaussians, dL_dimage=None, accumulate=0, absgrad=False):
        """accumulate: add this frame's gradients with respect to the
        Gaussians (the opacities' and absolute sums included) to the
        buffers' contents; the 2D planes hold this frame's own."""
        self.rasterize_backward(g, dL_dimage, absgrad=absgrad, accumulate=2 if accumulate else 0)
        self.project_backward(g, accumulate)


class BatchFrame:
    """Forward of a batch of cameras (one image size) with one launch per
    stage: projection, binning + sort, compositing.  Per-camera outputs are
    blocks [c] of each buffer; only the binning synchronises.  ``schedule``
    as for Frame."""

    def __init__(self, ld, sh_degree, width, height, num_cams, capacity=None, settings=None,
                 background=(0.0, 0.0, 0.0), with_depth_alpha=False, device="cuda",
                 schedule=True):
        import torch
        self.torch = torch
        self.device = device
        self.ld, self.sh_degree, self.W, self.H = int(ld), int(sh_degree), int(width), int(height)
        self.C = int(num_cams)
        self.settings = settings if settings is not None else default_settings()
        self.background = tuple(float(x) for x in background)
        self.T = num_tiles(width, height)
        C_, ld_ = self.C, self.ld
        f32, i32 = torch.float32, torch.int32
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
        self.means2d, self.conics = z((C_, 2, ld_), f32), z((C_, 3, ld_), f32)
        self.chol = z((C_, 3, ld_), f32)
        self.depths, self.radii = z((C_, ld_), f32), z((C_, ld_), i32)
        self.colors, self.tiles = z((C_, 3, ld_), f32), z((C_, ld_), i32)
        self.offsets = z((max(C_ * ld_, 1),), i32)
        self.rec_bytes = gs_rasterize_workspace_size(C_ * ld_)
        self.records = z((self.rec_bytes // 4,), f32)
        self.ranges = z((C_ * self.T, 2), i32)
        self.order = z((C_ * self.T,), i32) if schedule else None
        self.image = z((C_, height, width, 3), f32)
        self.final_T = z((C_, height, width), f32)
        self.last_idx = z((C_, height, width), i32)
        self.out_depth = z((C_, height, width), f32) if with_depth_alpha else None
        self.out_alpha = z((C_, height, width), f32) if with_depth_alpha else None
        self.m_host = torch.zeros((1,), dtype=torch.int64, pin_memory=True)
        self.M = 0
        # backward: per-camera images and 2D gradient planes, 3D gradients
        # (and the opacity gradient) summed over the batch's cameras
        K = (sh_degree + 1) ** 2
        self.dL_dimage = z((C_, height, width, 3), f32)
        self.g_means2d, self.g_conics = z((C_, 2, ld_), f32), z((C_, 3, ld_), f32)
        self.g_opacities_cams, self.g_colors = z((C_, ld_), f32), z((C_, 3, ld_), f32)
        self.g_abs = z((C_, 2, ld_), f32)
        self.g_means, self.g_scales = z((3, ld_), f32), z((3, ld_), f32)
        self.g_quats, self.g_opacities = z((4, ld_), f32), z((ld_,), f32)
        self.g_sh = z((3 * K, ld_), f32)
        self._alloc_sort(capacity if capacity else max(1024, 4 * C_ * ld_))

    def _alloc_sort(self, capacity):
        torch = self.torch
        self.capacity = int(capacity)
        self.keys = torch.zeros((self.capacity,), dtype=torch.int64, device=self.device)
        self.ids = torch.zeros((self.capacity,), dtype=torch.int32, device=self.device)
        self.partials = torch.empty((self.capacity, 12), dtype=torch.float32, device=self.device)
        self.ws_bytes = gs_bin_and_sort_batched_workspace_size(self.C, self.ld, self.capacity,
                                                               self.W, self.H)
        self.workspace = torch.zeros((self.ws_bytes + 256,), dtype=torch.uint8,
                                     device=self.device)
        off = (-self.workspace.data_ptr()) % 256
        self.ws = self.workspace[off:off + self.ws_bytes]

    def planes(self, g: "Gaussians") -> SplatPlanes:
        return SplatPlanes(self.means2d, self.conics, self.chol, g.opacities, self.colors,
                           self.radii, self.depths)

    def forward(self, g: "Gaussians", cams, target=None, kind=1, loss=None):
        """The batch's forward; with ``target`` ([C][H][W][3]) the loss
        gradient (kind 0: L2, 1: L1) goes to dL_dimage in the same pass, and
        the summed loss to ``loss`` (a device float) when given."""
        assert len(cams) == self.C
        self.cams = [c if isinstance(c, gs_camera) else make_camera(c) for c in cams]
        gs_project_fwd_batched(self.cams, g.N, g.ld, g.sh_degree, g.means, g.scales, g.quats,
                               g.sh, self.settings, self.means2d, self.conics, self.chol,
                               self.depths, self.radii, self.colors, self.tiles)
        args = lambda: (self.C, self.ld, self.means2d, self.radii, self.depths, self.tiles,
                        self.W, self.H, self.offsets, self.capacity, self.keys, self.ids,
                        self.ranges, self.ws, self.ws_bytes, self.m_host)
        st, M = gs_bin_and_sort_batched(*args())
        if st == GS_ERR_CAPACITY:
            self._alloc_sort(int(M * 1.25) + 1024)
            st, M = gs_bin_and_sort_batched(*args())
            _check(st)
        self.M = M
        if self.order is not None:
            gs_tile_order(self.C, self.W, self.H, self.ranges, self.order)
        if target is None:
            gs_rasterize_fwd_batched(self.C, self.ld, self.W, self.H, self.ranges, self.ids,
                                     self.planes(g), self.background, self.settings,
                                     self.image, self.final_T, self.last_idx, self.records,
                                     self.rec_bytes, self.out_depth, self.out_alpha,
                                     tile_order=self.order)
        else:
            # the loss gradient into dL_dimage, fused into the compositing
            gs_rasterize_fwd_loss_batched(self.C, self.ld, self.W, self.H, self.ranges,
                                          self.ids, self.planes(g), self.background,
                                          self.settings, kind, target, self.image,
                                          self.final_T, self.last_idx, self.dL_dimage,
                                          self.records, self.rec_bytes, self.out_depth,
                                          self.out_alpha, loss=loss, tile_order=self.order)
        return self.image

    def backward(self, g: "Gaussians", dL_dimage=None, accumulate=0, absgrad=False):
        """Compositing backward of every camera (per-camera 2D gradient
        planes), then the projection backward summed over the cameras into
        g_means ... g_sh, and the opacity gradients summed into g_opacities."""
        dl = self.dL_dimage if dL_dimage is None else dL_dimage
        g2 = Grad2D(self.g_means2d, self.g_conics, self.g_opacities_cams, self.g_colors,
                    self.g_abs if absgrad else None)
        gs_rasterize_bwd_batched(self.C, self.ld, self.W, self.H, self.ranges, self.ids,
                                 self.planes(g), self.offsets, self.tiles, self.M,
                                 self.background, self.settings, self.final_T, self.last_idx,
                                 dl, self.records, self.rec_bytes, 1, self.partials,
                                 self.capacity, g2, 0, tile_order=self.order)
        gs_project_bwd_batched(self.cams, g.N, g.ld, g.sh_degree, g.means, g.scales, g.quats,
                               g.sh, self.settings, self.radii, self.g_means2d, self.g_conics,
                               self.g_colors, self.g_opacities_cams, self.g_means, self.g_scales,
                               self.g_quats, self.g_opacities, self.g_sh, accumulate)
