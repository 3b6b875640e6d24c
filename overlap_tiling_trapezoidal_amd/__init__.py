"""Python binding of libtdp: tiled-data-parallel latent tiling on MI355X.

Thin ctypes layer over the C ABI declared in ``include/tdp.h``: the names are
the C names, and every step of the hot path runs in the library's HIP
kernels.  This module only marshals arguments: it checks tensors (device,
dtype, contiguity and size against the plan) before any pointer reaches the
library, so a wrong buffer raises here instead of reaching a kernel.

PyTorch supplies device memory and streams; nothing here computes.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
DEFAULT_LIB_PATH = os.path.join(_HERE, "libtdp.so")
# TDP_LIBRARY names another build to load instead, e.g. the host-only planner
# built with address and undefined-behaviour sanitizers for the CPU tests
# (build.py --host-sanitized); such a build may lack the device entry points.
LIB_PATH = os.environ.get("TDP_LIBRARY") or DEFAULT_LIB_PATH
DEVICE_FUNCTIONS = ("tdp_extract", "tdp_extract_noalloc", "tdp_set_lookback_polls", "tdp_pipeline_step",
                    "tdp_extract_positions", "tdp_extract_latent", "tdp_pipeline_latent_step", "tdp_blend",
                    "tdp_blend_tile", "tdp_blend_finish", "tdp_pixel_blend", "tdp_rope_apply", "tdp_qk_norm_rope",
                    "tdp_qk_norm_rope_backward", "tdp_attention", "tdp_attention_backward", "tdp_layer_norm",
                    "tdp_layer_norm_backward", "tdp_window_attention", "tdp_window_attention_backward",
                    "tdp_grouped_product", "tdp_grouped_product_backward")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "tdp.h")

# ---- constants (mirror include/tdp.h) --------------------------------------
TDP_OK = 0
TDP_EINVAL = -1
TDP_EGUARD = -2
TDP_ESHAPE = -3
TDP_EHIP = -4
TDP_F32 = 0
TDP_BF16 = 1
TDP_NORMALIZE_POSITIONS = 0x1
TDP_UNGUARDED = 0x2
TDP_MAX_TILES_PER_AXIS = 32
TDP_STATIC_SCRATCH_BYTES = 1 << 20
TDP_PAIR_INTERLEAVED = 0
TDP_PAIR_HALVES = 1
TDP_POINT_MIDDLE = 0
TDP_POINT_START = 1
TDP_MAX_ROPE_DIM = 256
TDP_MAX_ATTENTION_DIM = 128
TDP_MAX_CHANNELS = 8192
TDP_WINDOW_ALL = 1 << 30
TDP_MAX_FEATURES = 65536

_DTYPES = {"f32": TDP_F32, "float32": TDP_F32, "bf16": TDP_BF16, "bfloat16": TDP_BF16}


class tdp_axis_tiling(ctypes.Structure):
    _fields_ = [("num_tiles", ctypes.c_int32), ("overlap", ctypes.c_int32)]


class tdp_config(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("channels", ctypes.c_int32),
        ("frames", ctypes.c_int32),
        ("height", ctypes.c_int32),
        ("width", ctypes.c_int32),
        ("num_cond", ctypes.c_int32),
        ("axis", tdp_axis_tiling * 3),
        ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
    ]


class tdp_tile_info(ctypes.Structure):
    _fields_ = [
        ("index", ctypes.c_int32),
        ("grid", ctypes.c_int32 * 3),
        ("origin", ctypes.c_int32 * 3),
        ("shape", ctypes.c_int32 * 3),
        ("gen_tokens", ctypes.c_int32),
        ("capacity", ctypes.c_int32),
        ("lat_offset", ctypes.c_int64),
        ("pos_offset", ctypes.c_int64),
        ("index_offset", ctypes.c_int64),
    ]


class tdp_sizes(ctypes.Structure):
    _fields_ = [
        ("num_slots", ctypes.c_int32),
        ("tile_lat_elems", ctypes.c_int64),
        ("tile_pos_floats", ctypes.c_int64),
        ("tile_index_ints", ctypes.c_int64),
        ("cond_row_ints", ctypes.c_int64),
        ("cond_k_ints", ctypes.c_int64),
        ("out_elems", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64),
    ]


class tdp_pixel_config(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("channels", ctypes.c_int32),
        ("frames", ctypes.c_int32),
        ("height", ctypes.c_int32),
        ("width", ctypes.c_int32),
        ("scale", ctypes.c_int32 * 2),
        ("axis", tdp_axis_tiling * 2),
        ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
    ]


class tdp_pixel_tile(ctypes.Structure):
    _fields_ = [
        ("index", ctypes.c_int32),
        ("grid", ctypes.c_int32 * 2),
        ("origin", ctypes.c_int32 * 2),
        ("shape", ctypes.c_int32 * 2),
        ("offset", ctypes.c_int64),
        ("elems", ctypes.c_int64),
    ]


class tdp_quality(ctypes.Structure):
    _fields_ = [
        ("total_cells", ctypes.c_int64),
        ("grid_cells", ctypes.c_int64),
        ("largest_cells", ctypes.c_int64),
        ("seams", ctypes.c_int64),
        ("max_rank_cells", ctypes.c_int64),
        ("area_ratio", ctypes.c_double),
        ("largest_fraction", ctypes.c_double),
        ("imbalance", ctypes.c_double),
    ]


class tdp_seqs(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("max_rows", ctypes.c_int32),
        ("total_rows", ctypes.c_int64),
        ("row_range", ctypes.c_void_p),
        ("seq_len", ctypes.c_void_p),
        ("len_group", ctypes.c_int32),
    ]


class tdp_heads(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("seq_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("heads", ctypes.c_int32),
    ]


class tdp_window(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("step", "back", "ahead", "sinks")]


class tdp_rows(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("seq_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
    ]


class tdp_rope_config(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32 * 3),
        ("pairing", ctypes.c_int32),
        ("point", ctypes.c_int32),
    ]


class TdpError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} [{status}]")
        self.status = status


_lib = None
HOST_ONLY = False  # the loaded build has the host planner only (no device entry points)


def load_library(path: str = LIB_PATH):
    """Load libtdp.so; raises ImportError when it has not been built."""
    global _lib, HOST_ONLY
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libtdp.so not found at {path}: build it first "
                          "(python overlap_tiling_trapezoidal_amd/build.py)")
    lib = ctypes.CDLL(path)
    vp, i32, i32p = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)
    f32, sq, hd = ctypes.c_float, ctypes.POINTER(tdp_seqs), ctypes.POINTER(tdp_heads)
    rw, wn = ctypes.POINTER(tdp_rows), ctypes.POINTER(tdp_window)
    sig = {
        "tdp_plan_create": (ctypes.c_int, [ctypes.POINTER(tdp_config), ctypes.POINTER(vp)]),
        "tdp_plan_create_rank": (ctypes.c_int, [ctypes.POINTER(tdp_config), i32, i32, ctypes.POINTER(vp)]),
        "tdp_plan_local_tiles": (ctypes.c_int, [vp, i32p, i32p, i32p]),
        "tdp_plan_destroy": (None, [vp]),
        "tdp_plan_num_tiles": (ctypes.c_int, [vp, i32p]),
        "tdp_plan_intervals": (ctypes.c_int, [vp, ctypes.c_int, i32p, i32p]),
        "tdp_plan_window": (ctypes.c_int, [vp, ctypes.c_int, i32, ctypes.POINTER(ctypes.c_float)]),
        "tdp_plan_tile": (ctypes.c_int, [vp, i32, ctypes.POINTER(tdp_tile_info)]),
        "tdp_plan_cell_tiles": (ctypes.c_int, [vp, ctypes.c_int, i32, i32p, i32p]),
        "tdp_plan_sizes": (ctypes.c_int, [vp, ctypes.POINTER(tdp_sizes)]),
        "tdp_plan_tile_rank": (ctypes.c_int, [vp, i32, i32, i32p]),
        "tdp_tiling_quality": (ctypes.c_int, [i32, i32p, i32p, i32p, i32p, i32, ctypes.POINTER(tdp_quality),
                                              ctypes.POINTER(ctypes.c_int64)]),
        "tdp_plan_quality": (ctypes.c_int, [vp, i32, ctypes.POINTER(tdp_quality), ctypes.POINTER(ctypes.c_int64)]),
        "tdp_extract": (ctypes.c_int, [vp] * 11),
        "tdp_extract_noalloc": (ctypes.c_int, [vp] * 10),
        "tdp_set_lookback_polls": (ctypes.c_int, [i32]),
        "tdp_pipeline_step": (ctypes.c_int, [vp] * 15),
        "tdp_extract_positions": (ctypes.c_int, [vp] * 9),
        "tdp_extract_latent": (ctypes.c_int, [vp] * 5),
        "tdp_pipeline_latent_step": (ctypes.c_int, [vp] * 9),
        "tdp_blend": (ctypes.c_int, [vp] * 6),
        "tdp_blend_tile": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, vp]),
        "tdp_blend_finish": (ctypes.c_int, [vp] * 4),
        "tdp_pixel_plan_create": (ctypes.c_int, [ctypes.POINTER(tdp_pixel_config), ctypes.POINTER(vp)]),
        "tdp_pixel_plan_destroy": (None, [vp]),
        "tdp_pixel_plan_tile": (ctypes.c_int, [vp, i32, ctypes.POINTER(tdp_pixel_tile)]),
        "tdp_pixel_plan_sizes": (ctypes.c_int, [vp, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
                                                i32p]),
        "tdp_pixel_blend": (ctypes.c_int, [vp] * 4),
        "tdp_plan_sequences": (ctypes.c_int, [vp, ctypes.POINTER(ctypes.c_int64)]),
        "tdp_rope_create": (ctypes.c_int, [ctypes.POINTER(tdp_rope_config), ctypes.POINTER(ctypes.c_double),
                                           ctypes.POINTER(vp)]),
        "tdp_rope_destroy": (None, [vp]),
        "tdp_rope_apply": (ctypes.c_int, [vp, sq, vp, hd, hd, i32, i32, vp]),
        "tdp_qk_norm_rope": (ctypes.c_int, [vp, sq, vp, hd, hd, vp, vp, hd, hd, f32, i32, vp]),
        "tdp_qk_norm_rope_workspace": (ctypes.c_int64, [vp, sq, i32, i32]),
        "tdp_qk_norm_rope_backward": (ctypes.c_int, [vp, sq, vp, hd, hd, vp, vp, hd, hd, hd, hd, vp, vp, f32, i32, vp,
                                                     vp]),
        "tdp_attention_workspace": (ctypes.c_int64, [sq, sq, i32, i32, i32]),
        "tdp_attention": (ctypes.c_int, [sq, sq, hd, hd, hd, vp, hd, vp, f32, i32, i32, vp, vp]),
        "tdp_attention_backward_workspace": (ctypes.c_int64, [sq, sq, i32, i32, i32]),
        "tdp_attention_backward": (ctypes.c_int, [sq, sq, hd, hd, hd, vp, hd, vp, hd, hd, hd, hd, f32, i32, i32, vp,
                                                  vp]),
        "tdp_window_attention_workspace": (ctypes.c_int64, [sq, sq, wn, i32, i32, i32]),
        "tdp_window_attention": (ctypes.c_int, [sq, sq, wn, hd, hd, hd, hd, vp, f32, i32, i32, vp, vp]),
        "tdp_window_attention_backward_workspace": (ctypes.c_int64, [sq, sq, wn, i32, i32, i32]),
        "tdp_window_attention_backward": (ctypes.c_int, [sq, sq, wn, hd, hd, hd, hd, vp, hd, hd, hd, hd, f32, i32, i32,
                                                         vp, vp]),
        "tdp_layer_norm": (ctypes.c_int, [sq, rw, vp, vp, i32, rw, f32, i32, i32, vp]),
        "tdp_layer_norm_workspace": (ctypes.c_int64, [sq, i32, i32]),
        "tdp_layer_norm_backward": (ctypes.c_int, [sq, rw, vp, i32, rw, rw, vp, vp, f32, i32, i32, vp, vp]),
        "tdp_grouped_product_workspace": (ctypes.c_int64, [sq, i32, i32, i32, i32]),
        "tdp_grouped_product": (ctypes.c_int, [sq, rw, vp, i32, rw, i32, i32, i32, vp, vp]),
        "tdp_grouped_product_backward_workspace": (ctypes.c_int64, [sq, i32, i32, i32, i32]),
        "tdp_grouped_product_backward": (ctypes.c_int, [sq, rw, vp, i32, rw, rw, vp, i32, i32, i32, vp, vp]),
        "tdp_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "tdp_last_error": (ctypes.c_char_p, []),
    }
    missing = [name for name in sig if not hasattr(lib, name)]
    if missing and (path == DEFAULT_LIB_PATH or any(m not in DEVICE_FUNCTIONS for m in missing)):
        raise ImportError(f"{path} does not export {', '.join(missing)}")
    for name, (res, args) in sig.items():
        if name in missing:
            continue
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    HOST_ONLY = bool(missing)
    _lib = lib
    return lib


def _header_functions_in(path: str) -> list[str]:
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tdp_[a-z_]+)\s*\(", text)))


def header_functions(path: str = HEADER_PATH) -> list[str]:
    """Names of the functions include/tdp.h declares."""
    return _header_functions_in(path)


def _check(status: int):
    if status != TDP_OK:
        lib = load_library()
        raise TdpError(status, lib.tdp_last_error().decode())


# ---- plan -----------------------------------------------------------------

def make_config(batch, channels, shape, tiling, num_cond=0, in_dtype="bf16", out_dtype=None,
                normalize=True, unguarded=False) -> tdp_config:
    """Fill a tdp_config.  ``shape`` = (F, H, W); ``tiling`` = ((n, o),) * 3."""
    cfg = tdp_config()
    cfg.batch, cfg.channels = batch, channels
    cfg.frames, cfg.height, cfg.width = shape
    cfg.num_cond = num_cond
    for d, (n, o) in enumerate(tiling):
        cfg.axis[d].num_tiles, cfg.axis[d].overlap = n, o
    cfg.in_dtype = _DTYPES[in_dtype] if isinstance(in_dtype, str) else in_dtype
    out_dtype = in_dtype if out_dtype is None else out_dtype
    cfg.out_dtype = _DTYPES[out_dtype] if isinstance(out_dtype, str) else out_dtype
    cfg.flags = (TDP_NORMALIZE_POSITIONS if normalize else 0) | (TDP_UNGUARDED if unguarded else 0)
    return cfg


class Plan:
    """Owns a tdp_plan handle (host memory only)."""

    def __init__(self, handle: int, cfg: tdp_config):
        self._h = ctypes.c_void_p(handle)
        self.cfg = cfg

    @property
    def handle(self):
        if not self._h:
            raise ValueError("plan was destroyed")
        return self._h

    def destroy(self):
        if self._h:
            load_library().tdp_plan_destroy(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    # derived geometry
    @property
    def shape(self):
        return (self.cfg.frames, self.cfg.height, self.cfg.width)

    @property
    def tokens(self):
        F, H, W = self.shape
        return F * H * W


def tdp_plan_create(cfg: tdp_config) -> Plan:
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.tdp_plan_create(ctypes.byref(cfg), ctypes.byref(h)))
    return Plan(h.value, cfg)


def tdp_plan_create_rank(cfg: tdp_config, world: int, rank: int) -> Plan:
    """Plan of rank ``rank``'s round-robin share of the tiles over ``world`` ranks."""
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.tdp_plan_create_rank(ctypes.byref(cfg), world, rank, ctypes.byref(h)))
    return Plan(h.value, cfg)


def tdp_plan_local_tiles(plan: Plan) -> tuple[int, int, int]:
    """(world, rank, number of tiles the plan holds)."""
    w, r, n = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(load_library().tdp_plan_local_tiles(plan.handle, ctypes.byref(w), ctypes.byref(r), ctypes.byref(n)))
    return w.value, r.value, n.value


def held_tiles(plan: Plan) -> list[int]:
    """Tile indices the plan holds, in slot order (t = rank + slot * world)."""
    world, rank, n = tdp_plan_local_tiles(plan)
    return [rank + j * world for j in range(n)]


def tdp_plan_destroy(plan: Plan):
    plan.destroy()


def tdp_plan_num_tiles(plan: Plan) -> int:
    n = ctypes.c_int32()
    _check(load_library().tdp_plan_num_tiles(plan.handle, ctypes.byref(n)))
    return n.value


def tdp_plan_intervals(plan: Plan, axis: int) -> list[tuple[int, int]]:
    n = plan.cfg.axis[axis].num_tiles if 0 <= axis < 3 else 1
    starts = (ctypes.c_int32 * max(n, 1))()
    ends = (ctypes.c_int32 * max(n, 1))()
    _check(load_library().tdp_plan_intervals(plan.handle, axis, starts, ends))
    return [(starts[i], ends[i]) for i in range(n)]


def tdp_plan_window(plan: Plan, axis: int, i: int):
    import numpy as np
    ivs = tdp_plan_intervals(plan, axis)
    if not 0 <= i < len(ivs):
        raise IndexError(i)
    size = ivs[i][1] - ivs[i][0]
    buf = (ctypes.c_float * size)()
    _check(load_library().tdp_plan_window(plan.handle, axis, i, buf))
    return np.ctypeslib.as_array(buf).copy()


def tdp_plan_cell_tiles(plan: Plan, axis: int, x: int) -> list[int]:
    tiles = (ctypes.c_int32 * 2)()
    n = ctypes.c_int32()
    _check(load_library().tdp_plan_cell_tiles(plan.handle, axis, x, tiles, ctypes.byref(n)))
    return [tiles[i] for i in range(n.value)]


def tdp_plan_tile(plan: Plan, t: int) -> tdp_tile_info:
    info = tdp_tile_info()
    _check(load_library().tdp_plan_tile(plan.handle, t, ctypes.byref(info)))
    return info


def tdp_plan_sizes(plan: Plan) -> tdp_sizes:
    s = tdp_sizes()
    _check(load_library().tdp_plan_sizes(plan.handle, ctypes.byref(s)))
    return s


def tdp_plan_tile_rank(plan: Plan, t: int, world: int) -> int:
    r = ctypes.c_int32()
    _check(load_library().tdp_plan_tile_rank(plan.handle, t, world, ctypes.byref(r)))
    return r.value


def tdp_status_string(status: int) -> str:
    return load_library().tdp_status_string(status).decode()


def tdp_last_error() -> str:
    return load_library().tdp_last_error().decode()


# ---- device buffers (torch) ----------------------------------------------

def _torch_dtype(code: int):
    import torch
    return torch.bfloat16 if code == TDP_BF16 else torch.float32


def _ptr(t, name, dtype, numel, device):
    """Pointer of a CUDA tensor after checking it can hold ``numel`` elements."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'a GPU'}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
    return ctypes.c_void_p(t.data_ptr())


def _quality_dict(q: tdp_quality, ranks) -> dict:
    d = {name: getattr(q, name) for name, _ in tdp_quality._fields_}
    d["rank_cells"] = list(ranks)
    return d


def tdp_tiling_quality(dims, intervals, world: int) -> dict:
    """Cost figures of a tiling given per-axis [start, end) intervals."""
    nd = len(dims)
    arr = lambda xs: (ctypes.c_int32 * max(1, len(xs)))(*xs)  # noqa: E731
    starts = [a for ivs in intervals for a, _ in ivs]
    ends = [b for ivs in intervals for _, b in ivs]
    q = tdp_quality()
    ranks = (ctypes.c_int64 * max(1, world))()
    _check(load_library().tdp_tiling_quality(nd, arr(list(dims)), arr([len(v) for v in intervals]), arr(starts),
                                              arr(ends), world, ctypes.byref(q), ranks))
    return _quality_dict(q, ranks[:world])


def tdp_plan_quality(plan: Plan, world: int) -> dict:
    """Cost figures of a plan's tiles on ``world`` round-robin ranks."""
    q = tdp_quality()
    ranks = (ctypes.c_int64 * max(1, world))()
    _check(load_library().tdp_plan_quality(plan.handle, world, ctypes.byref(q), ranks))
    return _quality_dict(q, ranks[:world])


def allocate_extract_outputs(plan: Plan, device="cuda"):
    """Caller-owned buffers for tdp_extract / tdp_blend, sized by the plan
    (the keys are tdp_extract's argument names)."""
    import torch
    s = tdp_plan_sizes(plan)
    dev = torch.device(device)
    return {
        "tile_lat": torch.empty(s.tile_lat_elems, dtype=_torch_dtype(plan.cfg.in_dtype), device=dev),
        "tile_pos": torch.empty(s.tile_pos_floats, dtype=torch.float32, device=dev),
        "tile_index": torch.empty(s.tile_index_ints, dtype=torch.int32, device=dev),
        "tile_count": torch.empty(max(s.num_slots, 1), dtype=torch.int32, device=dev),
        "cond_row": torch.empty(max(s.cond_row_ints, 1), dtype=torch.int32, device=dev),
        "cond_k": torch.empty(max(s.cond_k_ints, 1), dtype=torch.int32, device=dev),
        "workspace": torch.empty(max(s.workspace_bytes, 1), dtype=torch.uint8, device=dev),
    }


def allocate_output(plan: Plan, device="cuda"):
    import torch
    s = tdp_plan_sizes(plan)
    c = plan.cfg
    return torch.empty(s.out_elems, dtype=_torch_dtype(c.out_dtype),
                       device=torch.device(device)).view(c.batch, plan.tokens + c.num_cond, c.channels)


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _extract_args(plan: Plan, latent, pos, tile_lat, tile_pos, tile_index, tile_count, cond_row, cond_k):
    import torch
    c = plan.cfg
    s = tdp_plan_sizes(plan)
    rows = plan.tokens + c.num_cond
    dev = latent.device
    none = ctypes.c_void_p(None)
    return [
        plan.handle,
        _ptr(latent, "latent", _torch_dtype(c.in_dtype), c.batch * rows * c.channels, dev),
        _ptr(pos, "pos", torch.float32, c.batch * 3 * rows * 2, dev),
        _ptr(tile_lat, "tile_lat", _torch_dtype(c.in_dtype), s.tile_lat_elems, dev),
        _ptr(tile_pos, "tile_pos", torch.float32, s.tile_pos_floats, dev),
        _ptr(tile_index, "tile_index", torch.int32, s.tile_index_ints, dev),
        _ptr(tile_count, "tile_count", torch.int32, s.num_slots, dev),
        _ptr(cond_row, "cond_row", torch.int32, s.cond_row_ints, dev) if c.num_cond else none,
        _ptr(cond_k, "cond_k", torch.int32, s.cond_k_ints, dev) if c.num_cond else none,
    ]


def tdp_extract(plan: Plan, latent, pos, tile_lat, tile_pos, tile_index, tile_count,
                cond_row=None, cond_k=None, workspace=None, stream=None):
    """Enqueue the tile gather on ``stream`` (default: torch's current stream)."""
    import torch
    s = tdp_plan_sizes(plan)
    dev = latent.device
    args = _extract_args(plan, latent, pos, tile_lat, tile_pos, tile_index, tile_count, cond_row, cond_k)
    args.append(_ptr(workspace, "workspace", torch.uint8, s.workspace_bytes, dev) if s.workspace_bytes
                else ctypes.c_void_p(None))
    args.append(_stream_handle(stream, dev))
    _check(load_library().tdp_extract(*args))


def tdp_set_lookback_polls(polls: int):
    """Reads of an unpublished look-back flag before a conditioning selection
    wave counts that chunk itself (process-wide; results do not depend on it)."""
    _check(load_library().tdp_set_lookback_polls(int(polls)))


def tdp_extract_noalloc(plan: Plan, latent, pos, tile_lat, tile_pos, tile_index, tile_count,
                        cond_row=None, cond_k=None, stream=None):
    """tdp_extract with the library's static per-GPU workspace in place of a
    caller's (for callers that cannot allocate device memory; calls that
    overlap on one GPU race)."""
    args = _extract_args(plan, latent, pos, tile_lat, tile_pos, tile_index, tile_count, cond_row, cond_k)
    args.append(_stream_handle(stream, latent.device))
    _check(load_library().tdp_extract_noalloc(*args))


def tdp_blend(plan: Plan, tile_out, cond_row, cond_k, out, stream=None):
    """Enqueue the blend of tile outputs into ``out`` on ``stream``
    (``cond_row`` and ``cond_k`` from tdp_extract; ignored when Nc == 0)."""
    import torch
    c = plan.cfg
    s = tdp_plan_sizes(plan)
    dev = tile_out.device
    none = ctypes.c_void_p(None)
    args = [
        plan.handle,
        _ptr(tile_out, "tile_out", _torch_dtype(c.in_dtype), s.tile_lat_elems, dev),
        _ptr(cond_row, "cond_row", torch.int32, s.cond_row_ints, dev) if c.num_cond else none,
        _ptr(cond_k, "cond_k", torch.int32, s.cond_k_ints, dev) if c.num_cond else none,
        _ptr(out, "out", _torch_dtype(c.out_dtype), s.out_elems, dev),
        _stream_handle(stream, dev),
    ]
    _check(load_library().tdp_blend(*args))


def tdp_pipeline_step(plan: Plan, latent, pos, tile_lat, tile_pos, tile_index, tile_count, cond_row=None,
                      cond_k=None, workspace=None, *, tile_out, blend_cond_row=None, blend_cond_k=None, out,
                      stream=None):
    """Enqueue tdp_extract of ``latent`` and tdp_blend of ``tile_out`` (an
    earlier latent's tile outputs, none of this extract's buffers) as one
    step, one launch where the plan allows."""
    import torch
    c = plan.cfg
    s = tdp_plan_sizes(plan)
    dev = latent.device
    none = ctypes.c_void_p(None)
    args = _extract_args(plan, latent, pos, tile_lat, tile_pos, tile_index, tile_count, cond_row, cond_k)
    args.append(_ptr(workspace, "workspace", torch.uint8, s.workspace_bytes, dev) if s.workspace_bytes else none)
    args += [
        _ptr(tile_out, "tile_out", _torch_dtype(c.in_dtype), s.tile_lat_elems, dev),
        _ptr(blend_cond_row, "blend_cond_row", torch.int32, s.cond_row_ints, dev) if c.num_cond else none,
        _ptr(blend_cond_k, "blend_cond_k", torch.int32, s.cond_k_ints, dev) if c.num_cond else none,
        _ptr(out, "out", _torch_dtype(c.out_dtype), s.out_elems, dev),
        _stream_handle(stream, dev),
    ]
    _check(load_library().tdp_pipeline_step(*args))


def tdp_extract_positions(plan: Plan, pos, tile_pos, tile_index, tile_count, cond_row=None, cond_k=None,
                          workspace=None, stream=None):
    """Enqueue what tdp_extract writes except the latent rows (tile positions,
    index map, counts, cond_row, cond_k): once per positions set."""
    import torch
    c = plan.cfg
    s = tdp_plan_sizes(plan)
    rows = plan.tokens + c.num_cond
    dev = pos.device
    none = ctypes.c_void_p(None)
    args = [
        plan.handle,
        _ptr(pos, "pos", torch.float32, c.batch * 3 * rows * 2, dev),
        _ptr(tile_pos, "tile_pos", torch.float32, s.tile_pos_floats, dev),
        _ptr(tile_index, "tile_index", torch.int32, s.tile_index_ints, dev),
        _ptr(tile_count, "tile_count", torch.int32, s.num_slots, dev),
        _ptr(cond_row, "cond_row", torch.int32, s.cond_row_ints, dev) if c.num_cond else none,
        _ptr(cond_k, "cond_k", torch.int32, s.cond_k_ints, dev) if c.num_cond else none,
        _ptr(workspace, "workspace", torch.uint8, s.workspace_bytes, dev) if s.workspace_bytes else none,
        _stream_handle(stream, dev),
    ]
    _check(load_library().tdp_extract_positions(*args))


def _gather_args(plan: Plan, latent, cond_row, tile_lat):
    import torch
    c = plan.cfg
    s = tdp_plan_sizes(plan)
    rows = plan.tokens + c.num_cond
    dev = latent.device
    return [
        plan.handle,
        _ptr(latent, "latent", _torch_dtype(c.in_dtype), c.batch * rows * c.channels, dev),
        _ptr(cond_row, "cond_row", torch.int32, s.cond_row_ints, dev) if c.num_cond else ctypes.c_void_p(None),
        _ptr(tile_lat, "tile_lat", _torch_dtype(c.in_dtype), s.tile_lat_elems, dev),
    ]


def tdp_extract_latent(plan: Plan, latent, cond_row, tile_lat, stream=None):
    """Enqueue the latent rows of every held tile into ``tile_lat``, at the
    slot rows ``cond_row`` (from tdp_extract_positions) gives."""
    args = _gather_args(plan, latent, cond_row, tile_lat)
    args.append(_stream_handle(stream, latent.device))
    _check(load_library().tdp_extract_latent(*args))


def tdp_pipeline_latent_step(plan: Plan, latent, cond_row, tile_lat, *, tile_out, blend_cond_row=None,
                             blend_cond_k=None, out, stream=None):
    """Enqueue tdp_extract_latent of ``latent`` and tdp_blend of ``tile_out``
    as one step (one launch for whole plans)."""
    import torch
    c = plan.cfg
    s = tdp_plan_sizes(plan)
    dev = latent.device
    none = ctypes.c_void_p(None)
    args = _gather_args(plan, latent, cond_row, tile_lat)
    args += [
        _ptr(tile_out, "tile_out", _torch_dtype(c.in_dtype), s.tile_lat_elems, dev),
        _ptr(blend_cond_row, "blend_cond_row", torch.int32, s.cond_row_ints, dev) if c.num_cond else none,
        _ptr(blend_cond_k, "blend_cond_k", torch.int32, s.cond_k_ints, dev) if c.num_cond else none,
        _ptr(out, "out", _torch_dtype(c.out_dtype), s.out_elems, dev),
        _stream_handle(stream, dev),
    ]
    _check(load_library().tdp_pipeline_latent_step(*args))


def allocate_accumulator(plan: Plan, device="cuda"):
    """fp32 (B, N+Nc, C) accumulator for the streaming blend."""
    import torch
    c = plan.cfg
    return torch.empty((c.batch, plan.tokens + c.num_cond, c.channels), dtype=torch.float32,
                       device=torch.device(device))


def tdp_blend_tile(plan: Plan, t: int, tile_out, cond_row, cond_k, acc, stream=None):
    """Enqueue the streaming blend of tile t's slot ``tile_out`` into ``acc``."""
    import torch
    c = plan.cfg
    info = tdp_plan_tile(plan, t)
    dev = acc.device
    rows = plan.tokens + c.num_cond
    none = ctypes.c_void_p(None)
    _check(load_library().tdp_blend_tile(
        plan.handle, t,
        _ptr(tile_out, "tile_out", _torch_dtype(c.in_dtype), c.batch * info.capacity * c.channels, dev),
        _ptr(cond_row, "cond_row", torch.int32, c.num_cond * tdp_plan_num_tiles(plan), dev) if c.num_cond else none,
        _ptr(cond_k, "cond_k", torch.int32, c.num_cond, dev) if c.num_cond else none,
        _ptr(acc, "acc", torch.float32, c.batch * rows * c.channels, dev),
        _stream_handle(stream, dev)))


def tdp_blend_finish(plan: Plan, acc, out, stream=None):
    """Enqueue the rounding of ``acc`` to the output dtype into ``out``."""
    import torch
    c = plan.cfg
    n = c.batch * (plan.tokens + c.num_cond) * c.channels
    dev = acc.device
    _check(load_library().tdp_blend_finish(plan.handle, _ptr(acc, "acc", torch.float32, n, dev),
                                           _ptr(out, "out", _torch_dtype(c.out_dtype), n, dev),
                                           _stream_handle(stream, dev)))


def tile_views(plan: Plan, buffers, counts=None):
    """Per-slot torch views into the tile-major buffers (every tile, or a
    rank plan's own tiles in slot order).

    ``counts`` (host list of tile_count) trims each view to its used rows;
    without it the views span the whole slot.  Returns a list of dicts with
    ``lat`` (B, rows, C), ``pos`` (B, 3, rows, 2), ``index`` (rows,) and
    ``info`` (its ``index`` is the tile).
    """
    c = plan.cfg
    views = []
    for j, t in enumerate(held_tiles(plan)):
        info = tdp_plan_tile(plan, t)
        cap = info.capacity
        used = cap if counts is None else int(counts[j])
        lat = buffers["tile_lat"][info.lat_offset: info.lat_offset + c.batch * cap * c.channels]
        pos = buffers["tile_pos"][info.pos_offset: info.pos_offset + c.batch * 6 * cap]
        idx = buffers["tile_index"][info.index_offset: info.index_offset + cap]
        views.append({
            "lat": lat.view(c.batch, cap, c.channels)[:, :used],
            "pos": pos.view(c.batch, 3, cap, 2)[:, :, :used],
            "index": idx[:used],
            "info": info,
        })
    return views


# ---------------------------------------------------------------------------
# Spatial blend of decoded pixel tiles
# ---------------------------------------------------------------------------

def make_pixel_config(batch, channels, frames, latent_hw, scale_hw, tiling_hw, in_dtype="bf16",
                      out_dtype=None) -> tdp_pixel_config:
    """Fill a tdp_pixel_config; ``tiling_hw`` = ((n_h, o_h), (n_w, o_w)) in latent cells."""
    cfg = tdp_pixel_config()
    cfg.batch, cfg.channels, cfg.frames = batch, channels, frames
    cfg.height, cfg.width = latent_hw
    for a in range(2):
        cfg.scale[a] = scale_hw[a]
        cfg.axis[a].num_tiles, cfg.axis[a].overlap = tiling_hw[a]
    code = lambda d: _DTYPES[d] if isinstance(d, str) else d  # noqa: E731
    cfg.in_dtype = code(in_dtype)
    cfg.out_dtype = code(in_dtype if out_dtype is None else out_dtype)
    return cfg


class PixelPlan:
    """Owning handle of a tdp_pixel_plan."""

    def __init__(self, handle, cfg):
        self.handle, self.cfg = handle, cfg

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.tdp_pixel_plan_destroy(self.handle)
            self.handle = None


def tdp_pixel_plan_create(cfg: tdp_pixel_config) -> PixelPlan:
    h = ctypes.c_void_p()
    _check(load_library().tdp_pixel_plan_create(ctypes.byref(cfg), ctypes.byref(h)))
    return PixelPlan(h, cfg)


def tdp_pixel_plan_tile(plan: PixelPlan, t: int) -> tdp_pixel_tile:
    info = tdp_pixel_tile()
    _check(load_library().tdp_pixel_plan_tile(plan.handle, t, ctypes.byref(info)))
    return info


def tdp_pixel_plan_sizes(plan: PixelPlan):
    """(tile buffer elements, output elements, tile count)."""
    a, b, n = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
    _check(load_library().tdp_pixel_plan_sizes(plan.handle, ctypes.byref(a), ctypes.byref(b), ctypes.byref(n)))
    return a.value, b.value, n.value


def tdp_pixel_blend(plan: PixelPlan, tiles, out, stream=None):
    """Enqueue the blend of packed pixel tiles into ``out`` (B, C, frames, H*s_h, W*s_w)."""
    c = plan.cfg
    tile_elems, out_elems, _ = tdp_pixel_plan_sizes(plan)
    dev = out.device
    _check(load_library().tdp_pixel_blend(plan.handle, _ptr(tiles, "tiles", _torch_dtype(c.in_dtype), tile_elems, dev),
                                          _ptr(out, "out", _torch_dtype(c.out_dtype), out_elems, dev),
                                          _stream_handle(stream, dev)))


# ---------------------------------------------------------------------------
# The tile's attention: rotation, norms, attention and their gradients
#
# Like the rest of this module the calls write into the caller's tensors through
# their addresses.  Autograd sees none of it, also for tensors that require
# gradients: a program calls the backward entry points itself (as
# examples/tile_attention.py does) or wraps the pairs in functions of its own.
# ---------------------------------------------------------------------------

class Sequences:
    """How the rows of (rows, heads, head_dim) tensors fall into sequences.

    ``num_seqs`` sequences of ``max_rows`` rows each, one after another; or
    sequence s owns rows [row_start[s], row_start[s + 1]) (``row_start``: S + 1
    int64, ascending) or row_range[s] (``row_range``: (S, 2) int64), none longer
    than ``max_rows``.  ``seq_len`` (int32) holds the used rows, entry
    s // len_group.  The tensors live on the GPU and are kept alive here;
    ``row_start`` is turned into ranges on the current stream.
    """

    def __init__(self, num_seqs, max_rows, row_start=None, row_range=None, total_rows=None, seq_len=None,
                 len_group=1):
        import torch
        if row_start is not None:
            if row_range is not None:
                raise ValueError("row_start and row_range are two forms of the same: give one")
            if row_start.numel() != num_seqs + 1:
                raise ValueError(f"row_start holds {row_start.numel()} entries, needs {num_seqs + 1}")
            row_range = torch.stack([row_start[:-1], row_start[1:]], dim=1)
        if row_range is None:
            rows = num_seqs * max_rows
            if total_rows not in (None, rows):
                raise ValueError(f"{num_seqs} sequences of {max_rows} rows span {rows} rows, not {total_rows}")
            total_rows = rows
        elif total_rows is None:
            raise ValueError("total_rows is required with row_start or row_range")
        if len_group < 1:
            raise ValueError("len_group must be >= 1")
        s = tdp_seqs()
        s.num_seqs, s.max_rows, s.total_rows, s.len_group = num_seqs, max_rows, total_rows, len_group
        dev = None
        if row_range is not None:
            row_range = row_range.contiguous()
            s.row_range = _ptr(row_range, "row_range", torch.int64, 2 * num_seqs, None)
            dev = row_range.device
        if seq_len is not None:
            s.seq_len = _ptr(seq_len, "seq_len", torch.int32, (num_seqs + len_group - 1) // len_group, dev)
            dev = seq_len.device
        self.c, self.device = s, dev
        self.num_seqs, self.max_rows, self.total_rows = num_seqs, max_rows, total_rows
        self._keep = (row_range, seq_len)
        self._layouts = {}


def tdp_plan_sequences(plan: Plan) -> list[tuple[int, int]]:
    """[start, end) rows of tile_lat per sequence: slot by slot, batch element by batch element."""
    n = tdp_plan_sizes(plan).num_slots * plan.cfg.batch
    buf = (ctypes.c_int64 * max(1, 2 * n))()
    _check(load_library().tdp_plan_sequences(plan.handle, buf))
    return [(buf[2 * i], buf[2 * i + 1]) for i in range(n)]


def plan_sequences(plan: Plan, tile_count=None, device="cuda") -> Sequences:
    """The Sequences of a plan's slots; ``tile_count`` (tdp_extract's) gives the
    used rows, otherwise every row of a slot counts as used."""
    import torch
    ranges = tdp_plan_sequences(plan)
    if not ranges:
        raise ValueError("the plan holds no tiles")
    rows = tdp_plan_sizes(plan).tile_pos_floats // 6
    return Sequences(len(ranges), max(b - a for a, b in ranges),
                     row_range=torch.tensor(ranges, dtype=torch.int64, device=torch.device(device)),
                     total_rows=rows, seq_len=tile_count, len_group=plan.cfg.batch)


class RopeConfig:
    """tdp_rope_config with its frequencies (see make_rope_config)."""

    def __init__(self, cfg: tdp_rope_config, freqs):
        self.cfg, self.freqs = cfg, freqs


def make_rope_config(head_dim, rot_dims, theta=10000.0, scale=(1.0, 1.0, 1.0), freqs=None, pairing="interleaved",
                     point="middle") -> RopeConfig:
    """Fill a tdp_rope_config.  ``rot_dims``: dims turned by (time, height, width).
    Pair i of an axis turns by scale * theta ** (-2 i / rot_dim) radians per
    position unit, or by freqs[axis][i]."""
    cfg = tdp_rope_config()
    cfg.head_dim = head_dim
    for a in range(3):
        cfg.rot_dim[a] = rot_dims[a]
    cfg.pairing = {"interleaved": TDP_PAIR_INTERLEAVED, "halves": TDP_PAIR_HALVES}.get(pairing, pairing)
    cfg.point = {"middle": TDP_POINT_MIDDLE, "start": TDP_POINT_START}.get(point, point)
    if freqs is None:
        freqs = [[scale[a] * theta ** (-2.0 * i / r) for i in range(r // 2)] for a, r in enumerate(rot_dims)]
    for a in range(3):
        if len(freqs[a]) != max(rot_dims[a], 0) // 2:
            raise ValueError(f"axis {a}: {len(freqs[a])} frequencies for {rot_dims[a]} dims")
    return RopeConfig(cfg, [float(f) for axis in freqs for f in axis])


class Rope:
    """Owns a tdp_rope handle (host memory only)."""

    def __init__(self, handle: int, cfg: tdp_rope_config):
        self.handle, self.cfg = ctypes.c_void_p(handle), cfg

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.tdp_rope_destroy(self.handle)
            self.handle = None


def tdp_rope_create(config: RopeConfig) -> Rope:
    h = ctypes.c_void_p()
    freqs = (ctypes.c_double * max(1, len(config.freqs)))(*config.freqs)
    _check(load_library().tdp_rope_create(ctypes.byref(config.cfg), freqs, ctypes.byref(h)))
    return Rope(h.value, config.cfg)


def _dtype_code(t, name):
    import torch
    if t.dtype == torch.bfloat16:
        return TDP_BF16
    if t.dtype == torch.float32:
        return TDP_F32
    raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")


def _layout(t, name, seqs: Sequences, head_dim, written):
    """(seq, row, head strides, heads) of a (total_rows, heads, head_dim) tensor, or of a
    (num_seqs, max_rows, heads, head_dim) one for uniform sequences, after checking it."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 4 and not seqs.c.row_range:
        if shape[0] != seqs.num_seqs or shape[1] != seqs.max_rows:
            raise ValueError(f"{name} is {tuple(shape)}, needs ({seqs.num_seqs}, {seqs.max_rows}, heads, {head_dim})")
        seq_stride, row_stride, head_stride = stride[:3]
    elif len(shape) == 3:
        if shape[0] != seqs.total_rows:
            raise ValueError(f"{name} holds {shape[0]} rows, needs {seqs.total_rows}")
        row_stride, head_stride = stride[:2]
        seq_stride = seqs.max_rows * row_stride
    else:
        raise ValueError(f"{name} must be (rows, heads, head_dim), or (sequences, rows, heads, head_dim) without row "
                         f"ranges; got {tuple(shape)}")
    if shape[-1] != head_dim or stride[-1] != 1:
        raise ValueError(f"{name} needs {head_dim} contiguous elements per head, got {tuple(shape)} with strides "
                         f"{stride}")
    if written:   # every element its own place
        reach = 1
        for st, n in sorted((st, n) for st, n in zip(stride, shape) if n > 1):
            if st < reach:
                raise ValueError(f"{name} is written and must not overlap itself (strides {stride})")
            reach = st * (n - 1) + reach
    # a dimension of one element is never stepped over: torch may report any stride for it
    heads, rows = shape[-2], shape[-3]
    if len(shape) == 4 and shape[0] == 1 or seqs.num_seqs == 1:
        seq_stride = 0
    return seq_stride, row_stride if rows > 1 else 0, head_stride if heads > 1 else 0, heads


def _heads(t, name, seqs: Sequences, head_dim, like, written=False):
    """tdp_heads of a tensor after checking it against ``like``'s device and dtype."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t is not like:
        if t.device != like.device:
            raise ValueError(f"{name} must be on {like.device}, got {t.device}")
        if t.dtype != like.dtype:
            raise ValueError(f"{name} must be {like.dtype}, got {t.dtype}")
    elif not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if seqs.device is not None and seqs.device != t.device:
        raise ValueError(f"{name} is on {t.device}, its sequences on {seqs.device}")
    key = (t.shape, t.stride(), head_dim, written)
    lay = seqs._layouts.get(key)   # layouts of these sequences checked before, whatever tensor had them
    if lay is None:
        lay = _layout(t, name, seqs, head_dim, written)
        if len(seqs._layouts) < 64:
            seqs._layouts[key] = lay
    return tdp_heads(t.data_ptr(), *lay)


def _on(device, call, *args):
    """A library call with `device` current, as its launches need."""
    import torch
    if device.index is None or device.index == torch.cuda.current_device():
        return _check(call(*args))
    with torch.cuda.device(device):
        return _check(call(*args))


def _vec(t, name, dtype, numel, device):
    return ctypes.c_void_p(None) if t is None else _ptr(t, name, dtype, numel, device)


def _pos_ptr(rope: Rope, seqs: Sequences, pos, device):
    import torch
    if not any(rope.cfg.rot_dim):
        return ctypes.c_void_p(None)
    return _ptr(pos, "pos", torch.float32, 6 * seqs.total_rows, device)


def tdp_rope_apply(rope: Rope, seqs: Sequences, pos, x, y, inverse=False, stream=None):
    """Enqueue y = x turned by the positions ``pos`` (tile_pos, or (S, 3, rows, 2));
    ``inverse`` turns back, which is also the gradient.  y may be x."""
    ref = ctypes.byref
    D = rope.cfg.head_dim
    _on(x.device, load_library().tdp_rope_apply,
        rope.handle, ref(seqs.c), _pos_ptr(rope, seqs, pos, x.device), ref(_heads(x, "x", seqs, D, x)),
        ref(_heads(y, "y", seqs, D, x, True)), _dtype_code(x, "x"), int(bool(inverse)),
        _stream_handle(stream, x.device))


def tdp_qk_norm_rope(rope: Rope, seqs: Sequences, pos, q, k, q_weight, k_weight, q_out, k_out, eps=1e-6, stream=None):
    """Enqueue the norm of every query and key head (times fp32 weights, None: ones) and its rotation."""
    import torch
    ref, D, dev = ctypes.byref, rope.cfg.head_dim, q.device
    _on(dev, load_library().tdp_qk_norm_rope,
        rope.handle, ref(seqs.c), _pos_ptr(rope, seqs, pos, dev), ref(_heads(q, "q", seqs, D, q)),
        ref(_heads(k, "k", seqs, D, q)), _vec(q_weight, "q_weight", torch.float32, D, dev),
        _vec(k_weight, "k_weight", torch.float32, D, dev), ref(_heads(q_out, "q_out", seqs, D, q, True)),
        ref(_heads(k_out, "k_out", seqs, D, q, True)), eps, _dtype_code(q, "q"), _stream_handle(stream, dev))


def allocate_qk_norm_rope_workspace(rope: Rope, seqs: Sequences, q_heads: int, k_heads: int, device="cuda"):
    import torch
    n = load_library().tdp_qk_norm_rope_workspace(rope.handle, ctypes.byref(seqs.c), q_heads, k_heads)
    if n <= 0:
        raise TdpError(TDP_EINVAL, tdp_last_error())
    return torch.empty(n, dtype=torch.uint8, device=torch.device(device))


def tdp_qk_norm_rope_backward(rope: Rope, seqs: Sequences, pos, q, k, q_weight, k_weight, dq_out, dk_out, dq, dk,
                              dq_weight, dk_weight, workspace, eps=1e-6, stream=None):
    """Enqueue the gradients of tdp_qk_norm_rope (dq may be dq_out, dk may be dk_out)."""
    import torch
    ref, D, dev = ctypes.byref, rope.cfg.head_dim, q.device
    sq, sk = _heads(q, "q", seqs, D, q), _heads(k, "k", seqs, D, q)
    need = load_library().tdp_qk_norm_rope_workspace(rope.handle, ref(seqs.c), sq.heads, sk.heads)
    _on(dev, load_library().tdp_qk_norm_rope_backward,
        rope.handle, ref(seqs.c), _pos_ptr(rope, seqs, pos, dev), ref(sq), ref(sk),
        _vec(q_weight, "q_weight", torch.float32, D, dev), _vec(k_weight, "k_weight", torch.float32, D, dev),
        ref(_heads(dq_out, "dq_out", seqs, D, q)), ref(_heads(dk_out, "dk_out", seqs, D, q)),
        ref(_heads(dq, "dq", seqs, D, q, True)), ref(_heads(dk, "dk", seqs, D, q, True)),
        _vec(dq_weight, "dq_weight", torch.float32, D, dev), _vec(dk_weight, "dk_weight", torch.float32, D, dev),
        eps, _dtype_code(q, "q"), _ptr(workspace, "workspace", torch.uint8, need, dev), _stream_handle(stream, dev))


def allocate_attention_workspace(q_seqs: Sequences, k_seqs: Sequences, q_heads: int, k_heads: int, head_dim: int,
                                 device="cuda"):
    """Workspace of tdp_attention, or None where it needs none."""
    import torch
    n = load_library().tdp_attention_workspace(ctypes.byref(q_seqs.c), ctypes.byref(k_seqs.c), q_heads, k_heads,
                                               head_dim)
    return torch.empty(n, dtype=torch.uint8, device=torch.device(device)) if n else None


def allocate_attention_backward_workspace(q_seqs: Sequences, k_seqs: Sequences, q_heads: int, k_heads: int,
                                          head_dim: int, device="cuda"):
    import torch
    n = load_library().tdp_attention_backward_workspace(ctypes.byref(q_seqs.c), ctypes.byref(k_seqs.c), q_heads,
                                                        k_heads, head_dim)
    if n <= 0:
        raise TdpError(TDP_EINVAL, tdp_last_error())
    return torch.empty(n, dtype=torch.uint8, device=torch.device(device))


def tdp_attention(q_seqs: Sequences, k_seqs: Sequences, q, k, v, out, lse=None, key_bias=None, scale=None,
                  workspace=None, stream=None):
    """Enqueue attention of each sequence's queries over its keys (scale: 1 / sqrt(head_dim)
    by default).  ``lse`` (heads, rows) fp32 is wanted by the backward."""
    import torch
    ref, D, dev = ctypes.byref, q.shape[-1], q.device
    sq, sk = _heads(q, "q", q_seqs, D, q), _heads(k, "k", k_seqs, D, q)
    need = load_library().tdp_attention_workspace(ref(q_seqs.c), ref(k_seqs.c), sq.heads, sk.heads, D)
    _on(dev, load_library().tdp_attention,
        ref(q_seqs.c), ref(k_seqs.c), ref(sq), ref(sk), ref(_heads(v, "v", k_seqs, D, q)),
        _vec(key_bias, "key_bias", torch.float32, k_seqs.total_rows, dev),
        ref(_heads(out, "out", q_seqs, D, q, True)),
        _vec(lse, "lse", torch.float32, sq.heads * q_seqs.total_rows, dev), D ** -0.5 if scale is None else scale, D,
        _dtype_code(q, "q"), _ptr(workspace, "workspace", torch.uint8, need, dev) if need else ctypes.c_void_p(None),
        _stream_handle(stream, dev))


def tdp_attention_backward(q_seqs: Sequences, k_seqs: Sequences, q, k, v, out, lse, dout, dq, dk, dv, workspace,
                           key_bias=None, scale=None, stream=None):
    """Enqueue the gradients of tdp_attention; ``out`` and ``lse`` are its results."""
    import torch
    ref, D, dev = ctypes.byref, q.shape[-1], q.device
    sq, sk = _heads(q, "q", q_seqs, D, q), _heads(k, "k", k_seqs, D, q)
    need = load_library().tdp_attention_backward_workspace(ref(q_seqs.c), ref(k_seqs.c), sq.heads, sk.heads, D)
    _on(dev, load_library().tdp_attention_backward,
        ref(q_seqs.c), ref(k_seqs.c), ref(sq), ref(sk), ref(_heads(v, "v", k_seqs, D, q)),
        _vec(key_bias, "key_bias", torch.float32, k_seqs.total_rows, dev), ref(_heads(out, "out", q_seqs, D, q)),
        _ptr(lse, "lse", torch.float32, sq.heads * q_seqs.total_rows, dev),
        ref(_heads(dout, "dout", q_seqs, D, q)), ref(_heads(dq, "dq", q_seqs, D, q, True)),
        ref(_heads(dk, "dk", k_seqs, D, q, True)), ref(_heads(dv, "dv", k_seqs, D, q, True)),
        D ** -0.5 if scale is None else scale, D, _dtype_code(q, "q"),
        _ptr(workspace, "workspace", torch.uint8, need, dev), _stream_handle(stream, dev))


def make_window(step=1, back=None, ahead=0, sinks=0) -> tdp_window:
    """A window over steps of ``step`` rows: ``back`` earlier and ``ahead`` later steps in view
    (None: all of them), the first ``sinks`` rows always."""
    every = lambda n: TDP_WINDOW_ALL if n is None else n  # noqa: E731
    return tdp_window(step, every(back), every(ahead), sinks)


def allocate_window_attention_workspace(q_seqs: Sequences, k_seqs: Sequences, window: tdp_window, q_heads: int,
                                        k_heads: int, head_dim: int, device="cuda"):
    """Workspace of tdp_window_attention, or None where it needs none."""
    import torch
    n = load_library().tdp_window_attention_workspace(ctypes.byref(q_seqs.c), ctypes.byref(k_seqs.c),
                                                      ctypes.byref(window), q_heads, k_heads, head_dim)
    return torch.empty(n, dtype=torch.uint8, device=torch.device(device)) if n else None


def allocate_window_attention_backward_workspace(q_seqs: Sequences, k_seqs: Sequences, window: tdp_window,
                                                 q_heads: int, k_heads: int, head_dim: int, device="cuda"):
    import torch
    n = load_library().tdp_window_attention_backward_workspace(
        ctypes.byref(q_seqs.c), ctypes.byref(k_seqs.c), ctypes.byref(window), q_heads, k_heads, head_dim)
    if n <= 0:
        raise TdpError(TDP_EINVAL, tdp_last_error())
    return torch.empty(n, dtype=torch.uint8, device=torch.device(device))


def tdp_window_attention(q_seqs: Sequences, k_seqs: Sequences, window: tdp_window, q, k, v, out, lse=None, scale=None,
                         workspace=None, stream=None):
    """Enqueue attention within a window (scale: 1 / sqrt(head_dim) by default); the queries are
    the newest rows of each sequence.  ``lse`` (heads, rows) fp32 is wanted by the backward."""
    import torch
    lib, ref, D, dev = load_library(), ctypes.byref, q.shape[-1], q.device
    sq, sk = _heads(q, "q", q_seqs, D, q), _heads(k, "k", k_seqs, D, q)
    need = lib.tdp_window_attention_workspace(ref(q_seqs.c), ref(k_seqs.c), ref(window), sq.heads, sk.heads, D)
    _on(dev, lib.tdp_window_attention, ref(q_seqs.c), ref(k_seqs.c), ref(window), ref(sq), ref(sk),
        ref(_heads(v, "v", k_seqs, D, q)), ref(_heads(out, "out", q_seqs, D, q, True)),
        _vec(lse, "lse", torch.float32, sq.heads * q_seqs.total_rows, dev), D ** -0.5 if scale is None else scale, D,
        _dtype_code(q, "q"), _ptr(workspace, "workspace", torch.uint8, need, dev) if need else ctypes.c_void_p(None),
        _stream_handle(stream, dev))


def tdp_window_attention_backward(q_seqs: Sequences, k_seqs: Sequences, window: tdp_window, q, k, v, out, lse, dout,
                                  dq, dk, dv, workspace, scale=None, stream=None):
    """Enqueue the gradients of tdp_window_attention; ``out`` and ``lse`` are its results."""
    import torch
    lib, ref, D, dev = load_library(), ctypes.byref, q.shape[-1], q.device
    sq, sk = _heads(q, "q", q_seqs, D, q), _heads(k, "k", k_seqs, D, q)
    need = lib.tdp_window_attention_backward_workspace(ref(q_seqs.c), ref(k_seqs.c), ref(window), sq.heads, sk.heads,
                                                       D)
    _on(dev, lib.tdp_window_attention_backward, ref(q_seqs.c), ref(k_seqs.c), ref(window), ref(sq), ref(sk),
        ref(_heads(v, "v", k_seqs, D, q)), ref(_heads(out, "out", q_seqs, D, q)),
        _ptr(lse, "lse", torch.float32, sq.heads * q_seqs.total_rows, dev),
        ref(_heads(dout, "dout", q_seqs, D, q)), ref(_heads(dq, "dq", q_seqs, D, q, True)),
        ref(_heads(dk, "dk", k_seqs, D, q, True)), ref(_heads(dv, "dv", k_seqs, D, q, True)),
        D ** -0.5 if scale is None else scale, D, _dtype_code(q, "q"),
        _ptr(workspace, "workspace", torch.uint8, need, dev), _stream_handle(stream, dev))


# ---------------------------------------------------------------------------
# The layer around the attention: layer norm and grouped products
# ---------------------------------------------------------------------------

def _rows_layout(t, name, seqs: Sequences, features, written):
    """(seq, row strides) of a (total_rows, features) tensor, or of a (num_seqs, max_rows,
    features) one for uniform sequences, after checking it."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3 and not seqs.c.row_range:
        if shape[0] != seqs.num_seqs or shape[1] != seqs.max_rows:
            raise ValueError(f"{name} is {tuple(shape)}, needs ({seqs.num_seqs}, {seqs.max_rows}, {features})")
        seq_stride, row_stride = stride[:2]
    elif len(shape) == 2:
        if shape[0] != seqs.total_rows:
            raise ValueError(f"{name} holds {shape[0]} rows, needs {seqs.total_rows}")
        row_stride = stride[0]
        seq_stride = seqs.max_rows * row_stride
    else:
        raise ValueError(f"{name} must be (rows, features), or (sequences, rows, features) without row ranges; got "
                         f"{tuple(shape)}")
    if shape[-1] != features or stride[-1] != 1:
        raise ValueError(f"{name} needs {features} contiguous elements per row, got {tuple(shape)} with strides "
                         f"{stride}")
    if written:   # every element its own place
        reach = 1
        for st, n in sorted((st, n) for st, n in zip(stride, shape) if n > 1):
            if st < reach:
                raise ValueError(f"{name} is written and must not overlap itself (strides {stride})")
            reach = st * (n - 1) + reach
    if seqs.num_seqs == 1:
        seq_stride = 0
    return seq_stride, row_stride if shape[-2] > 1 else 0


def _rows(t, name, seqs: Sequences, features, like, written=False):
    """tdp_rows of a tensor after checking it against ``like``'s device and dtype."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t is not like:
        if t.device != like.device:
            raise ValueError(f"{name} must be on {like.device}, got {t.device}")
        if t.dtype != like.dtype:
            raise ValueError(f"{name} must be {like.dtype}, got {t.dtype}")
    elif not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if seqs.device is not None and seqs.device != t.device:
        raise ValueError(f"{name} is on {t.device}, its sequences on {seqs.device}")
    key = (t.shape, t.stride(), features, written, "rows")
    lay = seqs._layouts.get(key)
    if lay is None:
        lay = _rows_layout(t, name, seqs, features, written)
        if len(seqs._layouts) < 64:
            seqs._layouts[key] = lay
    return tdp_rows(t.data_ptr(), *lay)


def _weight_sets(t, name, channels, sets, device):
    """Pointer of (channels) or (sets, channels) fp32 weights (None: null)."""
    import torch
    if t is None:
        return ctypes.c_void_p(None)
    if tuple(t.shape) not in ((sets, channels),) + (((channels,),) if sets == 1 else ()):
        raise ValueError(f"{name} is {tuple(t.shape)}, needs ({sets}, {channels})")
    return _ptr(t, name, torch.float32, sets * channels, device)


def _num_sets(*ts):
    """Weight rows of the first tensor given: 1 for a vector."""
    for t in ts:
        if t is not None:
            return t.shape[0] if t.dim() == 2 else 1
    return 1


def tdp_layer_norm(seqs: Sequences, x, weight, bias, y, eps=1e-5, stream=None):
    """Enqueue the layer norm of every used row.  ``weight`` and ``bias``: (channels) fp32 for
    all, or (n, channels), of which sequence s takes row s mod n (None: ones, zeros).  y may be x."""
    ref, C, dev, n = ctypes.byref, x.shape[-1], x.device, _num_sets(weight, bias)
    _on(dev, load_library().tdp_layer_norm, ref(seqs.c), ref(_rows(x, "x", seqs, C, x)),
        _weight_sets(weight, "weight", C, n, dev), _weight_sets(bias, "bias", C, n, dev), n,
        ref(_rows(y, "y", seqs, C, x, True)), eps, C, _dtype_code(x, "x"), _stream_handle(stream, dev))


def allocate_layer_norm_workspace(seqs: Sequences, channels: int, num_weights: int = 1, device="cuda"):
    import torch
    n = load_library().tdp_layer_norm_workspace(ctypes.byref(seqs.c), channels, num_weights)
    if n <= 0:
        raise TdpError(TDP_EINVAL, tdp_last_error())
    return torch.empty(n, dtype=torch.uint8, device=torch.device(device))


def tdp_layer_norm_backward(seqs: Sequences, x, weight, dy, dx, dweight, dbias, workspace, eps=1e-5, stream=None):
    """Enqueue the gradients of tdp_layer_norm (dx may be dy or x; dweight, dbias None: not wanted)."""
    import torch
    ref, C, dev, n = ctypes.byref, x.shape[-1], x.device, _num_sets(weight, dweight, dbias)
    need = load_library().tdp_layer_norm_workspace(ref(seqs.c), C, n)
    _on(dev, load_library().tdp_layer_norm_backward, ref(seqs.c), ref(_rows(x, "x", seqs, C, x)),
        _weight_sets(weight, "weight", C, n, dev), n, ref(_rows(dy, "dy", seqs, C, x)),
        ref(_rows(dx, "dx", seqs, C, x, True)), _weight_sets(dweight, "dweight", C, n, dev),
        _weight_sets(dbias, "dbias", C, n, dev), eps, C, _dtype_code(x, "x"),
        _ptr(workspace, "workspace", torch.uint8, need, dev), _stream_handle(stream, dev))


def _product_weight(t, name, dtype, device, shape=None):
    """(pointer, (weights, out features, in features)) of an (out, in) or (weights, out, in) tensor."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be (out features, in features) or (weights, out features, in features), got "
                         f"{tuple(t.shape)}")
    own = tuple(t.shape) if t.dim() == 3 else (1, *t.shape)
    if shape is not None and own != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, needs {shape}")
    return _ptr(t, name, dtype, t.numel(), device), own


def allocate_grouped_product_workspace(seqs: Sequences, num_weights: int, out_features: int, in_features: int,
                                       dtype="bf16", device="cuda"):
    """Workspace of tdp_grouped_product, or None where it needs none."""
    import torch
    n = load_library().tdp_grouped_product_workspace(ctypes.byref(seqs.c), num_weights, in_features, out_features,
                                                     _product_dtype(dtype))
    return torch.empty(n, dtype=torch.uint8, device=torch.device(device)) if n else None


def allocate_grouped_product_backward_workspace(seqs: Sequences, num_weights: int, out_features: int,
                                                in_features: int, dtype="bf16", device="cuda"):
    """Workspace of tdp_grouped_product_backward, or None where it needs none."""
    import torch
    n = load_library().tdp_grouped_product_backward_workspace(ctypes.byref(seqs.c), num_weights, in_features,
                                                              out_features, _product_dtype(dtype))
    return torch.empty(n, dtype=torch.uint8, device=torch.device(device)) if n else None


def _product_dtype(dtype) -> int:
    import torch
    code = {torch.float32: TDP_F32, torch.bfloat16: TDP_BF16}.get(dtype, dtype)
    return _DTYPES[code] if isinstance(code, str) else code


def tdp_grouped_product(seqs: Sequences, x, weight, y, workspace=None, stream=None):
    """Enqueue y = x W^T for every used row: ``weight`` (out, in) for all, or (n, out, in), of which
    the rows of sequence s take weight s mod n (experts: a sequence each)."""
    import torch
    lib, ref, dev = load_library(), ctypes.byref, x.device
    code = _dtype_code(x, "x")
    w, (n, N, K) = _product_weight(weight, "weight", x.dtype, dev)
    need = lib.tdp_grouped_product_workspace(ref(seqs.c), n, K, N, code)
    _on(dev, lib.tdp_grouped_product, ref(seqs.c), ref(_rows(x, "x", seqs, K, x)), w, n,
        ref(_rows(y, "y", seqs, N, x, True)), K, N, code,
        _ptr(workspace, "workspace", torch.uint8, need, dev) if need else ctypes.c_void_p(None),
        _stream_handle(stream, dev))


def tdp_grouped_product_backward(seqs: Sequences, x, weight, dy, dx, dweight, workspace=None, stream=None):
    """Enqueue the gradients of tdp_grouped_product: ``dx`` like x, ``dweight`` like weight in fp32
    (either None: not wanted)."""
    import torch
    lib, ref, dev = load_library(), ctypes.byref, x.device
    code = _dtype_code(x, "x")
    w, shape = _product_weight(weight, "weight", x.dtype, dev)
    n, N, K = shape
    need = lib.tdp_grouped_product_backward_workspace(ref(seqs.c), n, K, N, code)
    _on(dev, lib.tdp_grouped_product_backward, ref(seqs.c), ref(_rows(x, "x", seqs, K, x)), w, n,
        ref(_rows(dy, "dy", seqs, N, x)), None if dx is None else ref(_rows(dx, "dx", seqs, K, x, True)),
        ctypes.c_void_p(None) if dweight is None else _product_weight(dweight, "dweight", torch.float32, dev, shape)[0],
        K, N, code, _ptr(workspace, "workspace", torch.uint8, need, dev) if need else ctypes.c_void_p(None),
        _stream_handle(stream, dev))
