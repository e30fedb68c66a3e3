"""ctypes binding of the C ABI in include/gemm.h, gemm_moe.h and gemm_scaled.h.

Argument marshalling only: every step of the product runs in the CUDA
library.  The functions keep the C names; a non-OK status raises GemmError.
Device operands may be given as integers (device addresses) or as objects
with a ``data_ptr()`` method (torch tensors); streams as integers or objects
with a ``cuda_stream`` attribute.
"""
from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpsm_gemm.so")

GEMM_F16, GEMM_BF16 = 0, 1
GEMM_ROW_MAJOR, GEMM_COL_MAJOR = 0, 1
GEMM_SCHED_DATA_PARALLEL, GEMM_SCHED_PERSISTENT, GEMM_SCHED_STREAMK, GEMM_SCHED_SPLITK = 0, 1, 2, 3
GEMM_SCHED_AUTO = 4
SCHEDULES = {"dp": 0, "persistent": 1, "streamk": 2, "splitk": 3, "auto": 4}

(GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_UNSUPPORTED, GEMM_ERR_WORKSPACE, GEMM_ERR_CUDA,
 GEMM_ERR_LAUNCH, GEMM_ERR_TIMEOUT, GEMM_ERR_NO_DEVICE) = range(8)

GEMM_OPT_GRID = 1
GEMM_OPT_GROUP_M = 2
GEMM_OPT_TILE_N = 3
GEMM_OPT_TWO_TILES = 4
GEMM_OPT_WAIT_LIMIT_US = 5
GEMM_OPT_INJECT_SKIP_POST = 6
GEMM_OPT_CLUSTER_M = 7
GEMM_OPT_SK_MODE = 8
GEMM_OPT_SPLIT_K = 9
GEMM_OPT_K_ROTATE = 10
GEMM_OPT_L2_PREFETCH = 11
GEMM_OPT_PAIR_MMA = 12
GEMM_OPT_RASTER = 13
GEMM_OPT_HOST_CHUNKS = 14
GEMM_OPT_HOST_COL_CHUNKS = 15
GEMM_OPT_SPLIT_K_CLUSTER = 16
GEMM_OPT_EARLY_PREFETCH = 17

INFO = {
    "tile_m": 1, "tile_n": 2, "tile_k": 3, "tiles_m": 4, "tiles_n": 5, "tiles": 6,
    "iters_per_tile": 7, "grid": 8, "sk_tiles": 9, "sk_iters_per_cta": 10,
    "sk_iters_rem": 11, "num_sms": 12, "stages": 13, "group_m": 14, "smem_bytes": 15, "cluster_m": 16,
    "a_rows_per_stage": 17, "split_k": 18, "k_rotate": 19,
    "l2_prefetch": 20, "pair_mma": 21, "schedule": 22, "sk_mode": 23, "raster": 24, "host_chunks": 25, "host_col_chunks": 26,
    "split_k_cluster": 27, "clusters_resident": 28, "early_prefetch": 29,
}
GEMM_INDEX_I32, GEMM_INDEX_I64 = 0, 1
GEMM_GROUPED_ROWS, GEMM_GROUPED_INNER = 0, 1
GEMM_MOE_MAX_EXPERTS = 1024
GEMM_GROUPED_OPT_CTAS, GEMM_GROUPED_OPT_INJECT_GIVE_UP = 1, 3
GROUPED_INFO = {"ctas": 1, "units": 2, "tile_m": 3, "tile_n": 4, "stages": 5, "smem_bytes": 6, "groups": 7}

GEMM_E4M3, GEMM_E5M2 = 0, 1
GEMM_F32 = 2                       # an output type of scaled products only
GEMM_SCALE_VECTOR, GEMM_SCALE_BLOCK = 0, 1
GEMM_SCALE_GROUP = 128
GEMM_QUANTIZE_ROWS, GEMM_QUANTIZE_COLS, GEMM_QUANTIZE_BLOCKS = 0, 1, 2
GEMM_NORM_MAX_HIDDEN = 32768
GEMM_SCALED_STRAIGHT, GEMM_SCALED_TURNED, GEMM_SCALED_FEW = 0, 1, 2
GEMM_SCALED_OPT_CTAS, GEMM_SCALED_OPT_FORM, GEMM_SCALED_OPT_INJECT_GIVE_UP = 1, 2, 3
SCALED_INFO = {"ctas": 1, "form": 2, "units": 3, "tiles": 4, "tile_width": 5, "shares": 6}

ROLE_FULL, ROLE_OWNER, ROLE_PEER, ROLE_CLUSTER_PART = 0, 1, 2, 3
TRACE_STAMPS = 6   # uint64 per CTA written by gemm_plan_set_trace: 4 timer + 2 clock stamps

# every entry point of the headers: name -> (restype, argtypes)
_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
_f32 = ctypes.c_float
_pp = ctypes.POINTER(ctypes.c_void_p)
SIGNATURES = {
    "gemm_plan_create": (_i32, [_pp, _i64, _i64, _i64, _i32, _i32, _i32, _i32]),
    "gemm_plan_create_offline": (_i32, [_pp, _i64, _i64, _i64, _i32, _i32, _i32, _i32, _i32]),
    "gemm_plan_set_option": (_i32, [_vp, _i32, _i64]),
    "gemm_plan_get_info": (_i32, [_vp, _i32, ctypes.POINTER(_i64)]),
    "gemm_workspace_size": (_i32, [_vp, ctypes.POINTER(ctypes.c_size_t)]),
    "gemm_run": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp]),
    "gemm_run_host": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "gemm_last_status": (_i32, [_vp, _vp]),
    "gemm_run_no_alloc": (_i32, [_vp, _vp, _vp, _vp, _vp]),
    "gemm_plan_units": (_i32, [_vp, _i64, ctypes.POINTER(ctypes.c_int32), _i64,
                               ctypes.POINTER(_i64)]),
    "gemm_plan_tile_coords": (_i32, [_vp, _i64, ctypes.POINTER(_i64), ctypes.POINTER(_i64)]),
    "gemm_plan_set_trace": (_i32, [_vp, _vp, ctypes.c_size_t]),
    "gemm_plan_destroy": (_i32, [_vp]),
    "gemm_status_string": (ctypes.c_char_p, [_i32]),
    "gemm_moe_sort_workspace_size": (_i32, [_i64, _i64, _i64, ctypes.POINTER(ctypes.c_size_t)]),
    "gemm_moe_sort": (_i32, [_vp, _i32, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "gemm_moe_dispatch": (_i32, [_vp, _i64, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _i64, _vp]),
    "gemm_moe_dispatch_grad": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _i32, _vp, _i64, _vp]),
    "gemm_moe_combine": (_i32, [_vp, _i64, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _i64, _vp]),
    "gemm_moe_combine_grad": (_i32, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i32,
                                     _vp, _i64, _vp, _vp]),
    "gemm_grouped_plan_create": (_i32, [_pp, _i32, _i64, _i64, _i64, _i64, _i32, _i32]),
    "gemm_grouped_plan_create_offline": (_i32, [_pp, _i32, _i64, _i64, _i64, _i64, _i32, _i32, _i32]),
    "gemm_grouped_plan_set_option": (_i32, [_vp, _i32, _i64]),
    "gemm_grouped_plan_get_info": (_i32, [_vp, _i32, ctypes.POINTER(_i64)]),
    "gemm_grouped_plan_units": (_i32, [_vp, ctypes.POINTER(ctypes.c_int32), _i64,
                                       ctypes.POINTER(ctypes.c_int32), _i64, ctypes.POINTER(_i64)]),
    "gemm_grouped_workspace_size": (_i32, [_vp, ctypes.POINTER(ctypes.c_size_t)]),
    "gemm_grouped_run": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "gemm_grouped_last_status": (_i32, [_vp, _vp]),
    "gemm_grouped_plan_destroy": (_i32, [_vp]),
    "gemm_scaled_quantize": (_i32, [_i32, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _i64, _vp, _vp]),
    "gemm_scaled_quantize_both": (_i32, [_vp, _i64, _i64, _i64, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _vp, _vp]),
    "gemm_rms_norm": (_i32, [_vp, _i64, _vp, _i64, _vp, _f32, _i64, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _i32,
                             _vp, _vp, _vp]),
    "gemm_rms_norm_grad_workspace_size": (_i32, [_i64, _i64, ctypes.POINTER(ctypes.c_size_t)]),
    "gemm_rms_norm_grad": (_i32, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _vp]),
    "gemm_scaled_plan_create": (_i32, [_pp, _i64, _i64, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "gemm_scaled_plan_create_offline": (_i32, [_pp, _i64, _i64, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "gemm_scaled_plan_set_option": (_i32, [_vp, _i32, _i64]),
    "gemm_scaled_plan_get_info": (_i32, [_vp, _i32, ctypes.POINTER(_i64)]),
    "gemm_scaled_workspace_size": (_i32, [_vp, ctypes.POINTER(ctypes.c_size_t)]),
    "gemm_scaled_run": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "gemm_scaled_last_status": (_i32, [_vp, _vp]),
    "gemm_scaled_plan_destroy": (_i32, [_vp]),
}

_lib = None
_packed = None  # psm_packed_call: its arguments as one array, a slot of 64 bits each


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__("%s: %s" % (where, gemm_status_string(status)))


def load(path: str = LIB_PATH):
    """Load the CUDA library; raise if it is missing (there is no fallback)."""
    global _lib, _packed
    if _lib is None:
        if not os.path.exists(path):
            raise ImportError(
                "libpsm_gemm.so is not built (%s); run persistent_stream_matmul_gb300.build.build()"
                % path)
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _packed = lib.psm_packed_call
        _packed.restype, _packed.argtypes = _i32, [_i32, ctypes.c_char_p]
        _lib = lib
    return _lib


def _addr(x) -> int | None:
    if x is None or type(x) is int:
        return x
    try:
        return x.data_ptr()
    except AttributeError:
        if isinstance(x, int):
            return x
        raise  # ctypes would take bytes and str as host pointers


def _stream(s) -> int | None:
    if s is None or type(s) is int:
        return s
    try:
        return s.cuda_stream
    except AttributeError:
        if isinstance(s, int):
            return s
        raise


def _check(st: int, where: str):
    if st != GEMM_OK:
        raise GemmError(st, where)


def gemm_status_string(status: int) -> str:
    return load().gemm_status_string(int(status)).decode()


def gemm_plan_create(M, N, K, dtype, layout_a, layout_b, schedule) -> int:
    h = ctypes.c_void_p()
    _check(load().gemm_plan_create(ctypes.byref(h), M, N, K, dtype, layout_a, layout_b, schedule),
           "gemm_plan_create")
    return h.value


def gemm_plan_create_offline(M, N, K, dtype, layout_a, layout_b, schedule, num_sms) -> int:
    h = ctypes.c_void_p()
    _check(load().gemm_plan_create_offline(ctypes.byref(h), M, N, K, dtype, layout_a, layout_b,
                                           schedule, num_sms), "gemm_plan_create_offline")
    return h.value


def gemm_plan_set_option(plan, key, value):
    _check(load().gemm_plan_set_option(plan, key, value), "gemm_plan_set_option")


def gemm_plan_get_info(plan, key) -> int:
    v = ctypes.c_int64()
    key = INFO[key] if isinstance(key, str) else key
    _check(load().gemm_plan_get_info(plan, key, ctypes.byref(v)), "gemm_plan_get_info")
    return v.value


def gemm_workspace_size(plan) -> int:
    v = ctypes.c_size_t()
    _check(load().gemm_workspace_size(plan, ctypes.byref(v)), "gemm_workspace_size")
    return v.value


def gemm_run(plan, A, B, C, workspace=None, stream=None):
    _check(load().gemm_run(plan, _addr(A), _addr(B), _addr(C), _addr(workspace), _stream(stream)),
           "gemm_run")


def gemm_run_host(plan, hA, hB, hC, dA, dB, dC, workspace=None, stream=None):
    _check(load().gemm_run_host(plan, _addr(hA), _addr(hB), _addr(hC), _addr(dA), _addr(dB),
                                _addr(dC), _addr(workspace), _stream(stream)), "gemm_run_host")


def gemm_run_no_alloc(plan, A, B, C, stream=None):
    """gemm_run without a workspace argument: the library's fixed scratch array
    is used instead, so nothing is allocated (for callers that cannot allocate)."""
    _check(load().gemm_run_no_alloc(plan, _addr(A), _addr(B), _addr(C), _stream(stream)),
           "gemm_run_no_alloc")


GEMM_NO_ALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def gemm_last_status(plan, stream=None) -> int:
    """Returns the status code (GEMM_OK or GEMM_ERR_TIMEOUT ...); does not raise."""
    return int(load().gemm_last_status(plan, _stream(stream)))


def gemm_plan_units(plan, cta: int):
    """[(tile, k0, k1, role, npeers), ...] of CTA ``cta``."""
    n = ctypes.c_int64()
    _check(load().gemm_plan_units(plan, cta, None, 0, ctypes.byref(n)), "gemm_plan_units")
    buf = (ctypes.c_int32 * (5 * max(n.value, 1)))()
    _check(load().gemm_plan_units(plan, cta, buf, n.value, ctypes.byref(n)), "gemm_plan_units")
    return [tuple(buf[5 * i:5 * i + 5]) for i in range(n.value)]


def gemm_plan_tile_coords(plan, tile: int):
    tm, tn = ctypes.c_int64(), ctypes.c_int64()
    _check(load().gemm_plan_tile_coords(plan, tile, ctypes.byref(tm), ctypes.byref(tn)),
           "gemm_plan_tile_coords")
    return tm.value, tn.value


def gemm_plan_set_trace(plan, device_buffer, nbytes: int):
    """Per-CTA stamps into a device buffer: %globaltimer at start, ready,
    loads done and end, then %clock64 at start and end (TRACE_STAMPS each)."""
    _check(load().gemm_plan_set_trace(plan, _addr(device_buffer), nbytes), "gemm_plan_set_trace")


def gemm_plan_destroy(plan):
    _check(load().gemm_plan_destroy(plan), "gemm_plan_destroy")


class Plan:
    """Owning wrapper around a plan handle (marshalling only)."""

    def __init__(self, M, N, K, dtype, layout_a, layout_b, schedule, offline_sms=None,
                 **options):
        if isinstance(schedule, str):
            schedule = SCHEDULES[schedule]
        self.M, self.N, self.K = M, N, K
        self.dtype, self.layout_a, self.layout_b, self.schedule = dtype, layout_a, layout_b, schedule
        if offline_sms is None:
            self.handle = gemm_plan_create(M, N, K, dtype, layout_a, layout_b, schedule)
        else:
            self.handle = gemm_plan_create_offline(M, N, K, dtype, layout_a, layout_b, schedule,
                                                   offline_sms)
        keys = {"grid": GEMM_OPT_GRID, "group_m": GEMM_OPT_GROUP_M, "tile_n": GEMM_OPT_TILE_N,
                "two_tiles": GEMM_OPT_TWO_TILES, "wait_limit_us": GEMM_OPT_WAIT_LIMIT_US,
                "inject_skip_post": GEMM_OPT_INJECT_SKIP_POST, "cluster_m": GEMM_OPT_CLUSTER_M,
                "sk_mode": GEMM_OPT_SK_MODE, "split_k": GEMM_OPT_SPLIT_K,
                "k_rotate": GEMM_OPT_K_ROTATE, "l2_prefetch": GEMM_OPT_L2_PREFETCH,
                "pair_mma": GEMM_OPT_PAIR_MMA, "raster": GEMM_OPT_RASTER,
                "host_chunks": GEMM_OPT_HOST_CHUNKS, "host_col_chunks": GEMM_OPT_HOST_COL_CHUNKS,
                "split_cluster": GEMM_OPT_SPLIT_K_CLUSTER, "early_prefetch": GEMM_OPT_EARLY_PREFETCH}
        for k, v in options.items():
            if v is not None:
                gemm_plan_set_option(self.handle, keys[k], int(v))

    def info(self, key):
        return gemm_plan_get_info(self.handle, key)

    def set_option(self, key, value):
        gemm_plan_set_option(self.handle, key, value)

    @property
    def workspace_size(self) -> int:
        return gemm_workspace_size(self.handle)

    def units(self, cta):
        return gemm_plan_units(self.handle, cta)

    def tile_coords(self, tile):
        return gemm_plan_tile_coords(self.handle, tile)

    def run(self, A, B, C, workspace=None, stream=None):
        gemm_run(self.handle, A, B, C, workspace, stream)

    def run_host(self, hA, hB, hC, dA, dB, dC, workspace=None, stream=None):
        gemm_run_host(self.handle, hA, hB, hC, dA, dB, dC, workspace, stream)

    def set_trace(self, device_buffer, nbytes):
        gemm_plan_set_trace(self.handle, device_buffer, nbytes)

    def last_status(self, stream=None) -> int:
        return gemm_last_status(self.handle, stream)

    def close(self):
        if getattr(self, "handle", None):
            gemm_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def gemm_moe_sort_workspace_size(tokens, topk, experts) -> int:
    v = ctypes.c_size_t()
    _check(load().gemm_moe_sort_workspace_size(tokens, topk, experts, ctypes.byref(v)),
           "gemm_moe_sort_workspace_size")
    return v.value


def gemm_moe_sort(ids, id_type, ld_ids, tokens, topk, experts, offsets, rows, slots, workspace=None,
                  stream=None):
    _check(load().gemm_moe_sort(_addr(ids), id_type, ld_ids, tokens, topk, experts, _addr(offsets),
                                _addr(rows), _addr(slots), _addr(workspace), _stream(stream)),
           "gemm_moe_sort")


def gemm_moe_dispatch(x, ldx, rows, slots, tokens, topk, hidden, dtype, xs, ldxs, stream=None):
    _check(load().gemm_moe_dispatch(_addr(x), ldx, _addr(rows), _addr(slots), tokens, topk, hidden,
                                    dtype, _addr(xs), ldxs, _stream(stream)), "gemm_moe_dispatch")


def gemm_moe_dispatch_grad(dxs, lddxs, rows, tokens, topk, hidden, dtype, dx, lddx, stream=None):
    _check(load().gemm_moe_dispatch_grad(_addr(dxs), lddxs, _addr(rows), tokens, topk, hidden, dtype,
                                         _addr(dx), lddx, _stream(stream)), "gemm_moe_dispatch_grad")


def gemm_moe_combine(ys, ldys, rows, weights, tokens, topk, hidden, dtype, y, ldy, stream=None):
    _check(load().gemm_moe_combine(_addr(ys), ldys, _addr(rows), _addr(weights), tokens, topk, hidden,
                                   dtype, _addr(y), ldy, _stream(stream)), "gemm_moe_combine")


def gemm_moe_combine_grad(dy, lddy, ys, ldys, rows, slots, weights, tokens, topk, hidden, dtype, dys,
                          lddys, dweights, stream=None):
    _check(load().gemm_moe_combine_grad(_addr(dy), lddy, _addr(ys), ldys, _addr(rows), _addr(slots),
                                        _addr(weights), tokens, topk, hidden, dtype, _addr(dys), lddys,
                                        _addr(dweights), _stream(stream)), "gemm_moe_combine_grad")


def gemm_grouped_plan_create(kind, groups, rows, N, K, dtype, layout_b) -> int:
    h = ctypes.c_void_p()
    _check(load().gemm_grouped_plan_create(ctypes.byref(h), kind, groups, rows, N, K, dtype, layout_b),
           "gemm_grouped_plan_create")
    return h.value


def gemm_grouped_plan_create_offline(kind, groups, rows, N, K, dtype, layout_b, num_sms) -> int:
    h = ctypes.c_void_p()
    _check(load().gemm_grouped_plan_create_offline(ctypes.byref(h), kind, groups, rows, N, K, dtype,
                                                   layout_b, num_sms),
           "gemm_grouped_plan_create_offline")
    return h.value


def gemm_grouped_plan_set_option(plan, key, value):
    _check(load().gemm_grouped_plan_set_option(plan, key, value), "gemm_grouped_plan_set_option")


def gemm_grouped_plan_get_info(plan, key) -> int:
    v = ctypes.c_int64()
    key = GROUPED_INFO[key] if isinstance(key, str) else key
    _check(load().gemm_grouped_plan_get_info(plan, key, ctypes.byref(v)), "gemm_grouped_plan_get_info")
    return v.value


def gemm_grouped_plan_units(plan, offsets, unit: int):
    """[(tile, group, tile along C's rows, first row, rows, width, k0, k1, k-blocks), ...] of
    scheduling unit ``unit`` for host offsets, one more than the plan has groups."""
    if len(offsets) != gemm_grouped_plan_get_info(plan, "groups") + 1:
        raise ValueError("gemm_grouped_plan_units: %d offsets for %d groups"
                         % (len(offsets), gemm_grouped_plan_get_info(plan, "groups")))
    off = (ctypes.c_int32 * len(offsets))(*[int(x) for x in offsets])
    n = ctypes.c_int64()
    _check(load().gemm_grouped_plan_units(plan, off, unit, None, 0, ctypes.byref(n)),
           "gemm_grouped_plan_units")
    buf = (ctypes.c_int32 * (9 * max(n.value, 1)))()
    _check(load().gemm_grouped_plan_units(plan, off, unit, buf, n.value, ctypes.byref(n)),
           "gemm_grouped_plan_units")
    return [tuple(buf[9 * i:9 * i + 9]) for i in range(n.value)]


def gemm_grouped_workspace_size(plan) -> int:
    v = ctypes.c_size_t()
    _check(load().gemm_grouped_workspace_size(plan, ctypes.byref(v)), "gemm_grouped_workspace_size")
    return v.value


def gemm_grouped_run(plan, A, B, C, offsets, workspace=None, stream=None):
    _check(load().gemm_grouped_run(plan, _addr(A), _addr(B), _addr(C), _addr(offsets),
                                   _addr(workspace), _stream(stream)), "gemm_grouped_run")


def gemm_grouped_last_status(plan, stream=None) -> int:
    """Returns the status code (GEMM_OK or GEMM_ERR_TIMEOUT ...); does not raise."""
    return int(load().gemm_grouped_last_status(plan, _stream(stream)))


def gemm_grouped_plan_destroy(plan):
    _check(load().gemm_grouped_plan_destroy(plan), "gemm_grouped_plan_destroy")


class GroupedPlan:
    """Owning wrapper around a grouped plan handle (marshalling only)."""

    def __init__(self, kind, groups, rows, N, K, dtype, layout_b, offline_sms=None, ctas=None):
        self.kind, self.groups, self.rows, self.N, self.K = kind, groups, rows, N, K
        self.dtype, self.layout_b = dtype, layout_b
        if offline_sms is None:
            self.handle = gemm_grouped_plan_create(kind, groups, rows, N, K, dtype, layout_b)
        else:
            self.handle = gemm_grouped_plan_create_offline(kind, groups, rows, N, K, dtype, layout_b,
                                                           offline_sms)
        if ctas is not None:
            self.set_option(GEMM_GROUPED_OPT_CTAS, int(ctas))

    def info(self, key):
        return gemm_grouped_plan_get_info(self.handle, key)

    def set_option(self, key, value):
        gemm_grouped_plan_set_option(self.handle, key, value)

    def units(self, offsets, unit):
        return gemm_grouped_plan_units(self.handle, offsets, unit)

    @property
    def workspace_size(self) -> int:
        return gemm_grouped_workspace_size(self.handle)

    def run(self, A, B, C, offsets, workspace=None, stream=None):
        gemm_grouped_run(self.handle, A, B, C, offsets, workspace, stream)

    def last_status(self, stream=None) -> int:
        return gemm_grouped_last_status(self.handle, stream)

    def close(self):
        if getattr(self, "handle", None):
            gemm_grouped_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


# The row operators' and the scaled products' calls are short and have many
# arguments, which ctypes would convert one by one.
_PACK_QUANTIZE, _PACK_BOTH = struct.Struct("11q").pack, struct.Struct("13q").pack
_PACK_NORM, _PACK_NORM_GRAD, _PACK_RUN = struct.Struct("5qd13q").pack, struct.Struct("16q").pack, struct.Struct("8q").pack


def _call(op, packed, where):
    st = (_packed or _loaded())(op, packed)
    if st != GEMM_OK:
        raise GemmError(st, where)


def _loaded():
    load()
    return _packed


def gemm_scaled_quantize(kind, x, ldx, rows, cols, dtype, type, q, ldq, scales, stream=None):
    _call(0, _PACK_QUANTIZE(kind, _addr(x) or 0, ldx, rows, cols, dtype, type, _addr(q) or 0, ldq, _addr(scales) or 0,
                            _stream(stream) or 0), "gemm_scaled_quantize")


def gemm_scaled_quantize_both(x, ldx, rows, cols, dtype, type, q_rows, ldq_rows, scales_rows, q_cols, ldq_cols,
                              scales_cols, stream=None):
    _call(1, _PACK_BOTH(_addr(x) or 0, ldx, rows, cols, dtype, type, _addr(q_rows) or 0, ldq_rows, _addr(scales_rows) or 0,
                        _addr(q_cols) or 0, ldq_cols, _addr(scales_cols) or 0, _stream(stream) or 0),
          "gemm_scaled_quantize_both")


def gemm_rms_norm(x, ldx, residual, ldres, weight, eps, rows, hidden, dtype, sum, ldsum, y, ldy, q, ldq, type, scales,
                  rstd, stream=None):
    _call(2, _PACK_NORM(_addr(x) or 0, ldx, _addr(residual) or 0, ldres, _addr(weight) or 0, eps, rows, hidden, dtype,
                        _addr(sum) or 0, ldsum, _addr(y) or 0, ldy, _addr(q) or 0, ldq, type, _addr(scales) or 0,
                        _addr(rstd) or 0, _stream(stream) or 0), "gemm_rms_norm")


def gemm_rms_norm_grad_workspace_size(rows, hidden) -> int:
    v = ctypes.c_size_t()
    _check(load().gemm_rms_norm_grad_workspace_size(rows, hidden, ctypes.byref(v)),
           "gemm_rms_norm_grad_workspace_size")
    return v.value


def gemm_rms_norm_grad(dy, lddy, s, lds, weight, rstd, dsum, lddsum, rows, hidden, dtype, dx, lddx, dweight,
                       workspace=None, stream=None):
    _call(3, _PACK_NORM_GRAD(_addr(dy) or 0, lddy, _addr(s) or 0, lds, _addr(weight) or 0, _addr(rstd) or 0,
                             _addr(dsum) or 0, lddsum, rows, hidden, dtype, _addr(dx) or 0, lddx, _addr(dweight) or 0,
                             _addr(workspace) or 0, _stream(stream) or 0), "gemm_rms_norm_grad")


def gemm_scaled_plan_create(M, N, K, type_a, type_b, out_dtype, layout_a, layout_b, scale_a, scale_b) -> int:
    h = ctypes.c_void_p()
    _check(load().gemm_scaled_plan_create(ctypes.byref(h), M, N, K, type_a, type_b, out_dtype, layout_a, layout_b,
                                          scale_a, scale_b), "gemm_scaled_plan_create")
    return h.value


def gemm_scaled_plan_create_offline(M, N, K, type_a, type_b, out_dtype, layout_a, layout_b, scale_a, scale_b,
                                    num_sms) -> int:
    h = ctypes.c_void_p()
    _check(load().gemm_scaled_plan_create_offline(ctypes.byref(h), M, N, K, type_a, type_b, out_dtype, layout_a,
                                                  layout_b, scale_a, scale_b, num_sms),
           "gemm_scaled_plan_create_offline")
    return h.value


def gemm_scaled_plan_set_option(plan, key, value):
    _check(load().gemm_scaled_plan_set_option(plan, key, value), "gemm_scaled_plan_set_option")


def gemm_scaled_plan_get_info(plan, key) -> int:
    v = ctypes.c_int64()
    key = SCALED_INFO[key] if isinstance(key, str) else key
    _check(load().gemm_scaled_plan_get_info(plan, key, ctypes.byref(v)), "gemm_scaled_plan_get_info")
    return v.value


def gemm_scaled_workspace_size(plan) -> int:
    v = ctypes.c_size_t()
    _check(load().gemm_scaled_workspace_size(plan, ctypes.byref(v)), "gemm_scaled_workspace_size")
    return v.value


def gemm_scaled_run(plan, A, scales_a, B, scales_b, C, workspace=None, stream=None):
    _call(4, _PACK_RUN(plan or 0, _addr(A) or 0, _addr(scales_a) or 0, _addr(B) or 0, _addr(scales_b) or 0,
                       _addr(C) or 0, _addr(workspace) or 0, _stream(stream) or 0), "gemm_scaled_run")


def gemm_scaled_last_status(plan, stream=None) -> int:
    """Returns the status code (GEMM_OK or GEMM_ERR_TIMEOUT ...); does not raise."""
    return int(load().gemm_scaled_last_status(plan, _stream(stream)))


def gemm_scaled_plan_destroy(plan):
    _check(load().gemm_scaled_plan_destroy(plan), "gemm_scaled_plan_destroy")


class ScaledPlan:
    """Owning wrapper around a scaled plan handle (marshalling only)."""

    def __init__(self, M, N, K, type_a, type_b, out_dtype, layout_a, layout_b, scale_a, scale_b, offline_sms=None,
                 ctas=None, form=None):
        self.M, self.N, self.K = M, N, K
        self.out_dtype = out_dtype
        args = (M, N, K, type_a, type_b, out_dtype, layout_a, layout_b, scale_a, scale_b)
        self.handle = (gemm_scaled_plan_create(*args) if offline_sms is None
                       else gemm_scaled_plan_create_offline(*args, offline_sms))
        if form is not None:
            self.set_option(GEMM_SCALED_OPT_FORM, int(form))
        if ctas is not None:
            self.set_option(GEMM_SCALED_OPT_CTAS, int(ctas))

    def info(self, key):
        return gemm_scaled_plan_get_info(self.handle, key)

    def set_option(self, key, value):
        gemm_scaled_plan_set_option(self.handle, key, value)

    @property
    def workspace_size(self) -> int:
        return gemm_scaled_workspace_size(self.handle)

    def run(self, A, scales_a, B, scales_b, C, workspace=None, stream=None):
        gemm_scaled_run(self.handle, A, scales_a, B, scales_b, C, workspace, stream)

    def last_status(self, stream=None) -> int:
        return gemm_scaled_last_status(self.handle, stream)

    def close(self):
        if getattr(self, "handle", None):
            gemm_scaled_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
