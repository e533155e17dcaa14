"""ctypes view of libchunkkv.so (the C-ABI declared in include/chunkkv.h)."""
from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libchunkkv.so")

MAX_BATCH = 1024
MAX_GATHER_LAYERS = 64
Q8_PAGE = 64                                   # CHUNKKV_Q8_PAGE
PROBE_THREADS, PROBE_CHAINS = 256, 16          # CHUNKKV_PROBE_THREADS, CHUNKKV_PROBE_CHAINS

STATUS = {
    0: "CHUNKKV_OK",
    1: "CHUNKKV_ERR_INVALID_ARG",
    2: "CHUNKKV_ERR_UNSUPPORTED",
    3: "CHUNKKV_ERR_WORKSPACE_TOO_SMALL",
    4: "CHUNKKV_ERR_CUDA",
    5: "CHUNKKV_ERR_TIMEOUT",
}
F32, BF16 = 0, 1


class Params(ctypes.Structure):
    """chunkkv_params."""
    _fields_ = [
        ("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
        ("w", ctypes.c_int32), ("c", ctypes.c_int32), ("L_max", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("cu_seqlens", ctypes.POINTER(ctypes.c_int32)),
        ("q_stride_b", ctypes.c_int64), ("q_stride_w", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("kv_stride_t", ctypes.c_int64), ("kv_stride_h", ctypes.c_int64),
        ("causal_window", ctypes.c_int32),
    ]


class PrefillParams(ctypes.Structure):
    """chunkkv_prefill_params."""
    _fields_ = [
        ("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
        ("cu_q", ctypes.POINTER(ctypes.c_int32)), ("cu_k", ctypes.POINTER(ctypes.c_int32)),
        ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("kv_stride_t", ctypes.c_int64), ("kv_stride_h", ctypes.c_int64),
        ("o_stride_t", ctypes.c_int64), ("o_stride_h", ctypes.c_int64),
    ]


class Q8CacheStruct(ctypes.Structure):
    """chunkkv_q8_cache."""
    _fields_ = [
        ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
        ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("ring", ctypes.c_void_p), ("state", ctypes.c_void_p),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
                          f"g.build()'` (the library has no non-CUDA fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(Params)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    pp = ctypes.POINTER(ctypes.c_void_p)
    i64 = ctypes.c_int64
    PP, Q8 = ctypes.POINTER(PrefillParams), ctypes.POINTER(Q8CacheStruct)
    sigs = {
        "chunkkv_out_capacity": [P, ctypes.POINTER(i32), ctypes.POINTER(i32)],
        "chunkkv_workspace_size": [P, i32, i32, ctypes.POINTER(sz)],
        "chunkkv_score": [P, vp, vp, vp, vp, sz, vp],
        "chunkkv_select": [P, vp, vp, vp, vp],
        "chunkkv_gather": [P, i32, vp, vp, pp, pp, pp, pp, vp],
        "chunkkv_compress_layers": [P, i32, i32, pp, pp, pp, pp, pp, vp, vp, vp, vp, sz, vp],
        "chunkkv_tail_sizes": [P, ctypes.POINTER(i32), i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32),
                               ctypes.POINTER(sz)],
        "chunkkv_compress_tail": [P, ctypes.POINTER(i32), i32, i32, pp, pp, pp, pp, pp, vp, vp, vp, vp, sz, vp],
        "chunkkv_status_check": [vp, vp, ctypes.POINTER(i32)],
        "chunkkv_score_path": [P],
        "chunkkv_score_noalloc": [P, vp, vp, vp, vp],
        "chunkkv_set_phase_events": [pp, i32],
        "chunkkv_selftest_wait_timeout": [vp, sz, vp],
        "chunkkv_layer_overlap": [P, i32, vp, vp, vp, vp, vp],
        "chunkkv_probe_ex2": [vp, i32, i32, vp],
        "chunkkv_prefill_workspace_size": [PP, ctypes.POINTER(sz)],
        "chunkkv_prefill_path": [PP],
        "chunkkv_prefill_attention": [PP, vp, vp, vp, vp, vp, sz, vp],
        "chunkkv_q8_resize": [Q8, vp, vp, i32, vp],
        "chunkkv_q8_append": [Q8, i32, vp, vp, i64, i64, i64, vp, vp, i32, vp],
        "chunkkv_q8_load": [Q8, i32, vp, i32, vp, vp, i64, vp],
        "chunkkv_q8_load_bounded": [Q8, i32, vp, i32, i64, vp, vp, i64, vp],
        "chunkkv_q8_workspace_size": [Q8, i32, ctypes.POINTER(sz)],
        "chunkkv_q8_attention": [Q8, i32, i32, ctypes.c_float, vp, i64, i64, vp, i64, i64, vp, sz, vp],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int32
    lib.chunkkv_status_string.argtypes = [ctypes.c_int32]
    lib.chunkkv_status_string.restype = ctypes.c_char_p
    lib.chunkkv_launch_count.argtypes = []
    lib.chunkkv_launch_count.restype = ctypes.c_uint64
    return lib


LIB = _load()
