"""ctypes loader for libsolattn.so (the C ABI of include/solattn.h)."""
from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsolattn.so")

# Every symbol declared in include/solattn.h.
EXPORTS = (
    "solattn_pooled_layout",
    "solattn_pool",
    "solattn_forward",
    "solattn_dense",
    "solattn_status",
    "solattn_strerror",
    "solattn_version",
    "solattn_forward_noalloc",
    "solattn_forward_ex",
    "solattn_pool_ex",
    "solattn_noalloc_status",
    "solattn_host_scratch_bytes",
    "solattn_forward_host",
    "solattn_rotary_frequencies",
    "solattn_rotary",
    "solattn_rotary_pool",
    "solattn_cache_append",
    "solattn_cache_workspace_bytes",
    "solattn_cache_attention",
)

OK = 0
ERR_ARG = 1
ERR_UNSUPPORTED = 2
ERR_ALIGN = 3
ERR_CUDA = 4
ERR_TIMEOUT = 5
ERR_DEVICE = 6
ERR_WORKSPACE = 7
ERR_SCRATCH = 8
ERR_PAGE = 9
WORKSPACE_BYTES = 256
NOALLOC_SCRATCH_BYTES = 16 << 20
BLOCK = 64
MAX_TOKENS = 262144
RULE_THRESHOLD, RULE_TOPK, RULE_TOPP = 0, 1, 2
BF16, F16, F32 = 0, 1, 2
ROTARY_INTERLEAVED, ROTARY_HALF = 0, 1
ROTARY_MAX_AXES = 4
SCALING_NONE, SCALING_LINEAR, SCALING_NTK, SCALING_YARN = 0, 1, 2, 3


class PooledStruct(ctypes.Structure):
    """Mirror of solattn_pooled_t."""

    _fields_ = [(name, ctypes.c_void_p) for name in ("qbar", "kbar", "vbar", "kmean", "kcov", "kbar16", "vbar16")]


class StridesStruct(ctypes.Structure):
    """Mirror of solattn_strides_t."""

    _fields_ = [("batch", ctypes.c_longlong), ("head", ctypes.c_longlong), ("token", ctypes.c_longlong)]


class OptionsStruct(ctypes.Structure):
    """Mirror of solattn_options_t."""

    _fields_ = [("rule", ctypes.c_int), ("beta", ctypes.c_float), ("topk", ctypes.c_int), ("topp", ctypes.c_float),
                ("n_forced", ctypes.c_int), ("strides", StridesStruct), ("correction", ctypes.c_int)]


class RotaryStruct(ctypes.Structure):
    """Mirror of solattn_rotary_t."""

    _fields_ = [("rot", ctypes.c_int), ("layout", ctypes.c_int), ("axes", ctypes.c_int), ("gain", ctypes.c_float),
                ("freq", ctypes.c_void_p), ("axis", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("position_batch", ctypes.c_longlong), ("position_token", ctypes.c_longlong)]


class CacheStruct(ctypes.Structure):
    """Mirror of solattn_cache_t."""

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int), ("heads", ctypes.c_int), ("d", ctypes.c_int),
                ("page_stride", ctypes.c_longlong), ("scale_stride", ctypes.c_longlong)]


_lib = None


def declare(L: ctypes.CDLL) -> ctypes.CDLL:
    """Sets the argument and result types of every exported call on a loaded
    copy of the library (the product build or its test-hook variant)."""
    i, vp, f, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    L.solattn_pooled_layout.argtypes = [i, i, i, i, vp, ctypes.POINTER(PooledStruct), ctypes.POINTER(sz)]
    L.solattn_pooled_layout.restype = i
    L.solattn_pool.argtypes = [vp, vp, vp, i, i, i, i, ctypes.POINTER(PooledStruct), vp]
    L.solattn_pool.restype = i
    L.solattn_forward.argtypes = [vp, vp, vp, i, i, i, i, ctypes.POINTER(PooledStruct), f, vp, vp, vp, vp, sz, vp]
    L.solattn_forward.restype = i
    L.solattn_dense.argtypes = [vp, vp, vp, i, i, i, i, vp, vp, vp, sz, vp]
    L.solattn_dense.restype = i
    L.solattn_status.argtypes = [vp, vp]
    L.solattn_status.restype = i
    L.solattn_strerror.argtypes = [i]
    L.solattn_strerror.restype = ctypes.c_char_p
    L.solattn_forward_noalloc.argtypes = [vp, vp, vp, i, i, i, i, f, vp, vp, vp, vp]
    L.solattn_forward_noalloc.restype = i
    L.solattn_noalloc_status.argtypes = [vp]
    L.solattn_noalloc_status.restype = i
    L.solattn_forward_ex.argtypes = [vp, vp, vp, i, i, i, i, ctypes.POINTER(PooledStruct),
                                     ctypes.POINTER(OptionsStruct), vp, vp, vp, vp, sz, vp]
    L.solattn_forward_ex.restype = i
    L.solattn_pool_ex.argtypes = [vp, vp, vp, i, i, i, i, ctypes.POINTER(StridesStruct), ctypes.POINTER(PooledStruct),
                                  vp]
    L.solattn_pool_ex.restype = i
    L.solattn_host_scratch_bytes.argtypes = [i, i, i, i, i, ctypes.POINTER(sz)]
    L.solattn_host_scratch_bytes.restype = i
    L.solattn_forward_host.argtypes = [vp, vp, vp, i, i, i, i, f, vp, vp, vp, i, vp, sz, vp]
    L.solattn_forward_host.restype = i
    ll, dbl, st = ctypes.c_longlong, ctypes.c_double, ctypes.POINTER(StridesStruct)
    L.solattn_rotary_frequencies.argtypes = [i, i, vp, dbl, i, dbl, dbl, dbl, dbl, vp, vp, ctypes.POINTER(f)]
    L.solattn_rotary_frequencies.restype = i
    L.solattn_rotary.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, st, st, st, st, ctypes.POINTER(RotaryStruct), i, vp]
    L.solattn_rotary.restype = i
    L.solattn_rotary_pool.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, st, st, ctypes.POINTER(RotaryStruct),
                                      ctypes.POINTER(PooledStruct), vp]
    L.solattn_rotary_pool.restype = i
    L.solattn_cache_append.argtypes = [vp, vp, i, i, i, st, ctypes.POINTER(CacheStruct), vp, i, ll, vp, vp, vp, sz, vp]
    L.solattn_cache_append.restype = i
    L.solattn_cache_workspace_bytes.argtypes = [i, i, i, i, i, i, ctypes.POINTER(sz)]
    L.solattn_cache_workspace_bytes.restype = i
    L.solattn_cache_attention.argtypes = [vp, i, i, i, i, i, st, ctypes.POINTER(CacheStruct), vp, i, ll, vp, vp, i, f,
                                          vp, st, vp, vp, sz, vp]
    L.solattn_cache_attention.restype = i
    L.solattn_version.argtypes = []
    L.solattn_version.restype = i
    return L


def lib() -> ctypes.CDLL:
    """The loaded library. Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing; build it with `python -m block_sparse_attention_cov_b200.build`"
        )
    _lib = declare(ctypes.CDLL(LIB_PATH))
    return _lib


def strerror(code: int) -> str:
    return lib().solattn_strerror(int(code)).decode()
