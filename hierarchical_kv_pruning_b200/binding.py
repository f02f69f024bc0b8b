"""ctypes binding of libatlaskv.so (the C ABI in include/atlaskv.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  The ``atlaskv_*`` functions mirror the C entry points one to one;
``HikvpTree`` is a thin convenience layer that takes torch tensors (torch is
used for device memory and streams), keeps them alive, and allocates outputs
and the workspace.  If the library is missing or fails to load, every call
raises: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libatlaskv.so")

ATLASKV_OK, ATLASKV_EINVAL, ATLASKV_ENOMEM, ATLASKV_ECUDA, ATLASKV_EUNSUPPORTED, ATLASKV_ETIMEOUT, ATLASKV_EDEVICE = range(7)
STATUS_NAMES = {0: "OK", 1: "EINVAL", 2: "ENOMEM", 3: "ECUDA", 4: "EUNSUPPORTED", 5: "ETIMEOUT", 6: "EDEVICE"}
ATLASKV_F32, ATLASKV_BF16 = 0, 1
ATLASKV_LEAVES_DEVICE, ATLASKV_LEAVES_HOST_PINNED = 0, 1
ATLASKV_PROFILE_TIMES, ATLASKV_PROFILE_COUNTERS = 1, 2
ATLASKV_DESCENT_AUTO, ATLASKV_DESCENT_FUSED, ATLASKV_DESCENT_PARENT_MAJOR = 0, 1, 2
ATLASKV_ROPE_HALF, ATLASKV_ROPE_INTERLEAVED = 0, 1
STAGE_NAMES = ("descend", "staging", "attend", "attend_seq", "attend_leaf")

# Every symbol include/atlaskv.h declares.
EXPORTED = ("atlaskv_create_tree", "atlaskv_workspace_size", "atlaskv_attend", "atlaskv_sync_status",
            "atlaskv_set_profiling", "atlaskv_stage_times", "atlaskv_refine_stats", "atlaskv_attend_static",
            "atlaskv_probe_wait_timeout", "atlaskv_destroy", "atlaskv_last_error", "atlaskv_workspace_size_layers",
            "atlaskv_attend_layers", "atlaskv_create_tree_csr", "atlaskv_workspace_size_csr", "atlaskv_attend_csr",
            "atlaskv_set_descent", "atlaskv_set_leaf_cache", "atlaskv_leaf_cache_stats", "atlaskv_rope_init",
            "atlaskv_rope", "atlaskv_cache_page_bytes", "atlaskv_create_cache", "atlaskv_destroy_cache",
            "atlaskv_cache_sync_status", "atlaskv_cache_append", "atlaskv_cache_read", "atlaskv_cache_workspace_size",
            "atlaskv_cache_attend", "atlaskv_workspace_size_cached", "atlaskv_attend_cached")
MAX_LAYERS = 32
MAX_LEVELS = 4
# Size of the library's static device scratch (ATLASKV_STATIC_SCRATCH_BYTES).
ATLASKV_STATIC_SCRATCH_BYTES = 16 * 1024 * 1024


class AtlaskvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), message))
        self.status = status


class atlaskv_tree_desc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("fanout", ctypes.c_int32 * 3),
        ("root_keys", ctypes.c_void_p),
        ("mid_keys", ctypes.c_void_p),
        ("leaf_keys", ctypes.c_void_p),
        ("leaf_values", ctypes.c_void_p),
        ("leaf_location", ctypes.c_int32),
        ("root_child", ctypes.c_void_p),
        ("mid_child", ctypes.c_void_p),
        ("mid_location", ctypes.c_int32),
    ]


class atlaskv_csr_tree_desc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("n_levels", ctypes.c_int32),
        ("rows", ctypes.c_int64 * 4),
        ("keys", ctypes.c_void_p * 4),
        ("child_off", ctypes.c_void_p * 3),
        ("child_id", ctypes.c_void_p * 3),
        ("leaf_values", ctypes.c_void_p),
    ]


class atlaskv_level_params(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32 * 4), ("scale", ctypes.c_float)]


class atlaskv_params(ctypes.Structure):
    _fields_ = [("K_root", ctypes.c_int32), ("K_mid", ctypes.c_int32), ("K_leaf", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class atlaskv_io(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("N", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
        ("q_kg", ctypes.c_void_p), ("q_seq", ctypes.c_void_p), ("k_seq", ctypes.c_void_p), ("v_seq", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("kept_root", ctypes.c_void_p), ("kept_mid", ctypes.c_void_p), ("kept_leaf", ctypes.c_void_p),
    ]


class atlaskv_rope_spec(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("amplitude", ctypes.c_double),
                ("freq", ctypes.c_double * 64)]


class atlaskv_rope_io(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("H", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("tokens", ctypes.c_int64),
        ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("positions", ctypes.c_void_p), ("y", ctypes.c_void_p),
        ("y_stride", ctypes.c_int64), ("backward", ctypes.c_int32),
    ]


class atlaskv_cache_desc(ctypes.Structure):
    _fields_ = [("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int64), ("pages", ctypes.c_void_p)]


class atlaskv_seqs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("q_len", ctypes.c_void_p)]


class atlaskv_append_io(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("positions", ctypes.c_void_p), ("H", ctypes.c_int32), ("q", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64), ("q_out", ctypes.c_void_p),
    ]


class atlaskv_cache_attend_io(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("H", ctypes.c_int32), ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("scale", ctypes.c_float),
    ]


_lib = None
_lock = threading.Lock()


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the in-tree library (raises OSError if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise OSError("libatlaskv.so not built at %s (run python -m hierarchical_kv_pruning_b200.build)" % p)
            lib = ctypes.CDLL(p)
            V, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            lib.atlaskv_create_tree.argtypes = [ctypes.POINTER(atlaskv_tree_desc), V, ctypes.POINTER(V)]
            lib.atlaskv_workspace_size.argtypes = [V, ctypes.POINTER(atlaskv_params), I32, I32, I32, I32,
                                                   ctypes.POINTER(SZ)]
            lib.atlaskv_attend.argtypes = [V, ctypes.POINTER(atlaskv_params), ctypes.POINTER(atlaskv_io), V, SZ, V]
            lib.atlaskv_attend_static.argtypes = [V, ctypes.POINTER(atlaskv_params), ctypes.POINTER(atlaskv_io), V]
            lib.atlaskv_workspace_size_layers.argtypes = [I32, ctypes.POINTER(V), ctypes.POINTER(atlaskv_params),
                                                          ctypes.POINTER(atlaskv_io), ctypes.POINTER(SZ)]
            lib.atlaskv_attend_layers.argtypes = [I32, ctypes.POINTER(V), ctypes.POINTER(atlaskv_params),
                                                  ctypes.POINTER(atlaskv_io), V, SZ, V]
            lib.atlaskv_create_tree_csr.argtypes = [ctypes.POINTER(atlaskv_csr_tree_desc), V, ctypes.POINTER(V)]
            lib.atlaskv_workspace_size_csr.argtypes = [V, ctypes.POINTER(atlaskv_level_params), I32, I32, I32, I32,
                                                       ctypes.POINTER(SZ)]
            lib.atlaskv_attend_csr.argtypes = [V, ctypes.POINTER(atlaskv_level_params), ctypes.POINTER(atlaskv_io),
                                               ctypes.POINTER(V), V, SZ, V]
            lib.atlaskv_sync_status.argtypes = [V, V]
            lib.atlaskv_set_profiling.argtypes = [V, I32]
            lib.atlaskv_set_descent.argtypes = [V, I32]
            lib.atlaskv_set_leaf_cache.argtypes = [V, ctypes.c_int64, V]
            lib.atlaskv_leaf_cache_stats.argtypes = [V, ctypes.POINTER(ctypes.c_uint64), I32]
            lib.atlaskv_stage_times.argtypes = [V, ctypes.POINTER(ctypes.c_float), I32]
            lib.atlaskv_refine_stats.argtypes = [V, ctypes.POINTER(ctypes.c_uint64), I32]
            lib.atlaskv_probe_wait_timeout.argtypes = [V, V]
            lib.atlaskv_destroy.argtypes = [V]
            F64, SEQS = ctypes.c_double, ctypes.POINTER(atlaskv_seqs)
            lib.atlaskv_rope_init.argtypes = [ctypes.POINTER(atlaskv_rope_spec), I32, I32, F64, F64, F64, F64, F64, F64]
            lib.atlaskv_rope.argtypes = [ctypes.POINTER(atlaskv_rope_spec), ctypes.POINTER(atlaskv_rope_io), V]
            lib.atlaskv_cache_page_bytes.argtypes = [I32, I32, I32, ctypes.POINTER(SZ)]
            lib.atlaskv_create_cache.argtypes = [ctypes.POINTER(atlaskv_cache_desc), V, ctypes.POINTER(V)]
            lib.atlaskv_destroy_cache.argtypes = [V]
            lib.atlaskv_cache_sync_status.argtypes = [V, V]
            lib.atlaskv_cache_append.argtypes = [V, ctypes.POINTER(atlaskv_rope_spec), SEQS,
                                                 ctypes.POINTER(atlaskv_append_io), V]
            lib.atlaskv_cache_read.argtypes = [V, SEQS, I32, V, V, V]
            lib.atlaskv_cache_workspace_size.argtypes = [V, I32, I32, I32, I32, ctypes.POINTER(SZ)]
            lib.atlaskv_cache_attend.argtypes = [V, SEQS, ctypes.POINTER(atlaskv_cache_attend_io), V, SZ, V]
            lib.atlaskv_workspace_size_cached.argtypes = [V, ctypes.POINTER(atlaskv_params), V, I32, I32, I32,
                                                          ctypes.POINTER(SZ)]
            lib.atlaskv_attend_cached.argtypes = [V, ctypes.POINTER(atlaskv_params), ctypes.POINTER(atlaskv_io), V, SEQS,
                                                  V, SZ, V]
            lib.atlaskv_last_error.argtypes = []
            lib.atlaskv_last_error.restype = ctypes.c_char_p
            for name in EXPORTED:
                if name != "atlaskv_last_error":
                    getattr(lib, name).restype = ctypes.c_int
            _lib = lib
    return _lib


def _check(status: int):
    if status:
        raise AtlaskvError(status, atlaskv_last_error())


# ---- one-to-one wrappers of the C entry points ------------------------------

def atlaskv_last_error() -> str:
    return load_library().atlaskv_last_error().decode()


def atlaskv_create_tree(desc: atlaskv_tree_desc, stream: int = 0) -> int:
    handle = ctypes.c_void_p()
    _check(load_library().atlaskv_create_tree(ctypes.byref(desc), ctypes.c_void_p(stream), ctypes.byref(handle)))
    return handle.value


def atlaskv_workspace_size(tree: int, params: atlaskv_params, B: int, N: int, H: int, T: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().atlaskv_workspace_size(ctypes.c_void_p(tree), ctypes.byref(params), B, N, H, T,
                                                 ctypes.byref(out)))
    return out.value


def atlaskv_attend(tree: int, params: atlaskv_params, io: atlaskv_io, workspace: int, workspace_bytes: int,
                   stream: int = 0) -> None:
    _check(load_library().atlaskv_attend(ctypes.c_void_p(tree), ctypes.byref(params), ctypes.byref(io),
                                         ctypes.c_void_p(workspace), workspace_bytes, ctypes.c_void_p(stream)))


def atlaskv_attend_static(tree: int, params: atlaskv_params, io: atlaskv_io, stream: int = 0) -> None:
    """atlaskv_attend without a caller workspace: the library's static device
    scratch (ATLASKV_STATIC_SCRATCH_BYTES) is used instead.  For callers that
    cannot allocate device memory; calls that overlap on the GPU race."""
    _check(load_library().atlaskv_attend_static(ctypes.c_void_p(tree), ctypes.byref(params), ctypes.byref(io),
                                                ctypes.c_void_p(stream)))


def atlaskv_workspace_size_layers(trees, params: atlaskv_params, ios) -> int:
    n = len(trees)
    th = (ctypes.c_void_p * n)(*trees)
    io_arr = (atlaskv_io * n)(*ios)
    out = ctypes.c_size_t()
    _check(load_library().atlaskv_workspace_size_layers(n, th, ctypes.byref(params), io_arr, ctypes.byref(out)))
    return out.value


def atlaskv_attend_layers(trees, params: atlaskv_params, ios, workspace: int, workspace_bytes: int,
                          stream: int = 0) -> None:
    n = len(trees)
    th = (ctypes.c_void_p * n)(*trees)
    io_arr = (atlaskv_io * n)(*ios)
    _check(load_library().atlaskv_attend_layers(n, th, ctypes.byref(params), io_arr, ctypes.c_void_p(workspace),
                                                workspace_bytes, ctypes.c_void_p(stream)))


def atlaskv_create_tree_csr(desc: atlaskv_csr_tree_desc, stream: int = 0) -> int:
    handle = ctypes.c_void_p()
    _check(load_library().atlaskv_create_tree_csr(ctypes.byref(desc), ctypes.c_void_p(stream), ctypes.byref(handle)))
    return handle.value


def atlaskv_workspace_size_csr(tree: int, params: atlaskv_level_params, B: int, N: int, H: int, T: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().atlaskv_workspace_size_csr(ctypes.c_void_p(tree), ctypes.byref(params), B, N, H, T,
                                                     ctypes.byref(out)))
    return out.value


def atlaskv_attend_csr(tree: int, params: atlaskv_level_params, io: atlaskv_io, kept, workspace: int,
                       workspace_bytes: int, stream: int = 0) -> None:
    """kept: a list of n_levels device pointers (or None entries), or None."""
    arr = None if kept is None else (ctypes.c_void_p * len(kept))(*kept)
    _check(load_library().atlaskv_attend_csr(ctypes.c_void_p(tree), ctypes.byref(params), ctypes.byref(io), arr,
                                             ctypes.c_void_p(workspace), workspace_bytes, ctypes.c_void_p(stream)))


def atlaskv_sync_status(tree: int, stream: int = 0) -> None:
    _check(load_library().atlaskv_sync_status(ctypes.c_void_p(tree), ctypes.c_void_p(stream)))


def atlaskv_set_profiling(tree: int, enable: int) -> None:
    """enable: bit mask of ATLASKV_PROFILE_TIMES and ATLASKV_PROFILE_COUNTERS (0: off)."""
    _check(load_library().atlaskv_set_profiling(ctypes.c_void_p(tree), int(enable)))


def atlaskv_set_descent(tree: int, mode: int) -> None:
    """mode: ATLASKV_DESCENT_AUTO, ATLASKV_DESCENT_FUSED or ATLASKV_DESCENT_PARENT_MAJOR."""
    _check(load_library().atlaskv_set_descent(ctypes.c_void_p(tree), int(mode)))


def atlaskv_set_leaf_cache(tree: int, blocks: int, stream: int = 0) -> None:
    """HBM cache of `blocks` staged leaf-key blocks across calls (0: none)."""
    _check(load_library().atlaskv_set_leaf_cache(ctypes.c_void_p(tree), int(blocks), ctypes.c_void_p(stream)))


def atlaskv_leaf_cache_stats(tree: int):
    """Cumulative cache counters: dict(hits, fills, bypasses)."""
    out = (ctypes.c_uint64 * 3)()
    _check(load_library().atlaskv_leaf_cache_stats(ctypes.c_void_p(tree), out, 3))
    return {"hits": int(out[0]), "fills": int(out[1]), "bypasses": int(out[2])}


def atlaskv_stage_times(tree: int):
    """Stage times (ms) of the last timed call, in the order of STAGE_NAMES."""
    buf = (ctypes.c_float * 5)()
    _check(load_library().atlaskv_stage_times(ctypes.c_void_p(tree), buf, 5))
    return [float(x) for x in buf]


def atlaskv_refine_stats(tree: int):
    """Descent counters of the last profiled call: per level [selections,
    selections needing exact refinement, ambiguous candidates, exact scores]."""
    buf = (ctypes.c_uint64 * 16)()
    _check(load_library().atlaskv_refine_stats(ctypes.c_void_p(tree), buf, 16))
    v = [int(x) for x in buf]
    names = ("root", "mid", "leaf", "level3")
    return {names[i]: dict(zip(("selections", "refined", "ambiguous", "exact_scores"), v[4 * i:4 * i + 4]))
            for i in range(4) if i < 3 or v[4 * i] > 0}


def atlaskv_probe_wait_timeout(tree: int, stream: int = 0) -> None:
    _check(load_library().atlaskv_probe_wait_timeout(ctypes.c_void_p(tree), ctypes.c_void_p(stream)))


def atlaskv_destroy(tree: int) -> None:
    _check(load_library().atlaskv_destroy(ctypes.c_void_p(tree)))


def atlaskv_rope_init(layout: int, rotary_dim: int, base: float, factor: float, original_len: float,
                      low_turns: float, high_turns: float, amplitude: float) -> atlaskv_rope_spec:
    spec = atlaskv_rope_spec()
    _check(load_library().atlaskv_rope_init(ctypes.byref(spec), layout, rotary_dim, base, factor, original_len,
                                            low_turns, high_turns, amplitude))
    return spec


def atlaskv_rope(spec: atlaskv_rope_spec, io: atlaskv_rope_io, stream: int = 0) -> None:
    _check(load_library().atlaskv_rope(ctypes.byref(spec), ctypes.byref(io), stream))


def atlaskv_cache_page_bytes(n_kv_heads: int, head_dim: int, page_size: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().atlaskv_cache_page_bytes(n_kv_heads, head_dim, page_size, ctypes.byref(out)))
    return out.value


def atlaskv_create_cache(desc: atlaskv_cache_desc, stream: int = 0) -> int:
    handle = ctypes.c_void_p()
    _check(load_library().atlaskv_create_cache(ctypes.byref(desc), stream, ctypes.byref(handle)))
    return handle.value


def atlaskv_destroy_cache(cache: int) -> None:
    _check(load_library().atlaskv_destroy_cache(cache))


def atlaskv_cache_sync_status(cache: int, stream: int = 0) -> None:
    _check(load_library().atlaskv_cache_sync_status(cache, stream))


def atlaskv_cache_append(cache: int, rope: Optional[atlaskv_rope_spec], seqs: atlaskv_seqs, io: atlaskv_append_io,
                         stream: int = 0) -> None:
    _check(load_library().atlaskv_cache_append(cache, None if rope is None else ctypes.byref(rope), ctypes.byref(seqs),
                                               ctypes.byref(io), stream))


def atlaskv_cache_read(cache: int, seqs: atlaskv_seqs, dtype: int, k_out: Optional[int], v_out: Optional[int],
                       stream: int = 0) -> None:
    _check(load_library().atlaskv_cache_read(cache, ctypes.byref(seqs), dtype, k_out, v_out, stream))


def atlaskv_cache_workspace_size(cache: int, dtype: int, B: int, N: int, H: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().atlaskv_cache_workspace_size(cache, dtype, B, N, H, ctypes.byref(out)))
    return out.value


def atlaskv_cache_attend(cache: int, seqs: atlaskv_seqs, io: atlaskv_cache_attend_io, workspace: Optional[int],
                         workspace_bytes: int, stream: int = 0) -> None:
    _check(load_library().atlaskv_cache_attend(cache, ctypes.byref(seqs), ctypes.byref(io), workspace,
                                               workspace_bytes, stream))


def atlaskv_workspace_size_cached(tree: int, params: atlaskv_params, cache: int, B: int, N: int, H: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().atlaskv_workspace_size_cached(tree, ctypes.byref(params), cache, B, N, H, ctypes.byref(out)))
    return out.value


def atlaskv_attend_cached(tree: int, params: atlaskv_params, io: atlaskv_io, cache: int, seqs: atlaskv_seqs,
                          workspace: int, workspace_bytes: int, stream: int = 0) -> None:
    _check(load_library().atlaskv_attend_cached(tree, ctypes.byref(params), ctypes.byref(io), cache,
                                                ctypes.byref(seqs), workspace, workspace_bytes, stream))


# ---- torch-facing convenience ------------------------------------------------

def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return ATLASKV_F32
    if t == torch.bfloat16:
        return ATLASKV_BF16
    raise AtlaskvError(ATLASKV_EINVAL, "dtype %s not supported (float32 or bfloat16)" % t)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise AtlaskvError(ATLASKV_EINVAL, "tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


class HikvpTree:
    """A key tree registered with the library.  Holds references to the
    tensors it borrows; call ``close()`` (or use ``with``) to release."""

    def __init__(self, root_keys, mid_keys, leaf_keys, leaf_values, fanout, root_child=None, mid_child=None,
                 stream=None):
        self._keep = (root_keys, mid_keys, leaf_keys, leaf_values, root_child, mid_child)
        self.dtype = root_keys.dtype
        self.fanout = tuple(int(f) for f in fanout)
        self.n_kv_heads, _, self.head_dim = root_keys.shape
        on_host = not leaf_keys.is_cuda
        mids_on_host = not mid_keys.is_cuda
        if on_host and not (leaf_keys.is_pinned() and leaf_values.is_pinned()):
            raise AtlaskvError(ATLASKV_EINVAL, "host-resident leaves must be pinned tensors")
        if mids_on_host and not mid_keys.is_pinned():
            raise AtlaskvError(ATLASKV_EINVAL, "host-resident mid keys must be a pinned tensor")
        d = atlaskv_tree_desc()
        d.dtype = _dtype_code(self.dtype)
        d.n_kv_heads = self.n_kv_heads
        d.head_dim = self.head_dim
        d.fanout[:] = self.fanout
        d.root_keys, d.mid_keys = _ptr(root_keys), _ptr(mid_keys)
        d.leaf_keys, d.leaf_values = _ptr(leaf_keys), _ptr(leaf_values)
        d.leaf_location = ATLASKV_LEAVES_HOST_PINNED if on_host else ATLASKV_LEAVES_DEVICE
        d.root_child, d.mid_child = _ptr(root_child), _ptr(mid_child)
        d.mid_location = ATLASKV_LEAVES_HOST_PINNED if mids_on_host else ATLASKV_LEAVES_DEVICE
        self.desc = d
        self.handle = atlaskv_create_tree(d, _stream(stream))
        self.leaves_on_host = on_host
        self.mids_on_host = mids_on_host

    @classmethod
    def from_workload(cls, w, stream=None):
        return cls(w.root_keys, w.mid_keys, w.leaf_keys, w.leaf_values, w.shape.fanout, w.root_child, w.mid_child,
                   stream)

    def close(self):
        if getattr(self, "handle", None):
            atlaskv_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def params(self, K, scale: float = 0.0) -> atlaskv_params:
        return atlaskv_params(int(K[0]), int(K[1]), int(K[2]), float(scale))

    def workspace_size(self, K, B, N, H, T, scale: float = 0.0) -> int:
        return atlaskv_workspace_size(self.handle, self.params(K, scale), B, N, H, T)

    def attend(self, q_kg, q_seq, k_seq, v_seq, K, scale: float = 0.0, out=None, lse=None, kept=None,
               workspace=None, want_kept: bool = True, want_lse: bool = True, stream=None):
        """Enqueue the whole path.  Returns dict(out, lse, kept_root, kept_mid,
        kept_leaf) of device tensors (lse / kept_* None when not requested)."""
        B, N, H, D = q_kg.shape
        T = k_seq.shape[1]
        dev = q_kg.device
        p = self.params(K, scale)
        if out is None:
            out = torch.empty_like(q_kg)
        if want_lse and lse is None:
            lse = torch.empty((B, N, H), dtype=torch.float32, device=dev)
        if want_kept and kept is None:
            kept = tuple(torch.empty((B, H, int(k)), dtype=torch.int32, device=dev) for k in K)
        if kept is None:
            kept = (None, None, None)
        if workspace is None:
            nbytes = atlaskv_workspace_size(self.handle, p, B, N, H, T)
            workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        io = atlaskv_io(B, N, H, T, _ptr(q_kg), _ptr(q_seq), _ptr(k_seq), _ptr(v_seq), _ptr(out), _ptr(lse),
                        _ptr(kept[0]), _ptr(kept[1]), _ptr(kept[2]))
        atlaskv_attend(self.handle, p, io, workspace.data_ptr(), workspace.numel(), _stream(stream))
        return {"out": out, "lse": lse, "kept_root": kept[0], "kept_mid": kept[1], "kept_leaf": kept[2],
                "workspace": workspace}

    def attend_cached(self, q_kg, q_seq, cache: "KvCache", block_table, kv_len, K, scale: float = 0.0, out=None, lse=None,
                      kept=None, workspace=None, want_kept: bool = True, want_lse: bool = True, stream=None):
        """attend() with the sequence's keys and values in `cache` (kv_len [B]
        stored tokens, the N query tokens being the newest).  Returns the same dict."""
        B, N, H, D = q_kg.shape
        p, new = self.params(K, scale), []

        def alloc(shape, dtype):
            new.append(torch.empty(shape, dtype=dtype, device=q_kg.device))
            return new[-1]

        if out is None:
            out = alloc(q_kg.shape, q_kg.dtype)
        if want_lse and lse is None:
            lse = alloc((B, N, H), torch.float32)
        if want_kept and kept is None:
            kept = tuple(alloc((B, H, int(k)), torch.int32) for k in K)
        if kept is None:
            kept = (None, None, None)
        if workspace is None:
            nbytes = atlaskv_workspace_size_cached(self.handle, p, cache.handle, B, N, H)
            workspace = alloc((max(nbytes, 256),), torch.uint8)
        s = _on_device(cache._index, stream, q_kg, q_seq, block_table, kv_len, out, lse, workspace, *kept)
        shape = (B, N, H, D)
        io = atlaskv_io(B, N, H, N, _dense("q_kg", q_kg, shape, self.dtype), _dense("q_seq", q_seq, shape, self.dtype),
                        None, None, _dense("out", out, shape, self.dtype),
                        None if lse is None else _dense("lse", lse, shape[:3], torch.float32),
                        *[_ints("kept", x, (B, H, int(k))) for x, k in zip(kept, K)])
        seqs = cache._seqs(B, N, block_table, kv_len, None)
        _used_on(stream, *new)
        atlaskv_attend_cached(self.handle, p, io, cache.handle, seqs, *_space(workspace), s)
        return {"out": out, "lse": lse, "kept_root": kept[0], "kept_mid": kept[1], "kept_leaf": kept[2],
                "workspace": workspace}

    def sync_status(self, stream=None):
        atlaskv_sync_status(self.handle, _stream(stream))

    def probe_wait_timeout(self, stream=None):
        atlaskv_probe_wait_timeout(self.handle, _stream(stream))

    def set_profiling(self, times: bool = True, counters: bool = True):
        atlaskv_set_profiling(self.handle, (ATLASKV_PROFILE_TIMES if times else 0) |
                              (ATLASKV_PROFILE_COUNTERS if counters else 0))

    def set_descent(self, mode: int):
        """ATLASKV_DESCENT_AUTO, ATLASKV_DESCENT_FUSED or ATLASKV_DESCENT_PARENT_MAJOR (same results)."""
        atlaskv_set_descent(self.handle, mode)

    def set_leaf_cache(self, blocks: int, stream=None):
        """HBM cache of staged leaf blocks across calls (host-resident leaves; 0 removes it)."""
        atlaskv_set_leaf_cache(self.handle, blocks, _stream(stream))

    def leaf_cache_stats(self):
        return atlaskv_leaf_cache_stats(self.handle)

    def stage_times(self):
        return atlaskv_stage_times(self.handle)

    def refine_stats(self):
        return atlaskv_refine_stats(self.handle)


def attend_layers(trees, inputs, K, scale: float = 0.0, workspace=None, stream=None):
    """Several layers' calls in one batch (atlaskv_attend_layers).  trees: a
    HikvpTree per layer; inputs: per layer (q_kg, q_seq, k_seq, v_seq).
    Returns per layer dict(out, lse, kept_root, kept_mid, kept_leaf)."""
    outs, ios = [], []
    for tree, (q_kg, q_seq, k_seq, v_seq) in zip(trees, inputs):
        B, N, H, D = q_kg.shape
        T = k_seq.shape[1]
        dev = q_kg.device
        r = {"out": torch.empty_like(q_kg), "lse": torch.empty((B, N, H), dtype=torch.float32, device=dev)}
        for name, k in zip(("kept_root", "kept_mid", "kept_leaf"), K):
            r[name] = torch.empty((B, H, int(k)), dtype=torch.int32, device=dev)
        ios.append(atlaskv_io(B, N, H, T, _ptr(q_kg), _ptr(q_seq), _ptr(k_seq), _ptr(v_seq), _ptr(r["out"]),
                              _ptr(r["lse"]), _ptr(r["kept_root"]), _ptr(r["kept_mid"]), _ptr(r["kept_leaf"])))
        outs.append(r)
    p = trees[0].params(K, scale)
    handles = [t.handle for t in trees]
    if workspace is None:
        nbytes = atlaskv_workspace_size_layers(handles, p, ios)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=inputs[0][0].device)
    atlaskv_attend_layers(handles, p, ios, workspace.data_ptr(), workspace.numel(), _stream(stream))
    for r in outs:
        r["workspace"] = workspace
    return outs


class CsrHikvpTree:
    """A CSR tree (any depth, variable numbers of children) registered with
    the library: keys[l] [H_kv][rows_l][D] per level, child_off[l]
    [H_kv][rows_l + 1], child_id[l] [H_kv][rows_{l+1}] or None, leaf values of
    the last level.  Holds references to the tensors it borrows."""

    def __init__(self, keys, leaf_values, child_off, child_id=None, stream=None):
        n = len(keys)
        child_id = child_id if child_id is not None else [None] * (n - 1)
        self._keep = (keys, leaf_values, child_off, child_id)
        self.n_levels = n
        self.dtype = keys[0].dtype
        self.n_kv_heads, _, self.head_dim = keys[0].shape
        d = atlaskv_csr_tree_desc()
        d.dtype = _dtype_code(self.dtype)
        d.n_kv_heads = self.n_kv_heads
        d.head_dim = self.head_dim
        d.n_levels = n
        for l, k in enumerate(keys):
            d.rows[l] = k.shape[1]
            d.keys[l] = _ptr(k)
        for l in range(n - 1):
            d.child_off[l] = _ptr(child_off[l])
            d.child_id[l] = _ptr(child_id[l])
        d.leaf_values = _ptr(leaf_values)
        self.desc = d
        self.handle = atlaskv_create_tree_csr(d, _stream(stream))

    @classmethod
    def from_workload(cls, w, stream=None):
        return cls(w.keys, w.leaf_values, w.child_off, w.child_id, stream)

    def close(self):
        if getattr(self, "handle", None):
            atlaskv_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def params(self, K, scale: float = 0.0) -> atlaskv_level_params:
        p = atlaskv_level_params()
        for l, k in enumerate(K):
            p.K[l] = int(k)
        p.scale = float(scale)
        return p

    def attend(self, q_kg, q_seq, k_seq, v_seq, K, scale: float = 0.0, workspace=None, stream=None):
        """Returns dict(out, lse, kept: a list of [B][H][K_l] per level)."""
        B, N, H, D = q_kg.shape
        T = k_seq.shape[1]
        dev = q_kg.device
        p = self.params(K, scale)
        out = torch.empty_like(q_kg)
        lse = torch.empty((B, N, H), dtype=torch.float32, device=dev)
        kept = [torch.empty((B, H, int(k)), dtype=torch.int32, device=dev) for k in K]
        if workspace is None:
            nbytes = atlaskv_workspace_size_csr(self.handle, p, B, N, H, T)
            workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        io = atlaskv_io(B, N, H, T, _ptr(q_kg), _ptr(q_seq), _ptr(k_seq), _ptr(v_seq), _ptr(out), _ptr(lse),
                        None, None, None)
        atlaskv_attend_csr(self.handle, p, io, [k.data_ptr() for k in kept], workspace.data_ptr(), workspace.numel(),
                           _stream(stream))
        return {"out": out, "lse": lse, "kept": kept, "workspace": workspace}

    def sync_status(self, stream=None):
        atlaskv_sync_status(self.handle, _stream(stream))

    def set_profiling(self, times: bool = True, counters: bool = True):
        atlaskv_set_profiling(self.handle, (ATLASKV_PROFILE_TIMES if times else 0) |
                              (ATLASKV_PROFILE_COUNTERS if counters else 0))

    def set_descent(self, mode: int):
        """ATLASKV_DESCENT_AUTO, ATLASKV_DESCENT_FUSED or ATLASKV_DESCENT_PARENT_MAJOR (same results)."""
        atlaskv_set_descent(self.handle, mode)

    def refine_stats(self):
        return atlaskv_refine_stats(self.handle)


# A decode step makes two of the calls below per layer, so their checks are
# kept to a few tensor queries each.

def _refuse(name: str, t: torch.Tensor, shape, dtype, what: str):
    raise AtlaskvError(ATLASKV_EINVAL, "%s must be a %s %s tensor of shape %s, not %s of shape %s and strides %s" %
                       (name, what, dtype, tuple(shape), t.dtype, tuple(t.shape), t.stride()))


def _rows(name: str, t: torch.Tensor, shape, dtype: torch.dtype) -> int:
    """Token stride of a token tensor [B][N][heads][D] whose token rows are
    dense and evenly spaced, as a slice of a wider projection's is (0: dense).
    Tokens that share memory, as an expanded tensor's do, are refused: the
    library takes a stride of 0 for a dense tensor."""
    if t.dtype is not dtype or t.shape != shape:
        _refuse(name, t, shape, dtype, "token")
    if t.is_contiguous():
        return 0
    s0, s1, s2, s3 = t.stride()
    if shape[1] == 1:      # one token per sequence: the stride between sequences is the token stride
        s1 = s0
    if shape[0] * shape[1] == 1:
        s1 = shape[2] * shape[3]
    if (s3 != 1 or (s2 != shape[3] and shape[2] > 1) or s1 < shape[2] * shape[3] or
            (shape[0] > 1 and s0 != shape[1] * s1)):
        _refuse(name, t, shape, dtype, "token")
    return s1


def _dense(name: str, t: torch.Tensor, shape, dtype: torch.dtype) -> int:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _refuse(name, t, shape, dtype, "contiguous")
    return t.data_ptr()


def _ints(name: str, t: Optional[torch.Tensor], shape) -> Optional[int]:
    return None if t is None else _dense(name, t, shape, torch.int32)


def _space(t: torch.Tensor):
    """(address, bytes) of a workspace: its own bytes, all of them, and no others."""
    if not t.is_contiguous():
        raise AtlaskvError(ATLASKV_EINVAL, "the workspace must be contiguous, not of shape %s and strides %s" %
                           (tuple(t.shape), t.stride()))
    return t.data_ptr(), t.nbytes


def _on_device(index: int, stream, *tensors) -> int:
    """The stream to launch on: `stream`, or the current one of the current
    device, where every tensor has to be."""
    if index != torch._C._cuda_getDevice():
        raise AtlaskvError(ATLASKV_EINVAL, "device %d is not the current device" % index)
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise AtlaskvError(ATLASKV_EINVAL, "a tensor on %s in a call on device %d" % (t.device, index))
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else int(stream.cuda_stream)


def _used_on(stream, *tensors):
    """Tensors allocated here belong to the current stream, whose earlier work may still use their memory: a call on
    another stream waits for that, and the memory for the call."""
    if stream is None or not tensors:
        return
    current = torch.cuda.current_stream()
    if stream.cuda_stream != current.cuda_stream:
        stream.wait_stream(current)
        for t in tensors:
            t.record_stream(stream)


class Rope:
    """Rotary positions: frequencies base^(-2 i / rotary_dim), rescaled for
    contexts `factor` times original_len (see atlaskv_rope_init)."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False, factor: float = 1.0,
                 original_len: float = 0, low_turns: float = 1.0, high_turns: float = 32.0, amplitude: float = 1.0):
        self.spec = atlaskv_rope_init(ATLASKV_ROPE_INTERLEAVED if interleaved else ATLASKV_ROPE_HALF, int(rotary_dim),
                                      float(base), float(factor), float(original_len), float(low_turns),
                                      float(high_turns), float(amplitude))


def rope(x, positions, spec: Rope, out=None, backward: bool = False, stream=None):
    """Rotate x [B][N][H][D] by positions [B][N] (int32) into out (a new
    tensor by default; x itself for in place).  backward=True is the transpose:
    it turns a gradient of the rotated tensor into that of the tensor.  An x
    that requires a gradient gets it so in autograd, on the stream that is
    current; not with out=, which is refused unless gradients are off."""
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise AtlaskvError(ATLASKV_EINVAL, "rope(out=) records no gradient, and x requires one")
        return _Rotation.apply(x, positions, spec, backward, stream)
    return _rotate(x, positions, spec, out, backward, stream)


def _rotate(x, positions, spec: Rope, out, backward: bool, stream):
    shape, dtype, new = x.shape, x.dtype, ()
    if len(shape) != 4 or not x.is_cuda:
        raise AtlaskvError(ATLASKV_EINVAL, "x must be a CUDA tensor [B][N][H][D]")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
        new = (out,)
    B, N, H, D = shape
    s = _on_device(x.get_device(), stream, positions, out)
    io = atlaskv_rope_io(_dtype_code(dtype), H, D, B * N, x.data_ptr(), _rows("x", x, shape, dtype),
                         _dense("positions", positions, (B, N), torch.int32), out.data_ptr(),
                         _rows("out", out, shape, dtype), 1 if backward else 0)
    _used_on(stream, *new)
    atlaskv_rope(spec.spec, io, s)
    return out


class _Rotation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, spec, backward, stream):
        ctx.save_for_backward(positions)
        ctx.spec, ctx.direction = spec, bool(backward)
        return _rotate(x, positions, spec, None, backward, stream)

    @staticmethod
    def backward(ctx, dy):
        positions, = ctx.saved_tensors
        # (a gradient may be expanded; one that a second pass needs is recorded in its turn)
        return rope(dy.contiguous(), positions, ctx.spec, backward=not ctx.direction), None, None, None, None


class KvCache:
    """A pool of 4-bit cache pages registered with the library.  pages: uint8
    [n_pages][page bytes] on the GPU (KvCache.page_bytes gives the width),
    borrowed and kept alive.  The calls take one batch's block_table
    [B][max_pages], kv_len [B] and q_len [B] (or None: every row), int32 on the
    GPU, as atlaskv_seqs describes them; a decode step appends its tokens and
    attends with the same three.  For serving: no call records a gradient."""

    def __init__(self, pages, n_kv_heads: int, head_dim: int, page_size: int, stream=None):
        self.handle = None
        self.n_kv_heads, self.head_dim, self.page_size = int(n_kv_heads), int(head_dim), int(page_size)
        width = self.page_bytes(n_kv_heads, head_dim, page_size)
        if pages.dtype != torch.uint8 or pages.dim() != 2 or pages.shape[1] != width or not pages.is_cuda:
            raise AtlaskvError(ATLASKV_EINVAL, "pages must be a uint8 [n_pages][%d] CUDA tensor" % width)
        self.pages, self.device = pages, pages.device
        d = atlaskv_cache_desc(self.n_kv_heads, self.head_dim, self.page_size, pages.shape[0], _ptr(pages))
        self._index = pages.get_device()
        self.handle = atlaskv_create_cache(d, _on_device(self._index, stream))

    @staticmethod
    def page_bytes(n_kv_heads: int, head_dim: int, page_size: int) -> int:
        return atlaskv_cache_page_bytes(int(n_kv_heads), int(head_dim), int(page_size))

    @classmethod
    def allocate(cls, n_pages: int, n_kv_heads: int, head_dim: int, page_size: int, device="cuda", stream=None):
        pages = torch.empty((int(n_pages), cls.page_bytes(n_kv_heads, head_dim, page_size)), dtype=torch.uint8,
                            device=device)
        return cls(pages, n_kv_heads, head_dim, page_size, stream)

    def close(self):
        if getattr(self, "handle", None):
            atlaskv_destroy_cache(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _seqs(self, B: int, N: int, block_table, kv_len, q_len) -> atlaskv_seqs:
        shape = block_table.shape
        if len(shape) != 2 or shape[0] != B:
            _refuse("block_table", block_table, (B, "max_pages"), torch.int32, "contiguous")
        return atlaskv_seqs(B, N, shape[1], _dense("block_table", block_table, shape, torch.int32),
                            _dense("kv_len", kv_len, (B,), torch.int32), _ints("q_len", q_len, (B,)))

    def append(self, k, v, block_table, kv_len, q_len=None, rope: Optional[Rope] = None, positions=None, q=None,
               q_out=None, stream=None):
        """Store the new tokens' k and v [B][N][H_kv][D] (k rotated when rope
        is given, by positions [B][N] or by slot) and rotate the queries
        q [B][N][H][D] into q_out along the way.  Returns q_out (None without q)."""
        if k.dim() != 4:
            raise AtlaskvError(ATLASKV_EINVAL, "k must be [B][N][H_kv][D]")
        B, N = k.shape[:2]
        dtype, new = k.dtype, ()
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=dtype, device=q.device)
            new = (q_out,)
        s = _on_device(self._index, stream, k, v, block_table, kv_len, q_len, positions, q, q_out)
        shape = (B, N, self.n_kv_heads, self.head_dim)
        qp = qo = None
        qs = H = 0
        if q is not None:
            H = q.shape[2] if q.dim() == 4 else 0
            q_shape = (B, N, H, self.head_dim)
            qp, qs, qo = q.data_ptr(), _rows("q", q, q_shape, dtype), _dense("q_out", q_out, q_shape, dtype)
        io = atlaskv_append_io(_dtype_code(dtype), k.data_ptr(), v.data_ptr(), _rows("k", k, shape, dtype),
                               _rows("v", v, shape, dtype), _ints("positions", positions, (B, N)), H, qp, qs, qo)
        seqs = self._seqs(B, N, block_table, kv_len, q_len)
        _used_on(stream, *new)
        atlaskv_cache_append(self.handle, None if rope is None else rope.spec, seqs, io, s)
        return q_out

    def read(self, N: int, block_table, kv_len, q_len=None, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
        """The q_len newest tokens of each sequence (q_len=kv_len: all of them)
        as k, v [B][N][H_kv][D]; rows past q_len are left as they were (zero
        in tensors allocated here)."""
        shape = (block_table.shape[0], int(N), self.n_kv_heads, self.head_dim)
        new = []
        if k_out is None:
            k_out = torch.zeros(shape, dtype=dtype, device=self.device)
            new.append(k_out)
        dtype = k_out.dtype
        if v_out is None:
            v_out = torch.zeros(shape, dtype=dtype, device=self.device)
            new.append(v_out)
        s = _on_device(self._index, stream, block_table, kv_len, q_len, k_out, v_out)
        seqs = self._seqs(shape[0], shape[1], block_table, kv_len, q_len)
        kp, vp = _dense("k_out", k_out, shape, dtype), _dense("v_out", v_out, shape, dtype)
        _used_on(stream, *new)   # which includes the zeros' writing
        atlaskv_cache_read(self.handle, seqs, _dtype_code(dtype), kp, vp, s)
        return k_out, v_out

    def workspace_size(self, dtype, B: int, N: int, H: int) -> int:
        return atlaskv_cache_workspace_size(self.handle, _dtype_code(dtype), B, N, H)

    def attend(self, q, block_table, kv_len, q_len=None, scale: float = 0.0, out=None, lse=None, workspace=None,
               stream=None):
        """Causal attention of q [B][N][H][D] over the stored sequences:
        (out, lse).  Rows past q_len are left as they were."""
        if q.dim() != 4:
            raise AtlaskvError(ATLASKV_EINVAL, "q must be [B][N][H][D]")
        B, N, H, _ = q.shape
        shape, dtype, new = (B, N, H, self.head_dim), q.dtype, []
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=q.device)
            new.append(out)
        if lse is None:
            lse = torch.empty((B, N, H), dtype=torch.float32, device=q.device)
            new.append(lse)
        code = _dtype_code(dtype)
        if workspace is None:
            nbytes = atlaskv_cache_workspace_size(self.handle, code, B, N, H)
            workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
            new.append(workspace)
        s = _on_device(self._index, stream, q, block_table, kv_len, q_len, out, lse, workspace)
        io = atlaskv_cache_attend_io(code, H, q.data_ptr(), _rows("q", q, shape, dtype),
                                     _dense("out", out, shape, dtype), _dense("lse", lse, (B, N, H), torch.float32),
                                     scale)
        seqs = self._seqs(B, N, block_table, kv_len, q_len)
        _used_on(stream, *new)
        atlaskv_cache_attend(self.handle, seqs, io, *_space(workspace), s)
        return out, lse

    def sync_status(self, stream=None):
        """Raises on a device-side error of the calls so far."""
        atlaskv_cache_sync_status(self.handle, _on_device(self._index, stream))
