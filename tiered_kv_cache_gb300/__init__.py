"""tiered_kv_cache_gb300: L1 (GPU HBM) <-> L2 (pinned host DRAM) paged KV movement
for GB300, as a thin ctypes binding over ``libhicache.so``.

The binding only marshals arguments: every step of a transfer (validation,
pre-pass, kernels) runs in the C/CUDA library.  There is no fallback: if the
library is not built, importing works but every call raises.

Names follow the C ABI in ``include/hicache.h``:
    Pool.backup / Pool.load / Pool.load_layer / Pool.load_pipelined / Pool.backup_load
    Pool.wait_layer / Pool.layer_event
    Pool.plan(...) -> Plan.execute / load_layer / load_layer_chained / load_layers / load_pipelined
    group_transfer / group_load_pipelined / group_plan(...) -> GroupPlan
    Engine (submission engine), PageAllocator (host pages)
    host_alloc / host_free, wait, prepass, segment_count, page_span, layer_checksum
    tp_share / tp_load_pipelined / Pool.layer_counters (tensor-parallel load of a replicated latent)
    append_kv / decode_attention / decode_workspace / decode_gave_up / evict_pages,
    query_attention / query_workspace / prefix_attention / prefix_workspace / merge_attention
    (operators on the device pages)
    stream_copy (roofline probe: plain zero-copy streaming copy)
    checked_build / check_status (the bounds-checked build, HICACHE_CHECKED=1)
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import numpy as np

__all__ = [
    "HiCacheError", "LAYER_FIRST", "PAGE_FIRST", "PAGE_FIRST_DIRECT", "LAYOUT_POOL", "LAYOUTS",
    "BACKUP", "LOAD", "library", "library_path", "PoolDesc", "DeviceKV", "Pool", "Plan", "PinnedHost",
    "PageAllocator", "Engine", "group_transfer", "group_load_pipelined", "group_plan", "GroupPlan",
    "MAX_GROUP", "PAGE_FIRST_DIRECT_KV",
    "host_alloc", "host_free", "wait", "prepass", "segment_count", "layer_checksum", "page_span",
    "launch_count", "version", "stream_copy", "tp_share", "tp_load_pipelined", "checked_build",
    "check_status", "append_kv", "decode_attention", "decode_workspace", "decode_gave_up", "evict_pages",
    "query_attention", "query_workspace", "prefix_attention", "prefix_workspace", "merge_attention", "MERGE_PARTS",
]

LAYOUT_POOL = -1
LAYER_FIRST = 0
PAGE_FIRST = 1
PAGE_FIRST_DIRECT = 2
PAGE_FIRST_DIRECT_KV = 3
LAYOUTS = {"layer_first": LAYER_FIRST, "page_first": PAGE_FIRST,
           "page_first_direct": PAGE_FIRST_DIRECT, "page_first_direct_kv": PAGE_FIRST_DIRECT_KV}
BACKUP = 0
LOAD = 1
HOST_THP = 0x1

STATUS = {0: "OK", -1: "INVALID_ARG", -2: "INDEX_RANGE", -3: "DUPLICATE_INDEX", -4: "ALIGNMENT",
          -5: "NOT_PINNED", -6: "CUDA", -7: "TIMEOUT", -8: "NOMEM"}

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    """libhicache.so, or the bounds-checked build libhicache_checked.so when
    the environment sets HICACHE_CHECKED=1 before the library is first loaded."""
    if os.environ.get("HICACHE_CHECKED") == "1":
        return os.path.join(_HERE, "libhicache_checked.so")
    return os.path.join(_HERE, "libhicache.so")


class HiCacheError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{STATUS.get(code, code)}: {message}")
        self.code = code
        self.status = STATUS.get(code, str(code))


class PoolDesc(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("num_buffers", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("elem_bytes", ctypes.c_int32),
                ("row_elems", ctypes.c_int64), ("host_num_pages", ctypes.c_int64),
                ("layout", ctypes.c_int32), ("launch_ctas", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _DeviceKVStruct(ctypes.Structure):
    _fields_ = [("buf_ptrs", ctypes.POINTER(ctypes.c_void_p)), ("device_num_pages", ctypes.c_int64)]


_lib = None
_lib_lock = threading.Lock()
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_P = ctypes.POINTER


def _bind(lib):
    sigs = {
        "hicache_version": (_i32, []),
        "hicache_last_error": (ctypes.c_char_p, []),
        "hicache_launch_count": (_i64, []),
        "hicache_host_alloc": (ctypes.c_int, [_sz, _i32, _P(_vp)]),
        "hicache_host_free": (ctypes.c_int, [_vp]),
        "hicache_pool_create": (ctypes.c_int, [_P(PoolDesc), _vp, _sz, _P(_vp)]),
        "hicache_pool_destroy": (ctypes.c_int, [_vp]),
        "hicache_backup": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _vp, _vp, _i64, _i32, _vp]),
        "hicache_load": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _vp, _vp, _i64, _i32, _vp]),
        "hicache_load_layer": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _vp, _vp, _i64, _i32, _i32, _vp]),
        "hicache_backup_load": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _vp, _vp, _i64, _vp, _vp, _i64,
                                               _i32, _vp]),
        "hicache_load_pipelined": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _vp, _vp, _i64, _i32, _vp]),
        "hicache_plan_load_pipelined": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _i32, _vp]),
        "hicache_load_pipelined_noalloc": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _vp, _vp, _i64, _i32, _vp]),
        "hicache_pipeline_status": (ctypes.c_int, [_vp, _i32, _P(ctypes.c_uint32), _P(ctypes.c_uint32)]),
        "hicache_group_transfer": (ctypes.c_int, [_P(_vp), _P(_DeviceKVStruct), _i32, _vp, _vp, _i64, _i32,
                                                  _i32, _i32, _vp]),
        "hicache_group_load_pipelined": (ctypes.c_int, [_P(_vp), _P(_DeviceKVStruct), _i32, _vp, _vp, _i64,
                                                        _i32, _vp]),
        "hicache_group_plan_create": (ctypes.c_int, [_P(_vp), _i32, _vp, _vp, _i64, _i64, _P(_vp)]),
        "hicache_group_plan_execute": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _i32, _i32, _vp]),
        "hicache_group_plan_load_layers": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _i32, _vp]),
        "hicache_group_plan_load_layer_chained": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _i32, _i32, _vp]),
        "hicache_group_plan_destroy": (ctypes.c_int, [_vp]),
        "hicache_plan_create": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i32, _P(_vp)]),
        "hicache_plan_execute": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _i32, _i32, _vp]),
        "hicache_plan_load_layer": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _i32, _i32, _vp]),
        "hicache_plan_load_layers": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _i32, _vp]),
        "hicache_plan_load_layer_chained": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _i32, _i32, _vp]),
        "hicache_plan_info": (ctypes.c_int, [_vp, _P(_i64), _P(_i64)]),
        "hicache_plan_destroy": (ctypes.c_int, [_vp]),
        "hicache_layer_event": (ctypes.c_int, [_vp, _i32, _P(_vp)]),
        "hicache_wait_layer": (ctypes.c_int, [_vp, _i32, _vp]),
        "hicache_wait": (ctypes.c_int, [_vp, _i64]),
        "hicache_stream_copy": (ctypes.c_int, [_vp, _vp, _sz, _i32, _i32, _vp]),
        "hicache_checked_build": (_i32, []),
        "hicache_check_status": (ctypes.c_int, [_P(ctypes.c_uint64), _P(ctypes.c_uint64), _i32]),
        "hicache_tp_share": (ctypes.c_int, [_i64, _i32, _i32, _P(_i64), _P(_i64)]),
        "hicache_pool_layer_counters": (ctypes.c_int, [_vp, _P(_vp)]),
        "hicache_tp_load_pipelined": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _P(_vp), _i32, _i32, _vp, _vp,
                                                     _i64, _i32, _vp]),
        "hicache_prepass": (ctypes.c_int, [_i64, _i64, _vp, _vp, _i64, _i32, _P(_i64), _vp, _i64]),
        "hicache_segment_count": (_i64, [_P(PoolDesc), _vp, _vp, _i64, _i32, _i32]),
        "hicache_page_span": (ctypes.c_int, [_P(PoolDesc), _i64, _i32, _P(_i64), _P(_i64)]),
        "hicache_engine_create": (ctypes.c_int, [_vp, _P(_vp)]),
        "hicache_engine_destroy": (ctypes.c_int, [_vp]),
        "hicache_engine_submit": (ctypes.c_int, [_vp, _P(_DeviceKVStruct), _vp, _vp, _i64, _i32, _i32, _i32,
                                                 _vp, _P(ctypes.c_uint64)]),
        "hicache_engine_wait": (ctypes.c_int, [_vp, ctypes.c_uint64, _i64]),
        "hicache_engine_wait_on_stream": (ctypes.c_int, [_vp, ctypes.c_uint64, _vp]),
        "hicache_engine_stats": (ctypes.c_int, [_vp, _P(_i64), _P(_i64)]),
        "hicache_allocator_create": (ctypes.c_int, [_i64, _P(_vp)]),
        "hicache_allocator_destroy": (ctypes.c_int, [_vp]),
        "hicache_allocator_alloc": (ctypes.c_int, [_vp, _i64, _vp]),
        "hicache_allocator_free": (ctypes.c_int, [_vp, _vp, _i64]),
        "hicache_allocator_available": (_i64, [_vp]),
        "hicache_append_kv": (ctypes.c_int, [_P(_DeviceKVStruct), _P(PoolDesc), _i32, ctypes.c_char_p, _vp]),
        "hicache_decode_attention": (ctypes.c_int, [_P(_DeviceKVStruct), _P(PoolDesc), _i32, ctypes.c_char_p, _vp]),
        "hicache_decode_workspace": (ctypes.c_int, [_P(PoolDesc), _i32, _i32, _i32, _i32, _i32, _i32, _P(_i64)]),
        "hicache_decode_status": (ctypes.c_int, [_vp, _P(_i32), _i32]),
        "hicache_query_attention": (ctypes.c_int, [_P(_DeviceKVStruct), _P(PoolDesc), _i32, ctypes.c_char_p, _vp]),
        "hicache_query_workspace": (ctypes.c_int, [_P(PoolDesc), _i32, _i64, _i32, _i32, _i32, _P(_i64)]),
        "hicache_prefix_attention": (ctypes.c_int, [_P(_DeviceKVStruct), _P(PoolDesc), _i32, ctypes.c_char_p, _vp]),
        "hicache_prefix_workspace": (ctypes.c_int, [_P(PoolDesc), _i32, _i32, _i32, _i32, _i32, _i32, _P(_i64)]),
        "hicache_merge_attention": (ctypes.c_int, [ctypes.c_char_p, _vp]),
        "hicache_evict_pages": (ctypes.c_int, [ctypes.c_char_p, _vp]),
        "hicache_layer_checksum": (ctypes.c_int, [_P(_DeviceKVStruct), _P(PoolDesc), _vp, _i64, _i32,
                                                  _i32, _vp, _vp]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


def library():
    """The loaded libhicache (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lib_lock:
            if _lib is None:
                path = library_path()
                if not os.path.exists(path):
                    raise RuntimeError(
                        f"{path} is missing: build it with tiered_kv_cache_gb300.build.build() "
                        "(there is no fallback path)")
                _lib = _bind(ctypes.CDLL(path))
    return _lib


def _check(rc: int):
    if rc != 0:
        msg = library().hicache_last_error().decode(errors="replace")
        raise HiCacheError(rc, msg)


def _stream(stream) -> int:
    """cudaStream_t handle from None (legacy default), an int, or a torch stream."""
    if stream is None:
        return 0
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _idx(a) -> np.ndarray:
    if type(a) is np.ndarray and a.dtype == np.int64 and a.ndim == 1 and a.flags.c_contiguous:
        return a
    return np.ascontiguousarray(np.asarray(a, dtype=np.int64).reshape(-1))


def _ptr(a: np.ndarray):
    """Address of a contiguous array's data (None when empty).  Through the
    buffer protocol where the array is writable: a third of the cost of
    ndarray.ctypes, which a small call pays twice."""
    if not a.size:
        return None
    if a.flags.writeable:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    return a.ctypes.data


def version() -> int:
    return library().hicache_version()


def launch_count() -> int:
    return library().hicache_launch_count()


def host_alloc(nbytes: int, thp: bool = False) -> int:
    """Page-locked, device-mapped host memory (HICACHE_HOST_THP: mmap + huge
    pages before locking).  Returns the host address."""
    out = ctypes.c_void_p()
    _check(library().hicache_host_alloc(nbytes, HOST_THP if thp else 0, ctypes.byref(out)))
    return out.value


def host_free(ptr: int):
    _check(library().hicache_host_free(ptr))


def wait(stream=None, timeout_us: int = -1):
    """Block until `stream` is idle, for at most timeout_us (raises TIMEOUT)."""
    _check(library().hicache_wait(_stream(stream), timeout_us))

def checked_build() -> bool:
    """True when the loaded library is the bounds-checked build."""
    return bool(library().hicache_checked_build())


def check_status(clear: bool = False):
    """(first failed bounds check, number of failed checks) of the current
    device since the last clear; (0, 0) when every check passed (and always in
    the plain build)."""
    first, count = ctypes.c_uint64(), ctypes.c_uint64()
    _check(library().hicache_check_status(ctypes.byref(first), ctypes.byref(count), int(clear)))
    return first.value, count.value


def tp_share(n: int, tp: int, rank: int):
    """(first, count): the pairs rank `rank` of a tensor-parallel group of tp
    loads out of n, a contiguous part in the caller's order."""
    first, count = ctypes.c_int64(), ctypes.c_int64()
    _check(library().hicache_tp_share(n, tp, rank, ctypes.byref(first), ctypes.byref(count)))
    return first.value, count.value


def tp_load_pipelined(pool, rank_kvs, rank_counters, rank: int, device_pages, host_pages,
                      layout=LAYOUT_POOL, stream=None):
    """This rank's part of a tensor-parallel load of a replicated latent: its
    share of the pages, read from ``pool``'s host memory and stored into every
    rank's buffers (``rank_kvs``), counted into every rank's per-layer
    counters (``rank_counters``: each rank's Pool.layer_counters())."""
    if len(rank_kvs) != len(rank_counters):
        raise ValueError("rank_kvs and rank_counters differ in length")
    dp, hp = _idx(device_pages), _idx(host_pages)
    if dp.size != hp.size:
        raise ValueError("device_pages and host_pages differ in length")
    if isinstance(layout, str):
        layout = LAYOUTS[layout]
    structs = (_DeviceKVStruct * len(rank_kvs))(*[k.struct for k in rank_kvs])
    counters = (ctypes.c_void_p * len(rank_counters))(*rank_counters)
    _check(library().hicache_tp_load_pipelined(pool.handle, structs, counters, len(rank_kvs), rank, _ptr(dp),
                                               _ptr(hp), dp.size, layout, _stream(stream)))


def stream_copy(dst_ptr: int, src_ptr: int, nbytes: int, grid: int = 0, vecs_per_thread: int = 4,
                stream=None):
    """Roofline probe: a plain zero-copy streaming copy of nbytes (no index
    decode) between device memory and/or pinned, mapped host memory."""
    _check(library().hicache_stream_copy(dst_ptr, src_ptr, nbytes, grid, vecs_per_thread, _stream(stream)))


class DeviceKV:
    """B*L device buffer pointers (buffer-major) plus the device pool size in
    pages.  ``tensors`` may be torch tensors (their data_ptr is taken) or raw
    integer addresses; the caller keeps the memory alive."""

    def __init__(self, tensors, device_num_pages: int):
        ptrs = [t if isinstance(t, int) else t.data_ptr() for t in tensors]
        self._arr = (ctypes.c_void_p * len(ptrs))(*ptrs)
        self._tensors = tensors
        self.struct = _DeviceKVStruct(ctypes.cast(self._arr, ctypes.POINTER(ctypes.c_void_p)),
                                      device_num_pages)
        self.ref = ctypes.byref(self.struct)      # made once: every call passes it
        self.device_num_pages = device_num_pages
        self.num_buffers_total = len(ptrs)
        self.checked = set()                      # pool shapes the tensors were checked for


def _desc(num_layers, num_buffers, page_size, row_elems, host_num_pages, layout,
          elem_bytes=2, launch_ctas=0) -> PoolDesc:
    if isinstance(layout, str):
        layout = LAYOUTS[layout]
    return PoolDesc(num_layers, num_buffers, page_size, elem_bytes, row_elems, host_num_pages,
                    layout, launch_ctas, 0, 0)


def prepass(host_num_pages: int, device_num_pages: int, device_pages, host_pages, direction: int):
    """Validate a transfer and return its runs as an (r, 3) int64 array of
    (first host page, first device page, page count)."""
    dp, hp = _idx(device_pages), _idx(host_pages)
    if dp.size != hp.size:
        raise ValueError("device_pages and host_pages differ in length")
    nr = ctypes.c_int64()
    out = np.zeros((max(1, dp.size), 3), np.int64)
    _check(library().hicache_prepass(host_num_pages, device_num_pages, _ptr(dp), _ptr(hp), dp.size,
                                     direction, ctypes.byref(nr), out.ctypes.data, out.shape[0]))
    return out[: nr.value].copy()


def segment_count(num_layers, num_buffers, page_size, row_elems, host_num_pages, layout,
                  device_pages, host_pages, layer: int = -1, elem_bytes: int = 2) -> int:
    d = _desc(num_layers, num_buffers, page_size, row_elems, host_num_pages, layout, elem_bytes)
    dp, hp = _idx(device_pages), _idx(host_pages)
    r = library().hicache_segment_count(ctypes.byref(d), _ptr(dp), _ptr(hp), dp.size, d.layout, layer)
    if r < 0:
        _check(int(r))
    return int(r)


def page_span(desc: PoolDesc, host_page: int, buffer: int = -1):
    """(offset, nbytes) of one host page's contiguous span in the host pool."""
    off, nb = ctypes.c_int64(), ctypes.c_int64()
    _check(library().hicache_page_span(ctypes.byref(desc), host_page, buffer, ctypes.byref(off),
                                       ctypes.byref(nb)))
    return off.value, nb.value


def layer_checksum(kv: DeviceKV, pool_or_desc, device_pages, layer: int, out_ptr: int,
                   reps: int = 1, stream=None):
    """Stand-in attention: adds the 32-bit words of `layer` of the given device
    pages (every buffer, `reps` passes) into the device uint64 at out_ptr."""
    desc = pool_or_desc.desc if isinstance(pool_or_desc, Pool) else pool_or_desc
    dp = _idx(device_pages)
    _check(library().hicache_layer_checksum(kv.ref, ctypes.byref(desc), _ptr(dp),
                                            dp.size, layer, reps, out_ptr, _stream(stream)))


MAX_GROUP = 4


def group_transfer(pools, kvs, device_pages, host_pages, direction: int, layer: int = -1,
                   layout=LAYOUT_POOL, stream=None):
    """Move the same page pairs for several pools (buffer kinds with different
    rows that share the page numbering) in one launch.  ``layer`` >= 0 loads
    that layer alone and records its event in every pool."""
    if len(pools) != len(kvs):
        raise ValueError("pools and kvs differ in length")
    dp, hp = _idx(device_pages), _idx(host_pages)
    if dp.size != hp.size:
        raise ValueError("device_pages and host_pages differ in length")
    if isinstance(layout, str):
        layout = LAYOUTS[layout]
    handles = (ctypes.c_void_p * len(pools))(*[p.handle for p in pools])
    structs = (_DeviceKVStruct * len(kvs))(*[k.struct for k in kvs])
    _check(library().hicache_group_transfer(handles, structs, len(pools), _ptr(dp), _ptr(hp), dp.size,
                                            layout, layer, direction, _stream(stream)))


def group_load_pipelined(pools, kvs, device_pages, host_pages, layout=LAYOUT_POOL, stream=None):
    """Every layer of every pool of a group in one launch, layer by layer;
    each pool's wait_layer then waits for that pool's layer alone."""
    if len(pools) != len(kvs):
        raise ValueError("pools and kvs differ in length")
    dp, hp = _idx(device_pages), _idx(host_pages)
    if dp.size != hp.size:
        raise ValueError("device_pages and host_pages differ in length")
    if isinstance(layout, str):
        layout = LAYOUTS[layout]
    handles = (ctypes.c_void_p * len(pools))(*[p.handle for p in pools])
    structs = (_DeviceKVStruct * len(kvs))(*[k.struct for k in kvs])
    _check(library().hicache_group_load_pipelined(handles, structs, len(pools), _ptr(dp), _ptr(hp), dp.size,
                                                  layout, _stream(stream)))


class GroupPlan:
    """A load plan for a buffer group: the page pairs pre-passed once for
    pools that share the page numbering, then loaded every layer at once, one
    layer, or layer by layer from a CUDA graph."""

    def __init__(self, pools, device_pages, host_pages, device_num_pages: int):
        dp, hp = _idx(device_pages), _idx(host_pages)
        if dp.size != hp.size:
            raise ValueError("device_pages and host_pages differ in length")
        handles = (ctypes.c_void_p * len(pools))(*[p.handle for p in pools])
        h = ctypes.c_void_p()
        _check(library().hicache_group_plan_create(handles, len(pools), _ptr(dp), _ptr(hp), dp.size,
                                                   device_num_pages, ctypes.byref(h)))
        self.pools = list(pools)
        self.handle = h.value

    def _kvs(self, kvs):
        if len(kvs) != len(self.pools):
            raise ValueError("one DeviceKV per pool of the plan")
        return (_DeviceKVStruct * len(kvs))(*[k.struct for k in kvs])

    def execute(self, kvs, layer: int = -1, layout=LAYOUT_POOL, stream=None):
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        _check(library().hicache_group_plan_execute(self.handle, self._kvs(kvs), layout, layer,
                                                    _stream(stream)))

    def load_layers(self, kvs, layout=LAYOUT_POOL, stream=None):
        """Every layer, layer by layer, each followed by its event in every
        pool, replayed from a CUDA graph the plan captures on first use."""
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        _check(library().hicache_group_plan_load_layers(self.handle, self._kvs(kvs), layout,
                                                        _stream(stream)))

    def load_layer_chained(self, kvs, layer: int, layout=LAYOUT_POOL, stream=None):
        """One layer of every pool in one launch, chained to this plan's
        previous layer on the same stream (nothing else on that stream in
        between); each pool's wait_layer waits for it on the device."""
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        _check(library().hicache_group_plan_load_layer_chained(self.handle, self._kvs(kvs), layout, layer,
                                                               _stream(stream)))

    def close(self):
        if getattr(self, "handle", None):
            library().hicache_group_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def group_plan(pools, device_pages, host_pages, device_num_pages: int) -> GroupPlan:
    return GroupPlan(pools, device_pages, host_pages, device_num_pages)


class PinnedHost:
    """Pinned host memory from host_alloc, freed when the last reference (the
    pool, or any numpy view of it) goes away."""

    def __init__(self, nbytes: int, thp: bool = False):
        self.nbytes = nbytes
        self.ptr = host_alloc(nbytes, thp)

    def free(self):
        if self.ptr:
            ptr, self.ptr = self.ptr, None
            host_free(ptr)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class Pool:
    """A host L2 pool of ``host_num_pages`` pages in one layout.

    If ``host_ptr`` is None the pool allocates its pinned memory with
    host_alloc (``thp`` selects the huge-page path); that memory lives as long
    as the pool or any array returned by host_array()."""

    def __init__(self, num_layers: int, num_buffers: int, page_size: int, row_elems: int,
                 host_num_pages: int, layout="layer_first", elem_bytes: int = 2,
                 host_ptr: int | None = None, host_bytes: int | None = None,
                 launch_ctas: int = 0, thp: bool = False):
        self.desc = _desc(num_layers, num_buffers, page_size, row_elems, host_num_pages, layout,
                          elem_bytes, launch_ctas)
        self.num_layers, self.num_buffers, self.page_size = num_layers, num_buffers, page_size
        self.row_elems, self.host_num_pages, self.elem_bytes = row_elems, host_num_pages, elem_bytes
        self.layout = self.desc.layout
        self.nbytes = num_buffers * num_layers * host_num_pages * page_size * row_elems * elem_bytes
        self._mem = PinnedHost(self.nbytes, thp) if host_ptr is None else None
        self.host_ptr = self._mem.ptr if host_ptr is None else host_ptr
        self.host_bytes = self.nbytes if host_bytes is None else host_bytes
        h = ctypes.c_void_p()
        _check(library().hicache_pool_create(ctypes.byref(self.desc), self.host_ptr,
                                             self.host_bytes, ctypes.byref(h)))
        self.handle = h.value

    def host_array(self, dtype=np.uint16) -> np.ndarray:
        """numpy view of the host pool (no copy); keeps the memory alive."""
        buf = (ctypes.c_uint8 * self.nbytes).from_address(self.host_ptr)
        buf._owner = self._mem
        return np.frombuffer(buf, dtype=np.uint8).view(dtype)

    def _xfer(self, fn, kv: DeviceKV, device_pages, host_pages, layout, stream, *extra):
        dp, hp = _idx(device_pages), _idx(host_pages)
        if dp.size != hp.size:
            raise ValueError("device_pages and host_pages differ in length")
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        rc = fn(self.handle, kv.ref, _ptr(dp), _ptr(hp), dp.size, layout, *extra, _stream(stream))
        if rc:
            _check(rc)

    def backup(self, kv: DeviceKV, device_pages, host_pages, layout=LAYOUT_POOL, stream=None):
        self._xfer(library().hicache_backup, kv, device_pages, host_pages, layout, stream)

    def load(self, kv: DeviceKV, device_pages, host_pages, layout=LAYOUT_POOL, stream=None):
        self._xfer(library().hicache_load, kv, device_pages, host_pages, layout, stream)

    def load_pipelined(self, kv: DeviceKV, device_pages, host_pages, layout=LAYOUT_POOL, stream=None):
        """Every layer in one launch, each layer marked done on the device as it
        lands (wait_layer then waits for that layer alone)."""
        self._xfer(library().hicache_load_pipelined, kv, device_pages, host_pages, layout, stream)

    def load_layer(self, kv: DeviceKV, device_pages, host_pages, layer: int, layout=LAYOUT_POOL,
                   stream=None):
        self._xfer(library().hicache_load_layer, kv, device_pages, host_pages, layout, stream, layer)

    def backup_load(self, kv: DeviceKV, backup_device_pages, backup_host_pages, load_device_pages,
                    load_host_pages, layout=LAYOUT_POOL, stream=None):
        """A backup and a load in one launch (both directions of the link at once)."""
        bd, bh = _idx(backup_device_pages), _idx(backup_host_pages)
        ld, lh = _idx(load_device_pages), _idx(load_host_pages)
        if bd.size != bh.size or ld.size != lh.size:
            raise ValueError("device and host page lists differ in length")
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        _check(library().hicache_backup_load(self.handle, kv.ref, _ptr(bd), _ptr(bh), bd.size,
                                             _ptr(ld), _ptr(lh), ld.size, layout, _stream(stream)))

    def page_span(self, host_page: int, buffer: int = -1):
        return page_span(self.desc, host_page, buffer)

    def page_view(self, host_page: int, buffer: int = -1) -> np.ndarray:
        """The bytes of one host page (no copy), ready for an L3 write."""
        off, nb = self.page_span(host_page, buffer)
        return self.host_array(np.uint8)[off:off + nb]

    def pipeline_status(self, layer: int):
        """(counter now, value it will reach) for a layer's pipelined loads."""
        d, t = ctypes.c_uint32(), ctypes.c_uint32()
        _check(library().hicache_pipeline_status(self.handle, layer, ctypes.byref(d), ctypes.byref(t)))
        return d.value, t.value

    def layer_counters(self) -> int:
        """Device address of the pool's per-layer counters (for the other ranks
        of a tensor-parallel load)."""
        out = ctypes.c_void_p()
        _check(library().hicache_pool_layer_counters(self.handle, ctypes.byref(out)))
        return out.value

    def wait_layer(self, layer: int, compute_stream=None):
        _check(library().hicache_wait_layer(self.handle, layer, _stream(compute_stream)))

    def layer_event(self, layer: int) -> int:
        ev = ctypes.c_void_p()
        _check(library().hicache_layer_event(self.handle, layer, ctypes.byref(ev)))
        return ev.value

    def plan(self, device_pages, host_pages, device_num_pages: int, direction: int) -> "Plan":
        return Plan(self, device_pages, host_pages, device_num_pages, direction)

    def close(self):
        if getattr(self, "handle", None):
            _check(library().hicache_pool_destroy(self.handle))
            self.handle = None
        self._mem = None   # freed once no host_array view is left

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Engine:
    """Submission engine over a pool (hicache_engine_*): queue backups and loads,
    one worker thread launches them in order, fusing adjacent opposite-direction
    requests into one launch."""

    def __init__(self, pool: "Pool"):
        h = ctypes.c_void_p()
        _check(library().hicache_engine_create(pool.handle, ctypes.byref(h)))
        self.handle = h.value
        self.pool = pool
        self._kvs = []

    def submit(self, kv: DeviceKV, device_pages, host_pages, direction: int, layout=LAYOUT_POOL,
               after_stream=None) -> int:
        dp, hp = _idx(device_pages), _idx(host_pages)
        if dp.size != hp.size:
            raise ValueError("device_pages and host_pages differ in length")
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        t = ctypes.c_uint64()
        _check(library().hicache_engine_submit(self.handle, kv.ref, _ptr(dp), _ptr(hp), dp.size,
                                               direction, layout, 0 if after_stream is None else 1,
                                               _stream(after_stream), ctypes.byref(t)))
        return t.value

    def wait(self, ticket: int, timeout_us: int = -1):
        _check(library().hicache_engine_wait(self.handle, ticket, timeout_us))

    def wait_on_stream(self, ticket: int, stream=None):
        _check(library().hicache_engine_wait_on_stream(self.handle, ticket, _stream(stream)))

    def stats(self):
        a, b = ctypes.c_int64(), ctypes.c_int64()
        _check(library().hicache_engine_stats(self.handle, ctypes.byref(a), ctypes.byref(b)))
        return a.value, b.value

    def close(self):
        if getattr(self, "handle", None):
            h, self.handle = self.handle, None
            _check(library().hicache_engine_destroy(h))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PageAllocator:
    """LIFO host-page allocator (hicache_allocator_*)."""

    def __init__(self, num_pages: int):
        h = ctypes.c_void_p()
        _check(library().hicache_allocator_create(num_pages, ctypes.byref(h)))
        self.handle = h.value
        self.num_pages = num_pages

    def alloc(self, n: int) -> np.ndarray:
        out = np.empty(n, np.int64)
        _check(library().hicache_allocator_alloc(self.handle, n, _ptr(out)))
        return out

    def free(self, pages):
        p = _idx(pages)
        _check(library().hicache_allocator_free(self.handle, _ptr(p), p.size))

    @property
    def available(self) -> int:
        r = library().hicache_allocator_available(self.handle)
        if r < 0:
            _check(int(r))
        return int(r)

    def close(self):
        if getattr(self, "handle", None):
            library().hicache_allocator_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Plan:
    """A validated, pre-passed transfer that can be executed many times (e.g.
    once per layer)."""

    def __init__(self, pool: Pool, device_pages, host_pages, device_num_pages: int, direction: int):
        dp, hp = _idx(device_pages), _idx(host_pages)
        if dp.size != hp.size:
            raise ValueError("device_pages and host_pages differ in length")
        h = ctypes.c_void_p()
        _check(library().hicache_plan_create(pool.handle, _ptr(dp), _ptr(hp), dp.size,
                                             device_num_pages, direction, ctypes.byref(h)))
        self.pool = pool
        self.handle = h.value

    def execute(self, kv: DeviceKV, layer: int = -1, layout=LAYOUT_POOL, stream=None):
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        _check(library().hicache_plan_execute(self.handle, kv.ref, layout, layer,
                                              _stream(stream)))

    def load_layers(self, kv: DeviceKV, layout=LAYOUT_POOL, stream=None):
        """Every layer, layer by layer, each followed by its layer event, replayed
        from a CUDA graph the plan captures on first use."""
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        _check(library().hicache_plan_load_layers(self.handle, kv.ref, layout,
                                                  _stream(stream)))

    def load_layer(self, kv: DeviceKV, layer: int, layout=LAYOUT_POOL, stream=None):
        """Load one layer of a load plan and record that layer's event."""
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        _check(library().hicache_plan_load_layer(self.handle, kv.ref, layout, layer,
                                                 _stream(stream)))

    def load_layer_chained(self, kv: DeviceKV, layer: int, layout=LAYOUT_POOL, stream=None):
        """Load one layer, chained to this plan's previous layer on the same
        stream (nothing else may go on that stream in between); the pool's
        wait_layer waits for it on the device."""
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        _check(library().hicache_plan_load_layer_chained(self.handle, kv.ref, layout, layer,
                                                         _stream(stream)))

    def load_pipelined(self, kv: DeviceKV, layout=LAYOUT_POOL, stream=None):
        if isinstance(layout, str):
            layout = LAYOUTS[layout]
        _check(library().hicache_plan_load_pipelined(self.handle, kv.ref, layout,
                                                     _stream(stream)))

    def info(self):
        n, r = ctypes.c_int64(), ctypes.c_int64()
        _check(library().hicache_plan_info(self.handle, ctypes.byref(n), ctypes.byref(r)))
        return n.value, r.value

    def close(self):
        if getattr(self, "handle", None):
            library().hicache_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- operators on the device pages ------------------------------------------------
# The descriptors of include/hicache.h, field by field in their order there.
_APPEND_DESC = struct.Struct("9P10q9i3f")
_DECODE_DESC = struct.Struct("7P8q8i4f")
_EVICT_DESC = struct.Struct("9P5q6i")
_QUERY_DESC = struct.Struct("7P8q8i3f")
_PREFIX_DESC = struct.Struct("9P8q8i3f")
_MERGE_DESC = struct.Struct("18P28q4i")
MERGE_PARTS = 8
BF16 = 0
FP16 = 1


def _tensor(name, t, dtype, shape, device):
    """Checks a torch tensor argument (type, shape, device index, a contiguous
    innermost dimension) and returns its strides."""
    strides = t.stride()
    if (t.dtype is dtype and t.shape == shape and t.get_device() == device
            and (strides[-1] == 1 or shape[-1] <= 1)):
        return strides
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, expected device {device}")
    raise ValueError(f"{name}: the innermost dimension must be contiguous")


def _written(name, t):
    """Refuses to write a tensor that requires grad while autograd records: it would
    not see it."""
    if _torch.is_grad_enabled():
        raise ValueError(f"{name}: written, but requires grad (these operators have no backward pass; use torch.no_grad())")


_torch = None


def _import_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _activations(name, t):
    """(dtype code, device index) of the tensor that decides both for a call: a
    [n, heads, dim] tensor on the current CUDA device."""
    torch = _import_torch()
    dt = t.dtype
    code = BF16 if dt is torch.bfloat16 else FP16 if dt is torch.float16 else -1
    if code < 0:
        raise ValueError(f"{name}: {dt}, expected bfloat16 or float16")
    if t.dim() != 3:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected 3")
    return code, _current(name, t)


def _current(name, t):
    device = t.get_device()
    if device < 0 or device != _torch._C._cuda_getDevice():
        raise ValueError(f"{name}: on {t.device}, expected the current CUDA device")
    return device


def _launch_stream(stream, device):
    """The handle of a stream as _stream() takes it, but for None: these calls take
    tensors that torch has just made, so torch's current stream (without its
    wrapper object, which costs a microsecond)."""
    return _torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _pool_desc(pool_or_desc) -> PoolDesc:
    return pool_or_desc.desc if isinstance(pool_or_desc, Pool) else pool_or_desc


def _check_cache(kv, desc, layer, device, dtype=None):
    """The cache must hold desc's buffers; its torch tensors must be on the
    call's device, hold the pages they are said to (raw addresses cannot be
    checked) and have elements of dtype, e4m3 in a 1-byte cache (or of no
    floating-point type: plain storage).  What kv has been checked for is not
    checked again."""
    layers, buffers, row_bytes = desc.num_layers, desc.num_buffers, desc.page_size * desc.row_elems * desc.elem_bytes
    shape = (layers, buffers, row_bytes, desc.elem_bytes, device, dtype)
    if shape in kv.checked:
        return buffers
    if kv.num_buffers_total != buffers * layers:
        raise ValueError(f"DeviceKV has {kv.num_buffers_total} buffers, the pool {buffers} x {layers}")
    if desc.elem_bytes == 1:
        dtype = _import_torch().float8_e4m3fn
    need = kv.device_num_pages * row_bytes
    for t in kv._tensors:
        if isinstance(t, int):
            continue
        if t.get_device() != device:
            raise ValueError(f"the cache is on {t.device}, expected device {device}")
        if t.numel() * t.element_size() < need or not t.is_contiguous():
            raise ValueError(f"a cache buffer has {t.numel() * t.element_size()} bytes, its pages need {need} contiguous")
        if dtype is not None and t.dtype is not dtype and t.dtype.is_floating_point:
            raise ValueError(f"a cache buffer is {t.dtype}, expected {dtype}")
    kv.checked.add(shape)
    return buffers


def append_kv(kv: DeviceKV, pool_or_desc, layer: int, q, k, v, slots, *, q_out=None, positions=None, cos_sin=None,
              rot_offset: int = 0, interleaved: bool = False, q_weight=None, k_weight=None, eps: float = 1e-6,
              k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Norms of the query and key heads (over the first len(weight) elements;
    none without a weight), the rotation of cos_sin.shape[1] elements from
    rot_offset on by row positions[n] of cos_sin (cosines, then sines), and the
    store of k and v into rows slots[n] of the layer's buffers.

    q [n, q_heads, dim] -> q_out (None: in place); k, v [n, kv_heads, dim] (v is
    None for a latent cache).  q, or k and v and slots, may be None.  stream: torch's
    current stream unless given."""
    torch = _import_torch()
    first = q if q is not None else k
    if first is None:
        raise ValueError("q and k are both None")
    code, dev = _activations("q" if q is not None else "k", first)
    dt = first.dtype
    desc = _pool_desc(pool_or_desc)
    buffers = _check_cache(kv, desc, layer, dev, dt)
    n, hq, dim = first.shape
    qp = op = kp = vp = qst = qsh = ost = osh = kst = ksh = vst = vsh = hk = sp = 0
    if q is not None:
        qst, qsh, _ = _tensor("q", q, dt, (n, hq, dim), dev)
        qp = op = q.data_ptr()
        ost, osh = qst, qsh
        if q_out is not None:
            ost, osh, _ = _tensor("q_out", q_out, dt, (n, hq, dim), dev)
            op = q_out.data_ptr()
            if q_out.requires_grad:
                _written("q_out", q_out)
        elif q.requires_grad:
            _written("q", q)
    else:
        hq = 0
    if k is not None:
        hk = k.shape[1] if k.dim() == 3 else 0
        kst, ksh, _ = _tensor("k", k, dt, (n, hk, dim), dev)
        kp = k.data_ptr()
        if (v is None) != (buffers == 1):
            raise ValueError("a K, V cache takes v, a latent cache none")
        if v is not None:
            vst, vsh, _ = _tensor("v", v, dt, (n, hk, dim), dev)
            vp = v.data_ptr()
        _tensor("slots", slots, torch.int64, (n,), dev)
        sp = slots.data_ptr()
    elif v is not None:
        raise ValueError("v without k")
    qw = kw = qn = kn = 0
    if q_weight is not None:
        qn = q_weight.numel()
        _tensor("q_weight", q_weight, dt, (qn,), dev)
        qw = q_weight.data_ptr()
    if k_weight is not None:
        kn = k_weight.numel()
        _tensor("k_weight", k_weight, dt, (kn,), dev)
        kw = k_weight.data_ptr()
    pp = cp = rows = rot = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be contiguous, of two dimensions")
        rows, rot = cos_sin.shape
        _tensor("cos_sin", cos_sin, torch.float32, (rows, rot), dev)
        if positions is None:
            raise ValueError("cos_sin without positions")
        _tensor("positions", positions, torch.int64, (n,), dev)
        pp, cp = positions.data_ptr(), cos_sin.data_ptr()
    a = _APPEND_DESC.pack(qp, op, kp, vp, qw, kw, sp, pp, cp, qst, qsh, ost, osh, kst, ksh, vst, vsh, n, rows,
                          code, hq, hk, dim, qn, kn, rot, rot_offset, bool(interleaved), eps, k_scale, v_scale)
    rc = library().hicache_append_kv(kv.ref, ctypes.byref(desc), layer, a, _launch_stream(stream, dev))
    if rc:
        _check(rc)


def decode_workspace(pool_or_desc, batch: int, q_heads: int, head_dim: int, v_dim: int, max_pages: int,
                     weights: bool = False) -> int:
    """Bytes of workspace a decode_attention of these sizes needs.  Zero-fill
    it once; calls that may run at the same time need one each."""
    out = ctypes.c_int64()
    _check(library().hicache_decode_workspace(ctypes.byref(_pool_desc(pool_or_desc)), batch, q_heads, head_dim, v_dim,
                                              max_pages, int(weights), ctypes.byref(out)))
    return out.value


def decode_attention(kv: DeviceKV, pool_or_desc, layer: int, q, page_table, seq_lens, out, workspace, *, scale=None,
                     window: int = 0, weights=None, decay: float = 1.0, lse=None, k_scale: float = 1.0,
                     v_scale: float = 1.0, stream=None):
    """Attention of one new token per sequence: q [batch, q_heads, head_dim]
    over the first seq_lens[b] tokens of the pages page_table[b] (int32; the last
    `window` of them if window > 0) into out [batch, q_heads, v_dim]; lse
    (optional) [batch, q_heads] the log of the softmax sums; weights (optional)
    [batch, max_pages] <- decay * weights + the attention each page received.
    scale: head_dim ** -0.5 unless given; stream: torch's current stream unless
    given."""
    torch = _import_torch()
    code, dev = _activations("q", q)
    dt = q.dtype
    desc = _pool_desc(pool_or_desc)
    _check_cache(kv, desc, layer, dev, dt)
    b, hq, d = q.shape
    qb, qh, _ = _tensor("q", q, dt, (b, hq, d), dev)
    dv, width = out.shape[-1], page_table.shape[-1]
    ob, oh, _ = _tensor("out", out, dt, (b, hq, dv), dev)
    if out.requires_grad:
        _written("out", out)
    tst = _tensor("page_table", page_table, torch.int32, (b, width), dev)[0]
    _tensor("seq_lens", seq_lens, torch.int32, (b,), dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: must be contiguous and on device {dev}")
    lp = wp = lst = wst = 0
    if lse is not None:
        lst = _tensor("lse", lse, torch.float32, (b, hq), dev)[0]
        if lse.requires_grad:
            _written("lse", lse)
        lp = lse.data_ptr()
    if weights is not None:
        wst = _tensor("weights", weights, torch.float32, (b, width), dev)[0]
        if weights.requires_grad:
            _written("weights", weights)
        wp = weights.data_ptr()
    a = _DECODE_DESC.pack(q.data_ptr(), out.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), lp, wp,
                          workspace.data_ptr(), workspace.numel() * workspace.element_size(), qb, qh, ob, oh,
                          tst, lst, wst, code, b, hq, d, dv, width, window, 0,
                          d ** -0.5 if scale is None else scale, k_scale, v_scale, decay)
    rc = library().hicache_decode_attention(kv.ref, ctypes.byref(desc), layer, a, _launch_stream(stream, dev))
    if rc:
        _check(rc)


def decode_gave_up(workspace, clear: bool = False) -> bool:
    """Whether a call with this workspace gave up waiting (it never should): its
    outputs are undefined then.  Waits for all work of the current device."""
    out = ctypes.c_int32()
    _check(library().hicache_decode_status(workspace.data_ptr(), ctypes.byref(out), int(clear)))
    return bool(out.value)


def query_workspace(pool_or_desc, batch: int, tokens: int, q_heads: int, head_dim: int, max_pages: int) -> int:
    """Bytes of workspace a query_attention of these sizes needs.  Zero-fill it
    once; calls that may run at the same time need one each."""
    out = ctypes.c_int64()
    _check(library().hicache_query_workspace(ctypes.byref(_pool_desc(pool_or_desc)), batch, tokens, q_heads, head_dim,
                                             max_pages, ctypes.byref(out)))
    return out.value


def query_attention(kv: DeviceKV, pool_or_desc, layer: int, q, q_starts, page_table, kv_lens, out, workspace, *,
                    causal: bool = False, scale=None, window: int = 0, lse=None, k_scale: float = 1.0,
                    v_scale: float = 1.0, stream=None):
    """Attention of several query tokens per sequence: sequence b has the tokens
    [q_starts[b], q_starts[b + 1]) (int32 [batch + 1]) of q [tokens, q_heads,
    head_dim] and kv_lens[b] cached ones on the pages page_table[b].  Each query
    attends to all of these (cross attention), or, causal, to those up to its own
    place when the sequence's queries are its last tokens (the last `window` of them
    if window > 0).  out as q; lse (optional) [tokens, q_heads]; rows of no sequence
    are left as they were.  V of the cached tokens must be finite.  scale: head_dim ** -0.5 unless given; stream: torch's
    current stream unless given."""
    torch = _import_torch()
    code, dev = _activations("q", q)
    dt = q.dtype
    desc = _pool_desc(pool_or_desc)
    _check_cache(kv, desc, layer, dev, dt)
    n, hq, d = q.shape
    qt, qh, _ = _tensor("q", q, dt, (n, hq, d), dev)
    b, width = kv_lens.shape[0], page_table.shape[-1]
    ot, oh, _ = _tensor("out", out, dt, (n, hq, d), dev)
    if out.requires_grad:
        _written("out", out)
    tst = _tensor("page_table", page_table, torch.int32, (b, width), dev)[0]
    _tensor("q_starts", q_starts, torch.int32, (b + 1,), dev)
    _tensor("kv_lens", kv_lens, torch.int32, (b,), dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: must be contiguous and on device {dev}")
    lp = lst = 0
    if lse is not None:
        lst = _tensor("lse", lse, torch.float32, (n, hq), dev)[0]
        if lse.requires_grad:
            _written("lse", lse)
        lp = lse.data_ptr()
    a = _QUERY_DESC.pack(q.data_ptr(), out.data_ptr(), q_starts.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(),
                         lp, workspace.data_ptr(), workspace.numel() * workspace.element_size(), qt, qh, ot, oh, tst,
                         lst, n, code, b, hq, d, width, window, bool(causal), 0, d ** -0.5 if scale is None else scale,
                         k_scale, v_scale)
    rc = library().hicache_query_attention(kv.ref, ctypes.byref(desc), layer, a, _launch_stream(stream, dev))
    if rc:
        _check(rc)


def prefix_workspace(pool_or_desc, batch: int, groups: int, q_heads: int, head_dim: int, max_prefix_pages: int,
                     max_pages: int) -> int:
    """Bytes of workspace a prefix_attention of these sizes needs.  Zero-fill it
    once; calls that may run at the same time need one each."""
    out = ctypes.c_int64()
    _check(library().hicache_prefix_workspace(ctypes.byref(_pool_desc(pool_or_desc)), batch, groups, q_heads, head_dim,
                                              max_prefix_pages, max_pages, ctypes.byref(out)))
    return out.value


def prefix_attention(kv: DeviceKV, pool_or_desc, layer: int, q, group_starts, prefix_table, prefix_lens, page_table,
                     seq_lens, out, workspace, *, scale=None, lse=None, k_scale: float = 1.0, v_scale: float = 1.0,
                     stream=None):
    """decode_attention where sequences share a prefix: the sequences
    [group_starts[g], group_starts[g + 1]) (int32 [groups + 1]) attend to the
    prefix_lens[g] tokens on the pages prefix_table[g], read once for all of them,
    and each to the seq_lens[b] tokens on its own pages page_table[b].  Sequences of
    no group have their own tokens alone, and there may be no group (arrays of 0 rows, and
    one start).  The faster call where reading the prefix for each sequence takes over
    some 270 MB (8 sequences on 8,192 tokens with rows of 2 KB); below, decode_attention is.  out as q [batch, q_heads, head_dim]; lse
    (optional) [batch, q_heads] over both.  scale: head_dim ** -0.5 unless given;
    stream: torch's current stream unless given."""
    torch = _import_torch()
    code, dev = _activations("q", q)
    dt, i32 = q.dtype, torch.int32
    desc = _pool_desc(pool_or_desc)
    _check_cache(kv, desc, layer, dev, dt)
    b, hq, d = q.shape
    qb, qh, _ = _tensor("q", q, dt, (b, hq, d), dev)
    groups, wide, width = prefix_lens.shape[0], prefix_table.shape[-1], page_table.shape[-1]
    ob, oh, _ = _tensor("out", out, dt, (b, hq, d), dev)
    if out.requires_grad:
        _written("out", out)
    pst = _tensor("prefix_table", prefix_table, i32, (groups, wide), dev)[0]
    _tensor("group_starts", group_starts, i32, (groups + 1,), dev)
    _tensor("prefix_lens", prefix_lens, i32, (groups,), dev)
    tst = _tensor("page_table", page_table, i32, (b, width), dev)[0]
    _tensor("seq_lens", seq_lens, i32, (b,), dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: must be contiguous and on device {dev}")
    lp = lst = 0
    if lse is not None:
        lst = _tensor("lse", lse, torch.float32, (b, hq), dev)[0]
        if lse.requires_grad:
            _written("lse", lse)
        lp = lse.data_ptr()
    a = _PREFIX_DESC.pack(q.data_ptr(), out.data_ptr(), group_starts.data_ptr(), prefix_table.data_ptr(),
                          prefix_lens.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), lp, workspace.data_ptr(),
                          workspace.numel() * workspace.element_size(), qb, qh, ob, oh, pst, tst, lst, code, b, groups,
                          hq, d, wide, width, 0, d ** -0.5 if scale is None else scale, k_scale, v_scale)
    rc = library().hicache_prefix_attention(kv.ref, ctypes.byref(desc), layer, a, _launch_stream(stream, dev))
    if rc:
        _check(rc)


def merge_attention(outs, lses, out, *, lse=None, stream=None):
    """Results over parts of the tokens, joined: outs and lses are sequences of up
    to MERGE_PARTS results [tokens, heads, dim] and their log-sums [tokens, heads];
    out (which may be one of outs) and lse (optional) are those over all parts.  A part whose
    log-sum is -infinity counts for nothing.  stream: torch's current stream unless
    given."""
    torch = _import_torch()
    parts = len(outs)
    if not 1 <= parts <= MERGE_PARTS or len(lses) != parts:
        raise ValueError(f"{parts} outs and {len(lses)} lses, expected 1 to {MERGE_PARTS} of each")
    code, dev = _activations("out", out)
    dt = out.dtype
    n, h, d = shape = out.shape
    ot, oh, _ = _tensor("out", out, dt, (n, h, d), dev)
    if out.requires_grad:
        _written("out", out)
    rest = [0] * (MERGE_PARTS - parts)
    strides = [_tensor("a part of outs", x, dt, shape, dev) for x in outs]
    rows = [_tensor("a part of lses", x, torch.float32, (n, h), dev)[0] for x in lses]
    lp = lst = 0
    if lse is not None:
        lst = _tensor("lse", lse, torch.float32, (n, h), dev)[0]
        if lse.requires_grad:
            _written("lse", lse)
        lp = lse.data_ptr()
    a = _MERGE_DESC.pack(*[x.data_ptr() for x in outs], *rest, *[x.data_ptr() for x in lses], *rest, out.data_ptr(), lp,
                         *[s[0] for s in strides], *rest, *[s[1] for s in strides], *rest, *rows, *rest, ot, oh, lst, n,
                         code, parts, h, d)
    rc = library().hicache_merge_attention(a, _launch_stream(stream, dev))
    if rc:
        _check(rc)


def evict_pages(page_size: int, page_table, seq_lens, weights, keep, victims, num_victims, *, sink: int = 0,
                recent: int = 1, out_table=None, out_lens=None, out_weights=None, stream=None):
    """Of each sequence's pages in [sink, n - recent) that are present (entries
    below 0 are absent pages, which keep their place), the ones with the lowest
    weights leave until keep[b] are left (or none may go, or victims is full):
    victims [batch, max_victims] receives their pages, num_victims their number,
    and out_table, out_lens, out_weights (None: in place) what stays.  stream:
    torch's current stream unless given."""
    torch = _import_torch()
    dev = _current("page_table", page_table)
    i32, f32 = torch.int32, torch.float32
    if page_table.dim() != 2 or victims.dim() != 2:
        raise ValueError("page_table and victims must have two dimensions")
    b, width = page_table.shape
    rows, one = (b, width), (b,)
    cap = victims.shape[1]
    tst = _tensor("page_table", page_table, i32, rows, dev)[0]
    wst = _tensor("weights", weights, f32, rows, dev)[0]
    _tensor("seq_lens", seq_lens, i32, one, dev)
    _tensor("keep", keep, i32, one, dev)
    _tensor("num_victims", num_victims, i32, one, dev)
    vst = _tensor("victims", victims, i32, (b, cap), dev)[0]
    tp = otp = page_table.data_ptr()
    wp = owp = weights.data_ptr()
    lp = olp = seq_lens.data_ptr()
    otst, owst = tst, wst
    if out_table is not None:
        otst = _tensor("out_table", out_table, i32, rows, dev)[0]
        otp = out_table.data_ptr()
    if out_weights is not None:
        owst = _tensor("out_weights", out_weights, f32, rows, dev)[0]
        owp = out_weights.data_ptr()
        if out_weights.requires_grad:
            _written("out_weights", out_weights)
    elif weights.requires_grad:
        _written("weights", weights)
    if out_lens is not None:
        _tensor("out_lens", out_lens, i32, one, dev)
        olp = out_lens.data_ptr()
    a = _EVICT_DESC.pack(tp, wp, lp, keep.data_ptr(), victims.data_ptr(), num_victims.data_ptr(), otp, owp, olp,
                         tst, wst, vst, otst, owst, page_size, b, width, cap, sink, recent)
    rc = library().hicache_evict_pages(a, _launch_stream(stream, dev))
    if rc:
        _check(rc)
