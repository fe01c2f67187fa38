"""ctypes binding of liblora_mi355x.so.

Argument marshalling only: every step of the adapter path (plan building,
shrink, expand, the fused layer) runs inside the library.  PyTorch is used for
device memory, pinned host memory and streams.  If the library has not been
built, every entry point raises -- there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
import threading
import weakref
from dataclasses import dataclass
from typing import Optional

import numpy as np

from . import build as _build

LORA_F32 = 0
LORA_BF16 = 1
DTYPES = {"f32": LORA_F32, "bf16": LORA_BF16}

LORA_OP_SGMV_SHRINK = 0
LORA_OP_SGMV_EXPAND = 1
LORA_OP_BGMV_SHRINK = 2
LORA_OP_BGMV_EXPAND = 3
LORA_OP_FUSED = 4
LORA_OP_SGMV = 5
LORA_OP_BGMV = 6
LORA_OP_SGMV_BACKWARD = 7
LORA_OP_FUSED_BACKWARD = 8
LORA_OP_LINEAR_BLOCK = 9
LORA_OP_FUSED_BLOCK = 10
LORA_OP_FUSED_BLOCK_BACKWARD = 11

LORA_SCALE_F32 = 0
LORA_SCALE_E8M0 = 1
SCALE_BLOCK = 128
DEVICE_PLAN_MAX_ADAPTERS = 7168

LORA_GRAD_ACCUMULATE = 1
LORA_ADAM_F32 = 0
LORA_ADAM_8BIT = 1
ADAM_BLOCK = 256

STATUS = {
    0: "LORA_OK", -1: "LORA_ERR_ARG", -2: "LORA_ERR_RANK", -3: "LORA_ERR_ADAPTER_ID",
    -4: "LORA_ERR_ALIGN", -5: "LORA_ERR_DTYPE", -6: "LORA_ERR_WORKSPACE", -7: "LORA_ERR_HIP",
    -8: "LORA_ERR_PLAN",
}

# Every symbol the public header declares.
EXPORTS = [
    "lora_segments_bytes", "lora_segments_bind", "lora_build_segments", "lora_segments_upload", "lora_sgmv_shrink",
    "lora_sgmv_expand", "lora_sgmv", "lora_bgmv_shrink", "lora_bgmv_expand", "lora_bgmv", "lora_fused_linear", "lora_fused_linear_e4m3",
    "lora_workspace_bytes", "lora_adapter_numel", "lora_status_string", "lora_last_error",
    "lora_version", "lora_profile_launches", "lora_profile_launches_used", "lora_bgmv_grouped",
    "lora_bgmv_grouped_workspace_bytes", "lora_cache_table_bytes", "lora_cache_create", "lora_cache_destroy",
    "lora_cache_register", "lora_cache_pin", "lora_cache_prepare", "lora_cache_view_get", "lora_cache_stats_get",
    "lora_pages_needed", "lora_page_alloc_create", "lora_page_alloc_destroy", "lora_page_alloc_take",
    "lora_page_alloc_give", "lora_page_alloc_free_count", "lora_pages_write", "lora_sgmv_paged", "lora_bgmv_paged",
    "lora_sgmv_grouped", "lora_sgmv_grouped_workspace_bytes", "lora_probe_empty", "lora_probe_stream",
    "lora_probe_chase", "lora_workspace_clear", "lora_debug_wait_limit", "lora_bgmv_noalloc",
    "lora_sgmv_backward", "lora_fused_linear_backward", "lora_adamw_plan_bytes", "lora_adamw_plan", "lora_adamw_upload", "lora_adamw",
    "lora_adam_state_values", "lora_build_segments_device", "lora_quantize_e4m3", "lora_linear_e4m3_block",
    "lora_fused_linear_e4m3_block", "lora_fused_linear_e4m3_block_backward",
]
LORA_CACHE_DRY = 1
MAX_PROJ = 8

PLAN_HEADER_BYTES = 96
CHUNK_BLOCKS = 4
PLAN_MAGIC = 0x4C6F5241
ROW_BLOCK = 16


class LoraError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")
        self.status = status


_i32, _i64, _u64, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_size_t
_LIB = None
_RAW_STREAM = None
_LOCK = threading.Lock()

_SIGS = {
    "lora_segments_bytes": (_sz, [_i32]),
    "lora_segments_bind": (ctypes.c_int, [_vp, _i32, _vp]),
    "lora_build_segments": (ctypes.c_int, [_i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp]),
    "lora_segments_upload": (ctypes.c_int, [_vp, _vp, _vp]),
    "lora_sgmv_shrink": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _i32, _vp, _vp, _i64, _vp, _sz]),
    "lora_sgmv_expand": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _vp, _vp, _i64, _i32, _vp, _sz]),
    "lora_sgmv": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _sz]),
    "lora_bgmv": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                 _vp, _i64, _i32, _vp, _sz]),
    "lora_bgmv_shrink": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _vp, _i64, _i32, _vp, _vp, _vp, _i32, _i32,
                                        _vp, _i64, _vp, _sz]),
    "lora_bgmv_expand": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32,
                                        _vp, _i64, _i32, _vp, _sz]),
    "lora_fused_linear": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _sz]),
    "lora_fused_linear_e4m3": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, ctypes.c_float, _i32, _vp, _vp, _i64, _vp,
                                              _sz]),
    "lora_workspace_bytes": (_sz, [ctypes.c_int, _i32, _i32, _i32, _i32]),
    "lora_adapter_numel": (_i64, [_i32, _i32, _i32]),
    "lora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "lora_last_error": (ctypes.c_char_p, []),
    "lora_version": (ctypes.c_char_p, []),
    "lora_profile_launches": (ctypes.c_int, [_vp, _vp, _i32]),
    "lora_profile_launches_used": (ctypes.c_int32, []),
    "lora_bgmv_grouped": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _vp, _i32, _vp, _i32, _vp, _sz]),
    "lora_bgmv_grouped_workspace_bytes": (_sz, [_i32, _vp, _i32]),
    "lora_cache_table_bytes": (_sz, [_i32]),
    "lora_cache_create": (ctypes.c_int, [_vp, _sz, _i32, ctypes.c_int, _i32, _i32, ctypes.c_uint, _vp]),
    "lora_cache_destroy": (None, [_vp]),
    "lora_cache_register": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i32, ctypes.c_float]),
    "lora_cache_pin": (ctypes.c_int, [_vp, _i32, ctypes.c_int]),
    "lora_cache_prepare": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp]),
    "lora_cache_view_get": (ctypes.c_int, [_vp, _vp]),
    "lora_cache_stats_get": (ctypes.c_int, [_vp, _vp]),
    "lora_pages_needed": (_i64, [_i64, _i64]),
    "lora_sgmv_grouped": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i32, _vp, _sz]),
    "lora_sgmv_grouped_workspace_bytes": (_sz, [_vp, _i32]),
    "lora_probe_empty": (ctypes.c_int, [_vp, _i32]),
    "lora_workspace_clear": (ctypes.c_int, [_vp, _vp, _sz]),
    "lora_debug_wait_limit": (ctypes.c_int, [_i32]),
    "lora_bgmv_noalloc": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _i32,
                                         _i32, _vp, _i64, _i32]),
    "lora_sgmv_backward": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _i32, _vp, _i64, _i32, _vp, _vp, _vp, _i32,
                                          ctypes.c_uint, _vp, _i64, _vp, _sz]),
    "lora_fused_linear_backward": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _vp,
                                                  _vp, _i32, ctypes.c_uint, _vp, _i64, _vp, _sz]),
    "lora_adamw_plan_bytes": (_sz, [_vp, _i32]),
    "lora_adamw_plan": (ctypes.c_int, [_vp, _i32, _i32, ctypes.c_int, ctypes.c_int, _vp, _sz]),
    "lora_adamw_upload": (ctypes.c_int, [_vp, _vp, _sz, _vp]),
    "lora_adamw": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32]),
    "lora_adam_state_values": (ctypes.c_int, [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "lora_build_segments_device": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _vp,
                                                  _vp]),
    "lora_quantize_e4m3": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _i32, _i32, _i32, ctypes.c_int, _vp, _i64, _vp,
                                          _i64]),
    "lora_linear_e4m3_block": (ctypes.c_int, [_vp, _i32, _vp, _i64, _vp, _i64, _i32, _vp, _vp, ctypes.c_int, _i32,
                                              ctypes.c_int, _vp, _i64, _vp, _sz]),
    "lora_fused_linear_e4m3_block": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp, ctypes.c_int, _i32, _vp, _vp, _i64,
                                                    _vp, _sz]),
    "lora_fused_linear_e4m3_block_backward": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp, ctypes.c_int, _vp, _i64,
                                                             _i32, _vp, _vp, _vp, _i32, ctypes.c_uint, _vp, _i64, _vp,
                                                             _sz]),
    "lora_probe_stream": (ctypes.c_int, [_vp, _vp, _i64, _vp, _i64, _vp, _i32]),
    "lora_probe_chase": (ctypes.c_int, [_vp, _vp, _i32, _vp]),
    "lora_page_alloc_create": (ctypes.c_int, [_i32, _vp]),
    "lora_page_alloc_destroy": (None, [_vp]),
    "lora_page_alloc_take": (ctypes.c_int, [_vp, _i32, _vp]),
    "lora_page_alloc_give": (ctypes.c_int, [_vp, _vp, _i32]),
    "lora_page_alloc_free_count": (_i32, [_vp]),
    "lora_pages_write": (ctypes.c_int, [_vp, _vp, _i64, _vp, _vp, _i64]),
    "lora_sgmv_paged": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _i32, _vp, _vp, _i64, _vp, _i64, _i32, _vp,
                                       _sz]),
    "lora_bgmv_paged": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _i32,
                                       _i32, _vp, _i64, _vp, _i64, _i32, _vp, _sz]),
}


class CacheStats(ctypes.Structure):
    """struct lora_cache_stats."""

    _fields_ = [("batches", _i64), ("hits", _i64), ("misses", _i64), ("evictions", _i64), ("bytes_copied", _i64),
                ("resident_bytes", _i64), ("resident", _i32), ("reserved", _i32)]


class CacheView(ctypes.Structure):
    """struct lora_cache_view."""

    _fields_ = [("pool_A_dev", _vp), ("pool_B_dev", _vp), ("rank_dev", _vp), ("alpha_dev", _vp),
                ("pool_A_host", _vp), ("pool_B_host", _vp), ("rank_host", _vp), ("alpha_host", _vp),
                ("n_adapters", _i32), ("max_rank", _i32)]


assert ctypes.sizeof(CacheStats) == 56 and ctypes.sizeof(CacheView) == 72


class LoraProj(ctypes.Structure):
    """struct lora_proj: one projection of a grouped BGMV call."""

    _fields_ = [("x", _vp), ("y", _vp), ("pool_A_dev", _vp), ("pool_B_dev", _vp), ("pool_rank_dev", _vp),
                ("pool_alpha_dev", _vp), ("ldx", _i64), ("ldy", _i64), ("d_in", _i32), ("d_out", _i32),
                ("max_rank", _i32), ("reserved", _i32)]


assert ctypes.sizeof(LoraProj) == 80


class LoraSegments(ctypes.Structure):
    """struct lora_segments: a batch's segments, bound to a host or device buffer."""

    _fields_ = [("num_segments", _i32), ("num_tokens", _i32), ("max_rank", _i32), ("capacity", _i32),
                ("perm", _vp), ("seg_indptr", _vp), ("seg_adapter", _vp), ("seg_rank", _vp), ("seg_A", _vp),
                ("seg_B", _vp), ("seg_scale", _vp), ("batch_tokens", _i32), ("reserved0", _i32), ("buf", _vp),
                ("host", _vp)]


assert ctypes.sizeof(LoraSegments) == 96


class LoraSgmvProj(ctypes.Structure):
    """struct lora_sgmv_proj: one projection of a grouped SGMV call."""

    _fields_ = [("x", _vp), ("y", _vp), ("seg", _vp), ("ldx", _i64), ("ldy", _i64), ("d_in", _i32), ("d_out", _i32)]


assert ctypes.sizeof(LoraSgmvProj) == 48


class LoraAdamTensor(ctypes.Structure):
    """struct lora_adam_tensor: one tensor of an AdamW plan."""

    _fields_ = [("param", _u64), ("grad", _u64), ("copy", _u64), ("m", _u64), ("v", _u64), ("m_scale", _u64),
                ("v_scale", _u64), ("n", _i64), ("group", _i32), ("reserved", _i32)]


assert ctypes.sizeof(LoraAdamTensor) == 72


def lib_path() -> str:
    return _build.lib_path()


def load():
    """Load the built library (raises if it is missing)."""
    global _LIB
    with _LOCK:
        if _LIB is not None:
            return _LIB
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built; run `python -m segmented_gather_gemm_lora_amd.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
        return lib


def _check(status: int, where: str):
    if status != 0:
        raise LoraError(status, where, load().lora_last_error().decode())


def last_error() -> str:
    return load().lora_last_error().decode()


# ------------------------------------------------------------------ raw C calls (same names)
def lora_segments_bytes(capacity: int) -> int:
    return int(load().lora_segments_bytes(capacity))


def lora_workspace_bytes(op: int, T: int, d_in: int, d_out: int, max_rank: int) -> int:
    return int(load().lora_workspace_bytes(op, T, d_in, d_out, max_rank))


def lora_adapter_numel(r: int, d_in: int, d_out: int) -> int:
    return int(load().lora_adapter_numel(r, d_in, d_out))


def lora_version() -> str:
    return load().lora_version().decode()


def lora_status_string(status: int) -> str:
    return load().lora_status_string(status).decode()


def lora_segments_bind(buf_ptr, capacity, seg_ptr) -> int:
    return int(load().lora_segments_bind(buf_ptr, capacity, seg_ptr))


def lora_build_segments(T, ids_ptr, n_adapters, pool_A_ptr, pool_B_ptr, pool_rank_ptr, pool_alpha_ptr,
                        seg_ptr) -> int:
    return int(load().lora_build_segments(T, ids_ptr, n_adapters, pool_A_ptr, pool_B_ptr, pool_rank_ptr,
                                          pool_alpha_ptr, seg_ptr))


def lora_segments_upload(host_ptr, dev_ptr, stream) -> int:
    return int(load().lora_segments_upload(host_ptr, dev_ptr, stream))


def lora_sgmv_shrink(stream, dtype, x, ldx, d_in, seg, v, ldv, ws, ws_bytes) -> int:
    return int(load().lora_sgmv_shrink(stream, dtype, x, ldx, d_in, seg, v, ldv, ws, ws_bytes))


def lora_sgmv_expand(stream, dtype, v, ldv, seg, y, ldy, d_out, ws, ws_bytes) -> int:
    return int(load().lora_sgmv_expand(stream, dtype, v, ldv, seg, y, ldy, d_out, ws, ws_bytes))


def lora_sgmv(stream, dtype, x, ldx, d_in, seg, y, ldy, d_out, ws, ws_bytes) -> int:
    return int(load().lora_sgmv(stream, dtype, x, ldx, d_in, seg, y, ldy, d_out, ws, ws_bytes))


def lora_bgmv(stream, dtype, T, x, ldx, d_in, ids, pool_A, pool_B, pool_rank, pool_alpha, n_adapters, max_rank,
              y, ldy, d_out, ws, ws_bytes) -> int:
    return int(load().lora_bgmv(stream, dtype, T, x, ldx, d_in, ids, pool_A, pool_B, pool_rank, pool_alpha,
                                n_adapters, max_rank, y, ldy, d_out, ws, ws_bytes))


def lora_bgmv_shrink(stream, dtype, T, x, ldx, d_in, ids, pool_A, pool_rank, n_adapters, max_rank, v, ldv,
                     ws, ws_bytes) -> int:
    return int(load().lora_bgmv_shrink(stream, dtype, T, x, ldx, d_in, ids, pool_A, pool_rank, n_adapters,
                                       max_rank, v, ldv, ws, ws_bytes))


def lora_bgmv_expand(stream, dtype, T, v, ldv, ids, pool_B, pool_rank, pool_alpha, n_adapters, max_rank,
                     y, ldy, d_out, ws, ws_bytes) -> int:
    return int(load().lora_bgmv_expand(stream, dtype, T, v, ldv, ids, pool_B, pool_rank, pool_alpha,
                                       n_adapters, max_rank, y, ldy, d_out, ws, ws_bytes))


def lora_bgmv_grouped(stream, dtype, T, ids, n_adapters, projs, n_proj, ws, ws_bytes) -> int:
    return int(load().lora_bgmv_grouped(stream, dtype, T, ids, n_adapters, projs, n_proj, ws, ws_bytes))


def lora_bgmv_grouped_workspace_bytes(T, projs, n_proj) -> int:
    return int(load().lora_bgmv_grouped_workspace_bytes(T, projs, n_proj))


class _Raw:
    """A raw device address where the calls expect a tensor."""

    def __init__(self, addr):
        self.addr = int(addr or 0)

    def data_ptr(self) -> int:
        return self.addr


class AdapterCache:
    """Residency cache over a device buffer (lora_cache_*): adapters registered
    from pinned host memory are copied in on a copy stream when a batch needs
    them, least recently used ones evicted.  dev_buf: a uint8 device tensor (or
    an int address when dry).  `pool()` gives the tables in the form the
    SGMV/BGMV calls take."""

    def __init__(self, dev_buf, n_adapters: int, dtype: str, d_in: int, d_out: int, dry: bool = False):
        lib = load()
        self._buf = dev_buf  # keeps the device memory alive
        addr = dev_buf if isinstance(dev_buf, int) else _ptr(dev_buf)
        nbytes = self.dry_bytes if isinstance(dev_buf, int) else dev_buf.numel()
        h = ctypes.c_void_p()
        _check(lib.lora_cache_create(addr, nbytes, n_adapters, DTYPES[dtype], d_in, d_out,
                                     LORA_CACHE_DRY if dry else 0, ctypes.byref(h)), "lora_cache_create")
        self.h, self.n_adapters, self.dtype, self.d_in, self.d_out = h, n_adapters, dtype, d_in, d_out
        self.dry = dry
        self._host = {}

    dry_bytes = 0

    @classmethod
    def dry_run(cls, nbytes: int, n_adapters: int, dtype: str, d_in: int, d_out: int):
        """A placement-only cache over a fake 256-byte aligned address range."""
        obj = cls.__new__(cls)
        obj.dry_bytes = nbytes
        cls.__init__(obj, 0x7F0000000000, n_adapters, dtype, d_in, d_out, dry=True)
        return obj

    def close(self):
        if getattr(self, "h", None) is not None and self.h.value:
            load().lora_cache_destroy(self.h)
            self.h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def register(self, adapter: int, A_host, B_host, rank: int, alpha: float):
        """A_host / B_host: host arrays or tensors (pinned for overlapped copies),
        kept referenced by the cache object."""
        self._host[adapter] = (A_host, B_host)
        pa = A_host.ctypes.data if isinstance(A_host, np.ndarray) else A_host.data_ptr()
        pb = B_host.ctypes.data if isinstance(B_host, np.ndarray) else B_host.data_ptr()
        _check(load().lora_cache_register(self.h, adapter, pa, pb, rank, alpha), "lora_cache_register")

    def pin(self, adapter: int, pinned: bool = True):
        _check(load().lora_cache_pin(self.h, adapter, int(pinned)), "lora_cache_pin")

    def prepare(self, ids, copy_stream=None, compute_stream=None):
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        streams = (None, None) if self.dry else (_stream_handle(copy_stream), _stream_handle(compute_stream))
        _check(load().lora_cache_prepare(self.h, ids.ctypes.data if ids.size else None, ids.shape[0], *streams),
               "lora_cache_prepare")

    def stats(self) -> dict:
        st = CacheStats()
        _check(load().lora_cache_stats_get(self.h, ctypes.byref(st)), "lora_cache_stats_get")
        return {f: getattr(st, f) for f, _ in CacheStats._fields_ if f != "reserved"}

    def view(self) -> CacheView:
        v = CacheView()
        _check(load().lora_cache_view_get(self.h, ctypes.byref(v)), "lora_cache_view_get")
        return v

    def pool(self) -> "DevicePool":
        """The current tables as a DevicePool: host mirrors for lora_build_segments,
        device tables for the BGMV calls.  Valid until the next prepare."""
        v = self.view()
        A, Bt, r, a = self.host_tables()
        return DevicePool(storage=self._buf, n_adapters=self.n_adapters, dtype=self.dtype, d_in=self.d_in,
                          d_out=self.d_out, addr_A=A, addr_B=Bt, rank=r, alpha=a, addr_A_dev=_Raw(v.pool_A_dev),
                          addr_B_dev=_Raw(v.pool_B_dev), rank_dev=_Raw(v.rank_dev), alpha_dev=_Raw(v.alpha_dev))

    def host_tables(self):
        """Copies of the host mirrors: (A addresses, B addresses, ranks, alphas)."""
        v, n = self.view(), self.n_adapters
        A = np.ctypeslib.as_array(ctypes.cast(v.pool_A_host, ctypes.POINTER(ctypes.c_uint64)), (n,)).copy()
        Bt = np.ctypeslib.as_array(ctypes.cast(v.pool_B_host, ctypes.POINTER(ctypes.c_uint64)), (n,)).copy()
        r = np.ctypeslib.as_array(ctypes.cast(v.rank_host, ctypes.POINTER(ctypes.c_int32)), (n,)).copy()
        a = np.ctypeslib.as_array(ctypes.cast(v.alpha_host, ctypes.POINTER(ctypes.c_float)), (n,)).copy()
        return A, Bt, r, a


def lora_fused_linear(stream, dtype, x, ldx, d_in, W0, d_out, seg, y, ldy, ws, ws_bytes) -> int:
    return int(load().lora_fused_linear(stream, dtype, x, ldx, d_in, W0, d_out, seg, y, ldy, ws, ws_bytes))


def lora_fused_linear_e4m3(stream, x, ldx, d_in, W0, w0_scale, d_out, seg, y, ldy, ws, ws_bytes) -> int:
    return int(load().lora_fused_linear_e4m3(stream, x, ldx, d_in, W0, w0_scale, d_out, seg, y, ldy, ws, ws_bytes))


def lora_profile_launches(start_events, stop_events, count) -> int:
    return int(load().lora_profile_launches(start_events, stop_events, count))


class KernelTimer:
    """Times the library's next kernel launches with HIP events attached to the
    kernels themselves (hipExtLaunchKernelGGL start/stop events)."""

    _hip = None

    def __init__(self, n: int):
        if KernelTimer._hip is None:
            hip = ctypes.CDLL("libamdhip64.so")
            hip.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
            hip.hipEventDestroy.argtypes = [ctypes.c_void_p]
            hip.hipEventSynchronize.argtypes = [ctypes.c_void_p]
            hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p, ctypes.c_void_p]
            KernelTimer._hip = hip
        self.n = n
        self.start = (ctypes.c_void_p * n)()
        self.stop = (ctypes.c_void_p * n)()
        for i in range(n):
            for arr in (self.start, self.stop):
                h = ctypes.c_void_p()
                if KernelTimer._hip.hipEventCreate(ctypes.byref(h)) != 0:
                    raise RuntimeError("hipEventCreate failed")
                arr[i] = h

    def arm(self, first: int, count: int):
        """The next `count` launches record events first .. first+count-1."""
        st = lora_profile_launches(ctypes.addressof(self.start) + 8 * first,
                                   ctypes.addressof(self.stop) + 8 * first, count)
        _check(st, "lora_profile_launches")

    def disarm(self):
        _check(lora_profile_launches(None, None, 0), "lora_profile_launches")

    @staticmethod
    def used() -> int:
        """Launches that took events since the last arm()."""
        return int(load().lora_profile_launches_used())

    def elapsed_us(self, i: int) -> float:
        hip = KernelTimer._hip
        hip.hipEventSynchronize(self.stop[i])
        ms = ctypes.c_float()
        if hip.hipEventElapsedTime(ctypes.byref(ms), self.start[i], self.stop[i]) != 0:
            raise RuntimeError("hipEventElapsedTime failed")
        return ms.value * 1e3

    def close(self):
        for i in range(self.n):
            KernelTimer._hip.hipEventDestroy(self.start[i])
            KernelTimer._hip.hipEventDestroy(self.stop[i])


class Prepared:
    """One library call with its arguments converted to C types once, for
    loops that repeat the same call (benchmarks, serving loops): calling the
    object makes the C call and raises on a non-zero status.  `keep` holds
    the tensors whose addresses the arguments carry."""

    __slots__ = ("_fn", "_args", "_name", "_keep")

    def __init__(self, name: str, args, keep=()):
        res, types = _SIGS[name]
        if len(types) != len(args):
            raise TypeError(f"{name} takes {len(types)} arguments, got {len(args)}")
        self._fn = getattr(load(), name)
        self._args = tuple(None if a is None else (a if isinstance(a, ctypes._SimpleCData) else t(a))
                           for t, a in zip(types, args))
        self._name = name
        self._keep = tuple(keep)

    def __call__(self):
        st = self._fn(*self._args)
        if st:
            _check(st, self._name)


# ------------------------------------------------------------------ torch-facing helpers
def _torch():
    import torch

    return torch


def _stream_handle(stream, device: Optional[int] = None) -> Optional[int]:
    if stream is None:
        return _current_stream(device)
    return stream.cuda_stream


def _current_stream(device: Optional[int] = None) -> int:
    """The current stream of the device (None: the current one), without building a
    stream object (2.5 us of a call whose kernel takes 4)."""
    global _RAW_STREAM
    torch = _torch()
    if _RAW_STREAM is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _RAW_STREAM = raw if raw is not None else lambda device: torch.cuda.current_stream(device).cuda_stream
    return _RAW_STREAM(torch.cuda.current_device() if device is None else device)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def torch_dtype(dtype: str):
    torch = _torch()
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def to_device(arr: np.ndarray, dtype: str, device="cuda"):
    """Host array (bf16 bit patterns as uint16, or float32) -> device tensor."""
    torch = _torch()
    if dtype == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(arr).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(arr, dtype=np.float32))
    return t.to(device)


def to_host_bits(t, dtype: str) -> np.ndarray:
    """Device tensor -> host array in the stored representation."""
    torch = _torch()
    t = t.detach().cpu().contiguous()
    if dtype == "bf16":
        return t.view(torch.int16).numpy().view(np.uint16)
    return t.numpy().astype(np.float32, copy=False)


@dataclass
class DevicePool:
    """Adapters resident in device memory, with their pointer and rank tables."""

    storage: object  # device tensor holding every A_i and B_i (unpadded)
    n_adapters: int
    dtype: str
    d_in: int
    d_out: int
    addr_A: np.ndarray  # uint64 host copies of the tables
    addr_B: np.ndarray
    rank: np.ndarray  # int32
    alpha: np.ndarray  # float32
    addr_A_dev: object = None  # device tables (for BGMV)
    addr_B_dev: object = None
    rank_dev: object = None
    alpha_dev: object = None

    @property
    def max_rank(self) -> int:
        return int(self.rank.max()) if self.rank.size else 0

    @classmethod
    def from_problem(cls, prob, device="cuda") -> "DevicePool":
        torch = _torch()
        storage = to_device(prob.pool, prob.dtype, device)
        base = storage.data_ptr()
        es = prob.esize
        addr_A = (base + prob.a_off.astype(np.uint64) * np.uint64(es)).astype(np.uint64)
        addr_B = (base + prob.b_off.astype(np.uint64) * np.uint64(es)).astype(np.uint64)
        rank = np.ascontiguousarray(prob.ranks, dtype=np.int32)
        alpha = np.ascontiguousarray(prob.alphas, dtype=np.float32)
        p = cls(storage=storage, n_adapters=prob.n_adapters, dtype=prob.dtype, d_in=prob.d_in, d_out=prob.d_out,
                addr_A=addr_A, addr_B=addr_B, rank=rank, alpha=alpha)
        p.addr_A_dev = torch.from_numpy(addr_A.view(np.int64)).to(device)
        p.addr_B_dev = torch.from_numpy(addr_B.view(np.int64)).to(device)
        p.rank_dev = torch.from_numpy(rank).to(device)
        p.alpha_dev = torch.from_numpy(alpha).to(device)
        return p


class PageAlloc:
    """The library's frame allocator of one page pool (host side)."""

    def __init__(self, n_frames: int):
        self._h = ctypes.c_void_p()
        _check(load().lora_page_alloc_create(int(n_frames), ctypes.byref(self._h)), "lora_page_alloc_create")
        self.n_frames = int(n_frames)

    def take(self, n: int) -> np.ndarray:
        out = np.zeros(max(int(n), 1), dtype=np.int32)
        _check(load().lora_page_alloc_take(self._h, int(n), out.ctypes.data), "lora_page_alloc_take")
        return out[: int(n)]

    def give(self, frames) -> None:
        f = np.ascontiguousarray(frames, dtype=np.int32)
        _check(load().lora_page_alloc_give(self._h, f.ctypes.data, int(f.size)), "lora_page_alloc_give")

    @property
    def free(self) -> int:
        return int(load().lora_page_alloc_free_count(self._h))

    def close(self):
        if self._h:
            load().lora_page_alloc_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def lora_pages_needed(nbytes: int, page_bytes: int) -> int:
    return int(load().lora_pages_needed(int(nbytes), int(page_bytes)))


@dataclass
class PagedPool:
    """Adapters held in fixed-size pages of one device pool, each matrix behind
    a device page table (int32 frames).  addr_A / addr_B hold the addresses of
    the page tables, so a Plan builds from this pool as from a DevicePool."""

    pages: object  # device uint8 [n_frames * page_bytes]
    page_bytes: int
    tables: object  # device int32: every page table, each 16-byte aligned
    table_host: np.ndarray
    frames_A: list  # host int32 frames of each adapter's A
    frames_B: list
    alloc: PageAlloc
    n_adapters: int
    dtype: str
    d_in: int
    d_out: int
    addr_A: np.ndarray
    addr_B: np.ndarray
    rank: np.ndarray
    alpha: np.ndarray
    addr_A_dev: object = None
    addr_B_dev: object = None
    rank_dev: object = None
    alpha_dev: object = None

    @property
    def max_rank(self) -> int:
        return int(self.rank.max()) if self.rank.size else 0

    @classmethod
    def from_problem(cls, prob, page_bytes: int = 16384, shuffle_seed: Optional[int] = 0, spare_frames: int = 0,
                     device="cuda", stream=None) -> "PagedPool":
        """Allocates frames for every adapter of `prob` and writes A_i and B_i
        into them with lora_pages_write.  shuffle_seed: frames are first taken
        and given back in a seeded random order, so each matrix lands in
        scattered frames (None: ascending frames)."""
        torch = _torch()
        es = prob.esize
        ranks = np.ascontiguousarray(prob.ranks, dtype=np.int32)
        nA = [lora_pages_needed(int(r) * prob.d_in * es, page_bytes) for r in ranks]
        nB = [lora_pages_needed(prob.d_out * int(r) * es, page_bytes) for r in ranks]
        if min(nA + nB, default=0) < 0:
            raise ValueError(f"page_bytes {page_bytes} is not a power of two in [64, 2^24]")
        n_frames = int(sum(nA) + sum(nB) + spare_frames)
        alloc = PageAlloc(max(n_frames, 1))
        if shuffle_seed is not None and n_frames > 0:
            all_frames = alloc.take(n_frames)
            alloc.give(np.random.default_rng(shuffle_seed).permutation(all_frames))
        frames_A = [alloc.take(n) for n in nA]
        frames_B = [alloc.take(n) for n in nB]
        # page tables, each starting on a 16-byte boundary
        offs_A, offs_B, parts, pos = [], [], [], 0
        for fa, fb in zip(frames_A, frames_B):
            for f, offs in ((fa, offs_A), (fb, offs_B)):
                offs.append(pos)
                pad = (-len(f)) % 4
                parts.append(np.concatenate([f, np.zeros(pad, dtype=np.int32)]))
                pos += len(f) + pad
        table_host = np.concatenate(parts) if parts else np.zeros(4, dtype=np.int32)
        tables = torch.from_numpy(table_host).to(device)
        base = tables.data_ptr()
        addr_A = np.array([base + 4 * o for o in offs_A], dtype=np.uint64)
        addr_B = np.array([base + 4 * o for o in offs_B], dtype=np.uint64)
        pages = torch.empty(max(n_frames, 1) * page_bytes, dtype=torch.uint8, device=device)
        dense = to_device(prob.pool, prob.dtype, device)
        sbase = dense.data_ptr()
        st = _stream_handle(stream)
        for i, r in enumerate(ranks):
            for off, nbytes, addr in ((int(prob.a_off[i]), int(r) * prob.d_in * es, addr_A[i]),
                                      (int(prob.b_off[i]), prob.d_out * int(r) * es, addr_B[i])):
                _check(load().lora_pages_write(st, pages.data_ptr(), page_bytes, int(addr), sbase + off * es,
                                               nbytes), "lora_pages_write")
        torch.cuda.synchronize()
        del dense
        alpha = np.ascontiguousarray(prob.alphas, dtype=np.float32)
        p = cls(pages=pages, page_bytes=int(page_bytes), tables=tables, table_host=table_host, frames_A=frames_A,
                frames_B=frames_B, alloc=alloc, n_adapters=prob.n_adapters, dtype=prob.dtype, d_in=prob.d_in,
                d_out=prob.d_out, addr_A=addr_A, addr_B=addr_B, rank=ranks, alpha=alpha)
        p.addr_A_dev = torch.from_numpy(addr_A.view(np.int64)).to(device)
        p.addr_B_dev = torch.from_numpy(addr_B.view(np.int64)).to(device)
        p.rank_dev = torch.from_numpy(ranks).to(device)
        p.alpha_dev = torch.from_numpy(alpha).to(device)
        return p


@dataclass
class GradPool:
    """fp32 gradients of adapters: dA_i [r_i, d_in] and dB_i [d_out, r_i],
    contiguous, reached through device tables of their addresses (0 = not
    wanted)."""

    storage: object  # the tensors that hold the gradients
    A: list  # per adapter: a tensor of r_i * d_in fp32, or None
    B: list
    addr_A_dev: object
    addr_B_dev: object

    @property
    def n_adapters(self) -> int:
        return len(self.A)

    @classmethod
    def from_tensors(cls, A, B, device=None) -> "GradPool":
        """A, B: one contiguous fp32 device tensor (or None) for each adapter."""
        torch = _torch()
        if len(A) != len(B):
            raise ValueError("A and B list different numbers of adapters")
        for t in (*A, *B):
            if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda):
                raise ValueError("gradients are contiguous fp32 device tensors")
        device = device or next((t.device for t in (*A, *B) if t is not None), "cuda")

        def table(ts):
            a = np.array([0 if t is None else t.data_ptr() for t in ts], dtype=np.uint64)
            return torch.from_numpy(a.view(np.int64)).to(device)

        return cls(storage=None, A=list(A), B=list(B), addr_A_dev=table(A), addr_B_dev=table(B))

    @classmethod
    def like(cls, pool, device="cuda") -> "GradPool":
        """Zero gradients for every adapter of a pool, in one buffer, 16-byte aligned."""
        torch = _torch()
        sizes = [int(r) * d for r in pool.rank for d in (pool.d_in, pool.d_out)]
        starts = np.concatenate([[0], np.cumsum([(s + 3) // 4 * 4 for s in sizes])]).astype(np.int64)
        storage = torch.zeros(max(int(starts[-1]), 4), device=device)
        parts = [storage[int(o): int(o) + s] for o, s in zip(starts, sizes)]
        A = [t.view(int(r), pool.d_in) for t, r in zip(parts[0::2], pool.rank)]
        B = [t.view(pool.d_out, int(r)) for t, r in zip(parts[1::2], pool.rank)]
        g = cls.from_tensors(A, B, device=device)
        g.storage = storage
        return g


SEG_DESC = np.dtype([("A", "<u8"), ("B", "<u8"), ("start", "<i4"), ("len", "<i4"), ("rank", "<i4"),
                     ("adapter", "<i4"), ("scale", "<f4"), ("blk0", "<i4")])
BLK_DESC = np.dtype([("A", "<u8"), ("B", "<u8"), ("scale", "<f4"), ("rank", "<i4"), ("n", "<i4"), ("p0", "<i4"),
                     ("seg", "<i4"), ("reserved", "<i4", (7,)), ("rows", "<i4", (ROW_BLOCK,))])
CHUNK_DESC = np.dtype([("A", "<u8"), ("B", "<u8"), ("scale", "<f4"), ("rank", "<i4"), ("n", "<i4"),
                       ("p0", "<i4"), ("seg", "<i4"), ("first_blk", "<i4"), ("nblk", "<i4"),
                       ("reserved", "<i4", (5,)), ("rows", "<i4", (ROW_BLOCK * CHUNK_BLOCKS,))])
assert SEG_DESC.itemsize == 40 and BLK_DESC.itemsize == 128 and CHUNK_DESC.itemsize == 320


def plan_header(h: np.ndarray) -> dict:
    """Fields of a plan header held in `h` (uint8, at least 96 bytes)."""
    i32 = h[:32].view(np.int32)
    u64 = h[32:96].view(np.uint64)
    return {"magic": int(h[:4].view(np.uint32)[0]), "num_tokens": int(i32[1]), "num_sorted": int(i32[2]),
            "num_segments": int(i32[3]), "num_blocks": int(i32[4]), "max_rank": int(i32[5]),
            "max_len": int(i32[6]), "num_chunks": int(i32[7]), "seg_offset": int(u64[0]),
            "blk_offset": int(u64[1]), "perm_offset": int(u64[2]), "bytes_used": int(u64[3]),
            "chunk_offset": int(u64[4]), "segidx_offset": int(u64[5]), "soa_offset": int(u64[6])}


def plan_arrays(buf: np.ndarray, h: dict) -> dict:
    """Segment descriptors, block descriptors and perm of a plan held in `buf` (uint8)."""
    S, nb, Tp = h["num_segments"], h["num_blocks"], h["num_sorted"]
    so, bo, po = h["seg_offset"], h["blk_offset"], h["perm_offset"]
    seg = np.frombuffer(buf[so: so + SEG_DESC.itemsize * S].tobytes(), dtype=SEG_DESC)
    blk = np.frombuffer(buf[bo: bo + BLK_DESC.itemsize * nb].tobytes(), dtype=BLK_DESC)
    perm = buf[po: po + 4 * Tp].view(np.int32).copy()
    rest = buf[po + 4 * Tp: po + 4 * h["num_tokens"]].view(np.int32).copy()
    out = {"desc": seg, "blocks": blk, "perm": perm, "unadapted": rest}
    if "segidx_offset" in h:
        xo = h["segidx_offset"]
        out["segidx"] = buf[xo: xo + 4 * Tp].view(np.int32).copy()
    if "chunk_offset" in h:
        co = h["chunk_offset"]
        out["chunks"] = np.frombuffer(buf[co: co + CHUNK_DESC.itemsize * h["num_chunks"]].tobytes(), dtype=CHUNK_DESC)
    return out


class Plan:
    """A batch's segments (struct lora_segments): a pinned host buffer and a
    device buffer, each bound to a struct; build() fills the host one,
    upload() copies it to the device one (one copy).  `seg` is the address of
    the device struct, which the calls take."""

    def __init__(self, capacity: int, device="cuda"):
        torch = _torch()
        self.capacity = int(capacity)
        self.nbytes = lora_segments_bytes(self.capacity)
        self.host = torch.empty(self.nbytes, dtype=torch.uint8, pin_memory=True)
        self.dev = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.h = LoraSegments()
        self.d = LoraSegments()
        _check(lora_segments_bind(self.host.data_ptr(), self.capacity, ctypes.addressof(self.h)), "lora_segments_bind")
        _check(lora_segments_bind(self.dev.data_ptr(), self.capacity, ctypes.addressof(self.d)), "lora_segments_bind")

    # (d_in, d_out, dtype) of the pool that build() took the adapters from, and whether
    # that is a PagedPool (the segments do not say); the GradPool that was last found to
    # fit them (weak)
    made_for = None
    paged = False
    grads_fit = None

    @property
    def seg(self) -> int:
        return ctypes.addressof(self.d)

    def build(self, ids: np.ndarray, pool: DevicePool):
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        if ids.shape[0] > self.capacity:
            raise ValueError("batch larger than the segments' capacity")
        self.made_for, self.grads_fit = (pool.d_in, pool.d_out, pool.dtype), None
        self.paged = isinstance(pool, PagedPool)
        st = lora_build_segments(ids.shape[0], ids.ctypes.data, pool.n_adapters, pool.addr_A.ctypes.data,
                                 pool.addr_B.ctypes.data, pool.rank.ctypes.data, pool.alpha.ctypes.data,
                                 ctypes.addressof(self.h))
        _check(st, "lora_build_segments")
        return self

    def upload(self, stream=None):
        _check(lora_segments_upload(ctypes.addressof(self.h), ctypes.addressof(self.d), _stream_handle(stream)),
               "lora_segments_upload")
        return self

    def header(self) -> dict:
        return plan_header(self.host[:PLAN_HEADER_BYTES].numpy())

    def arrays(self) -> dict:
        """Host copies of the plan's arrays (for tests)."""
        return plan_arrays(self.host.numpy(), self.header())

    def segment_table(self) -> dict:
        """The host struct's segment table as numpy arrays (copies)."""
        return segment_table(self.h)


class DevicePlan:
    """A batch's segments built on the device (lora_build_segments_device): build()
    enqueues one launch that reads the adapters and lengths of the requests, and the
    pool's tables, from device memory, so it and the calls that take the plan can be
    captured together and replayed for other batches of up to `rows` rows.  The
    gradient calls take a Plan.  max_rank and rank_multiple (the pool's, where not given)
    bound what the tables may hold at any build; requests of adapters outside them count
    as having none.  Every build reads the table tensors that the pool has now: changes go into them."""

    def __init__(self, rows: int, pool, max_rank: Optional[int] = None, rank_multiple: Optional[int] = None):
        torch = _torch()
        self.rows, self.pool = int(rows), pool
        ranks = np.asarray(pool.rank, dtype=np.int64)
        self.max_rank = int(max_rank or max(pool.max_rank, 1))
        step = int(np.gcd.reduce(ranks)) if ranks.size else 1
        self.rank_multiple = int(rank_multiple or max(min(step & -step, 16), 1))
        for t, dt in ((pool.addr_A_dev, torch.int64), (pool.addr_B_dev, torch.int64), (pool.rank_dev, torch.int32),
                      (pool.alpha_dev, torch.float32)):
            if not isinstance(t, _Raw) and (t is None or t.dtype != dt or not t.is_cuda or not t.is_contiguous()
                                            or t.numel() < pool.n_adapters):
                raise ValueError("the pool has no device tables of its adapters")
        device = pool.rank_dev.device if hasattr(pool.rank_dev, "device") else "cuda"
        # a plan of no rows is built without a launch: its counts on the device are these zeros
        self.dev = (torch.empty if self.rows else torch.zeros)(lora_segments_bytes(self.rows), dtype=torch.uint8, device=device)
        self.geometry = (ctypes.c_uint64 * (PLAN_HEADER_BYTES // 8))()
        self.h = LoraSegments()  # no segment on the host
        self.h.batch_tokens = self.rows
        self.d = LoraSegments()
        self.made_for, self.paged, self.grads_fit = (pool.d_in, pool.d_out, pool.dtype), isinstance(pool, PagedPool), None
        _check(lora_segments_bind(self.dev.data_ptr(), self.rows, ctypes.addressof(self.d)), "lora_segments_bind")
        self._device, self._fn, self._tables = self.dev.get_device(), load().lora_build_segments_device, None
        self._held = (pool.addr_A_dev, pool.addr_B_dev, pool.rank_dev, pool.alpha_dev)  # builds, and graphs, read these
        self._pool_args = (pool.n_adapters, *map(_ptr, self._held),
                           self.max_rank, self.rank_multiple, self.geometry, ctypes.addressof(self.d))

    @property
    def seg(self) -> int:
        return ctypes.addressof(self.d)

    def build(self, adapters, lengths=None, stream=None):
        """adapters: int32 device tensor, the adapter of each request (-1: none); lengths:
        int32 device tensor of the requests' rows, or None: one row each."""
        torch = _torch()
        device = torch.cuda.current_device()
        n, = adapters.shape
        if self._device != device or adapters.get_device() != device:
            raise ValueError("the plan or adapters are not on the current device")
        if adapters.dtype is not torch.int32 or (n > 1 and adapters.stride(0) != 1):
            raise ValueError("adapters are adjacent int32 elements, one a request")
        if n >> 31:  # the C call's count has 32 bits
            raise ValueError(f"{n} requests")
        at = None
        if lengths is not None:
            if lengths.dtype is not torch.int32 or lengths.shape != adapters.shape or lengths.get_device() != device or (
                    n > 1 and lengths.stride(0) != 1):
                raise ValueError("lengths are adjacent int32 elements on the current device, one a request")
            at = lengths.data_ptr()
        st = self._fn(_stream_handle(stream, device), self.rows, n, adapters.data_ptr(), at, *self._pool_args)
        if st:
            _check(st, "lora_build_segments_device")
        return self

    def bounds(self) -> dict:
        """The geometry: bounds of the counts, and the tables' offsets."""
        return plan_header(np.frombuffer(self.geometry, dtype=np.uint8))

    def tables(self) -> dict:
        """Views of the last build's tables in the device buffer (int32): counts (rows, adapted
        rows, segments, blocks, largest rank, longest segment, chunks), segments [S, 10], blocks
        [n, 32], chunks [n, 80] (the records' words), perm and segidx."""
        if self._tables is not None:  # their places do not change from build to build
            return self._tables
        h, w = self.bounds(), self.dev[: self.dev.numel() // 4 * 4].view(_torch().int32)
        if h["magic"] != PLAN_MAGIC:
            raise ValueError("nothing has been built")

        def at(key, n, width):
            o = h[key] // 4
            return w[o: o + n * width].view(n, width)

        T = h["num_tokens"]
        self._tables = {"counts": w[1:8], "segments": at("seg_offset", h["num_segments"], SEG_DESC.itemsize // 4),
                        "blocks": at("blk_offset", h["num_blocks"], BLK_DESC.itemsize // 4),
                        "chunks": at("chunk_offset", h["num_chunks"], CHUNK_DESC.itemsize // 4),
                        "perm": w[h["perm_offset"] // 4:][:T], "segidx": w[h["segidx_offset"] // 4:][: h["num_sorted"]]}
        return self._tables

    def header(self) -> dict:
        """The last build's header, from the device (synchronises)."""
        return plan_header(self.dev[:PLAN_HEADER_BYTES].cpu().numpy())

    def arrays(self) -> dict:
        """Host copies of the last build's arrays, cut to its counts (synchronises; for tests)."""
        return plan_arrays(self.dev.cpu().numpy(), self.header())


_NP_OF = {ctypes.c_int32: np.int32, ctypes.c_uint64: np.uint64, ctypes.c_float: np.float32}


def segment_table(h: LoraSegments) -> dict:
    """perm, seg_indptr, seg_adapter, seg_rank, seg_A, seg_B, seg_scale of a
    host-bound struct, as numpy copies."""
    S, Tp = h.num_segments, h.num_tokens

    def arr(ptr, ctype, n):
        if n == 0 or not ptr:
            return np.zeros(0, dtype=_NP_OF[ctype])
        return np.ctypeslib.as_array(ctypes.cast(ptr, ctypes.POINTER(ctype)), (n,)).copy()

    return {"perm": arr(h.perm, ctypes.c_int32, Tp), "seg_indptr": arr(h.seg_indptr, ctypes.c_int32, S + 1),
            "seg_adapter": arr(h.seg_adapter, ctypes.c_int32, S), "seg_rank": arr(h.seg_rank, ctypes.c_int32, S),
            "seg_A": arr(h.seg_A, ctypes.c_uint64, S), "seg_B": arr(h.seg_B, ctypes.c_uint64, S),
            "seg_scale": arr(h.seg_scale, ctypes.c_float, S)}


def sgmv_shrink(x, plan: Plan, v, dtype: str, stream=None):
    d_in = x.shape[1]
    _check(lora_sgmv_shrink(_stream_handle(stream), DTYPES[dtype], _ptr(x), x.stride(0), d_in,
                            plan.seg, _ptr(v), v.stride(0), None, 0),
           "lora_sgmv_shrink")


def sgmv_expand(v, plan: Plan, y, dtype: str, stream=None):
    _check(lora_sgmv_expand(_stream_handle(stream), DTYPES[dtype], _ptr(v), v.stride(0), plan.seg, _ptr(y),
                            y.stride(0), y.shape[1], None, 0),
           "lora_sgmv_expand")


def workspace(op: int, T: int, d_in: int, d_out: int, max_rank: int, device="cuda"):
    """A zero-filled device workspace of the size the library asks for (uint8
    tensor; lora_bgmv needs its control words zero before the first call)."""
    torch = _torch()
    n = lora_workspace_bytes(op, T, d_in, d_out, max_rank)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def workspace_clear(ws, stream=None):
    """lora_workspace_clear on a workspace tensor."""
    _check(load().lora_workspace_clear(_stream_handle(stream), _ptr(ws), ws.numel() * ws.element_size()),
           "lora_workspace_clear")


def workspace_status(ws) -> int:
    """The status word at the start of a BGMV workspace (synchronises)."""
    return int(ws[:4].view(_torch().int32).item())


def debug_wait_limit(polls: int):
    _check(load().lora_debug_wait_limit(int(polls)), "lora_debug_wait_limit")


def sgmv(x, plan: Plan, y, ws, dtype: str, stream=None):
    """y[perm] += scale (x[perm] A) B for the whole plan (shrink + expand)."""
    _check(lora_sgmv(_stream_handle(stream), DTYPES[dtype], _ptr(x), x.stride(0), x.shape[1], plan.seg, _ptr(y),
                     y.stride(0), y.shape[1], _ptr(ws), ws.numel() * ws.element_size()),
           "lora_sgmv")


def bgmv(x, ids_dev, pool: DevicePool, y, ws, dtype: str, max_rank: Optional[int] = None, stream=None):
    """Decode: y[t] += scale (x[t] A_ids[t]) B_ids[t] (shrink + expand)."""
    _check(lora_bgmv(_stream_handle(stream), DTYPES[dtype], x.shape[0], _ptr(x), x.stride(0), x.shape[1],
                     _ptr(ids_dev), _ptr(pool.addr_A_dev), _ptr(pool.addr_B_dev), _ptr(pool.rank_dev),
                     _ptr(pool.alpha_dev), pool.n_adapters, max_rank or pool.max_rank, _ptr(y), y.stride(0),
                     y.shape[1], _ptr(ws), ws.numel() * ws.element_size()),
           "lora_bgmv")


def sgmv_prepared(x, plan: Plan, y, ws, dtype: str, stream) -> Prepared:
    """lora_sgmv with its arguments converted once (see Prepared)."""
    return Prepared("lora_sgmv", (_stream_handle(stream), DTYPES[dtype], _ptr(x), x.stride(0), x.shape[1],
                                  plan.seg, _ptr(y), y.stride(0), y.shape[1],
                                  _ptr(ws), ws.numel() * ws.element_size()), keep=(x, plan, y, ws))


def bgmv_prepared(x, ids_dev, pool, y, ws, dtype: str, stream, max_rank: Optional[int] = None) -> Prepared:
    """lora_bgmv with its arguments converted once (see Prepared)."""
    return Prepared("lora_bgmv", (_stream_handle(stream), DTYPES[dtype], x.shape[0], _ptr(x), x.stride(0),
                                  x.shape[1], _ptr(ids_dev), _ptr(pool.addr_A_dev), _ptr(pool.addr_B_dev),
                                  _ptr(pool.rank_dev), _ptr(pool.alpha_dev), pool.n_adapters,
                                  max_rank or pool.max_rank, _ptr(y), y.stride(0), y.shape[1], _ptr(ws),
                                  ws.numel() * ws.element_size()), keep=(x, ids_dev, pool, y, ws))


def sgmv_paged_prepared(x, plan: Plan, pool: "PagedPool", y, ws, dtype: str, stream) -> Prepared:
    return Prepared("lora_sgmv_paged", (_stream_handle(stream), DTYPES[dtype], _ptr(x), x.stride(0), x.shape[1],
                                        plan.seg, _ptr(pool.pages),
                                        pool.page_bytes, _ptr(y), y.stride(0), y.shape[1], _ptr(ws),
                                        ws.numel() * ws.element_size()), keep=(x, plan, pool, y, ws))


def bgmv_paged_prepared(x, ids_dev, pool: "PagedPool", y, ws, dtype: str, stream,
                        max_rank: Optional[int] = None) -> Prepared:
    return Prepared("lora_bgmv_paged", (_stream_handle(stream), DTYPES[dtype], x.shape[0], _ptr(x), x.stride(0),
                                        x.shape[1], _ptr(ids_dev), _ptr(pool.addr_A_dev), _ptr(pool.addr_B_dev),
                                        _ptr(pool.rank_dev), _ptr(pool.alpha_dev), pool.n_adapters,
                                        max_rank or pool.max_rank, _ptr(pool.pages), pool.page_bytes, _ptr(y),
                                        y.stride(0), y.shape[1], _ptr(ws), ws.numel() * ws.element_size()),
                    keep=(x, ids_dev, pool, y, ws))


def fused_prepared(x, W0, plan: Plan, y, ws, dtype: str, stream) -> Prepared:
    return Prepared("lora_fused_linear", (_stream_handle(stream), DTYPES[dtype], _ptr(x), x.stride(0), x.shape[1],
                                          _ptr(W0), W0.shape[0], plan.seg,
                                          _ptr(y), y.stride(0), _ptr(ws), ws.numel() * ws.element_size()),
                    keep=(x, W0, plan, y, ws))


def fused_e4m3_prepared(x, W0, w0_scale: float, plan: Plan, y, ws, stream) -> Prepared:
    """W0: uint8 E4M3 codes [d_out, d_in] standing for w0_scale * code."""
    return Prepared("lora_fused_linear_e4m3", (_stream_handle(stream), _ptr(x), x.stride(0), x.shape[1], _ptr(W0),
                                               float(w0_scale), W0.shape[0], plan.seg, _ptr(y), y.stride(0), _ptr(ws),
                                               ws.numel() * ws.element_size()),
                    keep=(x, W0, plan, y, ws))


def sgmv_grouped_prepared(projs, ws, dtype: str, stream, keep=()) -> Prepared:
    return Prepared("lora_sgmv_grouped", (_stream_handle(stream), DTYPES[dtype], ctypes.cast(projs, _vp).value,
                                          len(projs), _ptr(ws), ws.numel() * ws.element_size()),
                    keep=(projs, ws, *keep))


def bgmv_grouped_prepared(T: int, ids_dev, n_adapters: int, projs, ws, dtype: str, stream, keep=()) -> Prepared:
    return Prepared("lora_bgmv_grouped", (_stream_handle(stream), DTYPES[dtype], T, _ptr(ids_dev), n_adapters,
                                          ctypes.cast(projs, _vp).value, len(projs), _ptr(ws),
                                          ws.numel() * ws.element_size()), keep=(ids_dev, projs, ws, *keep))


def sgmv_paged(x, plan: Plan, pool: PagedPool, y, ws, dtype: str, stream=None):
    """lora_sgmv over paged adapters (plan built from the PagedPool)."""
    _check(load().lora_sgmv_paged(_stream_handle(stream), DTYPES[dtype], _ptr(x), x.stride(0), x.shape[1],
                                  plan.seg, _ptr(pool.pages), pool.page_bytes,
                                  _ptr(y), y.stride(0), y.shape[1], _ptr(ws), ws.numel() * ws.element_size()),
           "lora_sgmv_paged")


def bgmv_paged(x, ids_dev, pool: PagedPool, y, ws, dtype: str, max_rank: Optional[int] = None, stream=None):
    """lora_bgmv over paged adapters."""
    _check(load().lora_bgmv_paged(_stream_handle(stream), DTYPES[dtype], x.shape[0], _ptr(x), x.stride(0),
                                  x.shape[1], _ptr(ids_dev), _ptr(pool.addr_A_dev), _ptr(pool.addr_B_dev),
                                  _ptr(pool.rank_dev), _ptr(pool.alpha_dev), pool.n_adapters,
                                  max_rank or pool.max_rank, _ptr(pool.pages), pool.page_bytes, _ptr(y), y.stride(0),
                                  y.shape[1], _ptr(ws), ws.numel() * ws.element_size()),
           "lora_bgmv_paged")


def sgmv_proj_array(xs, plans, ys):
    """Host array of struct lora_sgmv_proj for projections (xs[p], plans[p], ys[p])."""
    arr = (LoraSgmvProj * len(xs))()
    for p, (x, plan, y) in enumerate(zip(xs, plans, ys)):
        arr[p] = LoraSgmvProj(_ptr(x), _ptr(y), plan.seg, x.stride(0), y.stride(0),
                              x.shape[1], y.shape[1])
    return arr


def sgmv_grouped_workspace(plans_or_projs, xs=None, ys=None, device="cuda"):
    """A device workspace for lora_sgmv_grouped (uint8 tensor)."""
    torch = _torch()
    projs = plans_or_projs if xs is None else sgmv_proj_array(xs, plans_or_projs, ys)
    n = int(load().lora_sgmv_grouped_workspace_bytes(projs, len(projs)))
    if n == 0:
        raise LoraError(-1, "lora_sgmv_grouped_workspace_bytes", "invalid projections")
    return torch.empty(n, dtype=torch.uint8, device=device)


def sgmv_grouped(xs, plans, ys, ws, dtype: str, stream=None, projs=None):
    """Prefill correction of several projections in one shrink and one expand
    launch: projection p applies plans[p] (built from the batch's ids with its
    own adapter tables) to xs[p] and accumulates into ys[p]."""
    projs = projs if projs is not None else sgmv_proj_array(xs, plans, ys)
    _check(load().lora_sgmv_grouped(_stream_handle(stream), DTYPES[dtype], projs, len(projs), _ptr(ws),
                                    ws.numel() * ws.element_size()), "lora_sgmv_grouped")


def proj_array(xs, pools, ys, max_ranks=None):
    """Host array of struct lora_proj for projections (xs[p], pools[p], ys[p])."""
    n = len(xs)
    arr = (LoraProj * n)()
    for p in range(n):
        x, pool, y = xs[p], pools[p], ys[p]
        arr[p] = LoraProj(_ptr(x), _ptr(y), _ptr(pool.addr_A_dev), _ptr(pool.addr_B_dev), _ptr(pool.rank_dev),
                          _ptr(pool.alpha_dev), x.stride(0), y.stride(0), x.shape[1], y.shape[1],
                          int(max_ranks[p]) if max_ranks is not None else max(pool.max_rank, 1), 0)
    return arr


def bgmv_grouped_workspace(T: int, projs, device="cuda"):
    torch = _torch()
    nbytes = lora_bgmv_grouped_workspace_bytes(T, ctypes.cast(projs, _vp), len(projs))
    if nbytes == 0 and T > 0:
        raise ValueError("invalid projections for a grouped workspace")
    # zero-filled: the status word at its start must begin at zero
    return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def bgmv_grouped(xs, ids_dev, pools, ys, ws, dtype: str, max_ranks=None, stream=None, projs=None):
    """Decode for several projections in one shrink and one expand launch:
    ys[p][t] += scale (xs[p][t] A_{ids[t],p}) B_{ids[t],p}.  All pools share the
    adapter numbering of ids_dev."""
    n_adapters = pools[0].n_adapters
    if any(p.n_adapters != n_adapters for p in pools):
        raise ValueError("every projection's pool must number the same adapters as ids_dev")
    if projs is None:
        projs = proj_array(xs, pools, ys, max_ranks)
    T = xs[0].shape[0]
    _check(lora_bgmv_grouped(_stream_handle(stream), DTYPES[dtype], T, _ptr(ids_dev), n_adapters,
                             ctypes.cast(projs, _vp), len(projs), _ptr(ws), ws.numel() * ws.element_size()),
           "lora_bgmv_grouped")


def bgmv_shrink(x, ids_dev, pool: DevicePool, v, dtype: str, max_rank: Optional[int] = None, stream=None):
    _check(lora_bgmv_shrink(_stream_handle(stream), DTYPES[dtype], x.shape[0], _ptr(x), x.stride(0), x.shape[1],
                            _ptr(ids_dev), _ptr(pool.addr_A_dev), _ptr(pool.rank_dev), pool.n_adapters,
                            max_rank or pool.max_rank, _ptr(v), v.stride(0), None, 0),
           "lora_bgmv_shrink")


def bgmv_expand(v, ids_dev, pool: DevicePool, y, dtype: str, max_rank: Optional[int] = None, stream=None):
    _check(lora_bgmv_expand(_stream_handle(stream), DTYPES[dtype], y.shape[0], _ptr(v), v.stride(0), _ptr(ids_dev),
                            _ptr(pool.addr_B_dev), _ptr(pool.rank_dev), _ptr(pool.alpha_dev), pool.n_adapters,
                            max_rank or pool.max_rank, _ptr(y), y.stride(0), y.shape[1], None, 0),
           "lora_bgmv_expand")


def fused_linear(x, W0, plan: Plan, y, ws, dtype: str = "bf16", stream=None):
    _check(lora_fused_linear(_stream_handle(stream), DTYPES[dtype], _ptr(x), x.stride(0), x.shape[1], _ptr(W0),
                             W0.shape[0], plan.seg, _ptr(y), y.stride(0),
                             _ptr(ws), ws.numel() * ws.element_size()),
           "lora_fused_linear")


def fused_linear_e4m3(x, W0, w0_scale: float, plan: Plan, y, ws, stream=None):
    """The fused layer over an FP8 base: W0 holds uint8 E4M3 codes [d_out, d_in]
    standing for w0_scale * code; x, y and the adapters are bf16."""
    _check(lora_fused_linear_e4m3(_stream_handle(stream), _ptr(x), x.stride(0), x.shape[1], _ptr(W0),
                                  float(w0_scale), W0.shape[0], plan.seg, _ptr(y), y.stride(0),
                                  _ptr(ws), ws.numel() * ws.element_size()),
           "lora_fused_linear_e4m3")


_SCALE_TYPES = None


def _scale_type(scales) -> int:
    """LORA_SCALE_F32 or LORA_SCALE_E8M0 by the tensor's type."""
    global _SCALE_TYPES
    if _SCALE_TYPES is None:
        torch = _torch()
        _SCALE_TYPES = {torch.float32: LORA_SCALE_F32, torch.uint8: LORA_SCALE_E8M0}
    kind = _SCALE_TYPES.get(scales.dtype)
    if kind is None:
        raise ValueError(f"scales are float32, or uint8 (E8M0), not {scales.dtype}")
    return kind


def _rows_of(t, dtype, rows, cols, device, least=False):
    """Address and row pitch of a matrix of `rows` (least: or more) x `cols` adjacent elements on the
    device; refuses what the C call cannot see.  The pitch of a single row is any."""
    n, d = t.shape
    ld, inner = t.stride()
    if (n != rows and not (least and n > rows)) or d != cols or t.dtype is not dtype or (inner != 1 and d > 1):
        raise ValueError(f"{rows} rows of {cols} adjacent elements of {dtype} are wanted, not {tuple(t.shape)} of {t.dtype} "
                         f"at strides {t.stride()}")
    if t.get_device() != device:
        raise ValueError(f"a tensor of {tuple(t.shape)} is not on the current device")
    if n >> 31 or d >> 31:  # the C call's counts have 32 bits
        raise ValueError(f"a tensor of {tuple(t.shape)} has 2^31 rows or columns or more")
    return t.data_ptr(), ld if n > 1 else (d + 15) // 16 * 16


def quantize_e4m3(x, codes, scales, block_rows: int = 1, stream=None):
    """E4M3 codes (uint8, x's shape) of a bf16 or fp32 matrix with a scale for each block of
    1 x 128 (block_rows 1; scales [groups, rows]) or 128 x 128 elements (block_rows 128;
    scales [row blocks, groups]).  The scales' type says which: float32, or uint8 for
    powers of two (E8M0)."""
    torch = _torch()
    device = torch.cuda.current_device()
    rows, cols = x.shape
    dt = x.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise ValueError(f"x is bf16 or fp32, not {dt}")
    groups = (cols + 127) // SCALE_BLOCK
    px, ldx = _rows_of(x, dt, rows, cols, device)
    pc, ldc = _rows_of(codes, torch.uint8, rows, cols, device)
    kind = _scale_type(scales)
    if block_rows == 1:
        ps, lds = _rows_of(scales, scales.dtype, groups, rows, device)
    else:
        ps, lds = _rows_of(scales, scales.dtype, (rows + 127) // SCALE_BLOCK, groups, device)
    st = load().lora_quantize_e4m3(_stream_handle(stream, device), LORA_BF16 if dt is torch.bfloat16 else LORA_F32, px, ldx,
                                   rows, cols, block_rows, kind, pc, ldc, ps, lds)
    if st:
        _check(st, "lora_quantize_e4m3")


def _block_base(W, w_scales, device):
    """d_out, d_in, addresses of codes and scales, and the scales' type of a block-scaled base."""
    torch = _torch()
    d_out, d_in = W.shape
    kind = _scale_type(w_scales)
    if not W.is_contiguous() or not w_scales.is_contiguous():
        raise ValueError("W and its scales are contiguous")
    pW, _ = _rows_of(W, torch.uint8, d_out, d_in, device)
    ps, _ = _rows_of(w_scales, w_scales.dtype, (d_out + 127) // SCALE_BLOCK, (d_in + 127) // SCALE_BLOCK, device)
    return d_out, d_in, pW, ps, kind


def linear_e4m3_block(x, x_scales, W, w_scales, y, ws=None, stream=None):
    """y = (x_scales x) (w_scales W)^T for E4M3 codes x [T, d_in] (scales [groups, T]) and W
    [d_out, d_in] (scales for each 128 x 128 block, of the same type); y bf16 or fp32,
    overwritten.  ws: a workspace of LORA_OP_LINEAR_BLOCK, which needs none (None)."""
    torch = _torch()
    device = torch.cuda.current_device()
    d_out, d_in, pW, pws, kind = _block_base(W, w_scales, device)
    T = x.shape[0]
    dt = y.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise ValueError(f"y is bf16 or fp32, not {dt}")
    px, ldx = _rows_of(x, torch.uint8, T, d_in, device)
    ps, lds = _rows_of(x_scales, w_scales.dtype, (d_in + 127) // SCALE_BLOCK, T, device)
    py, ldy = _rows_of(y, dt, T, d_out, device)
    if ws is not None and ws.get_device() != device:
        raise ValueError("the workspace is not on the current device")
    st = load().lora_linear_e4m3_block(_stream_handle(stream, device), T, px, ldx, ps, lds, d_in, pW, pws, kind, d_out,
                                       LORA_BF16 if dt is torch.bfloat16 else LORA_F32, py, ldy, _ptr(ws),
                                       0 if ws is None else ws.numel() * ws.element_size())
    if st:
        _check(st, "lora_linear_e4m3_block")


def fused_linear_e4m3_block(x, W0, w_scales, plan, y, ws, stream=None):
    """The fused layer over an E4M3 base with a scale for each 128 x 128 block: x (bf16) is
    quantized by the call, in groups of 128 columns with scales of the same type; the
    correction is x's own.  plan: a Plan or a DevicePlan; ws: of LORA_OP_FUSED_BLOCK."""
    torch = _torch()
    device = torch.cuda.current_device()
    d_out, d_in, pW, pws, kind = _block_base(W0, w_scales, device)
    T = plan.h.batch_tokens
    px, ldx = _rows_of(x, torch.bfloat16, T, d_in, device, least=True)
    py, ldy = _rows_of(y, torch.bfloat16, T, d_out, device, least=True)
    if plan.paged:
        raise ValueError("the plan's adapters are paged; this call takes whole matrices")
    if plan.made_for is not None and plan.made_for != (d_in, d_out, "bf16"):
        raise ValueError(f"a call of ({d_in}, {d_out}, bf16) on a plan of adapters of {plan.made_for}")
    if ws.get_device() != device or plan.dev.get_device() != device:
        raise ValueError("the plan or the workspace is not on the current device")
    st = load().lora_fused_linear_e4m3_block(_stream_handle(stream, device), px, ldx, d_in, pW, pws, kind, d_out, plan.seg, py,
                                             ldy, ws.data_ptr(), ws.numel() * ws.element_size())
    if st:
        _check(st, "lora_fused_linear_e4m3_block")


def _gradient_rows(dtype: str, tokens: int, others, rows):
    """Refuses what the C call cannot see: matrices (pairs of one, or None, and its
    columns, None for any; the first is not None) of another type, shape or device than
    the call's, and other tensors of another device.  Returns the device and, for each
    matrix, its address and row pitch (its columns for None)."""
    torch = _torch()
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    device = torch.cuda.current_device() if rows[0][0].get_device() >= 0 else -1
    out = []
    for t, cols in rows:
        if t is None:
            out += (None, cols)
            continue
        n, d = t.shape
        if t.get_device() != device or device < 0:
            raise ValueError(f"a tensor of {tuple(t.shape)} is not on the current device")
        ld, inner = t.stride()
        if n < tokens or (cols is not None and d != cols) or t.dtype is not dt or (inner != 1 and d > 1):
            raise ValueError(f"{tokens} rows of {d if cols is None else cols} adjacent elements of {dt} are wanted, "
                             f"not {tuple(t.shape)} of {t.dtype}")
        out += (t.data_ptr(), ld)
    for t in others:
        if t.get_device() != device:
            raise ValueError("the plan, the workspace or grads are not on the current device")
    return device, out


def _fits_plan(plan: Plan, d_in: int, d_out: int, dtype: str, grads: Optional[GradPool], device: int):
    """Refuses sizes other than those of the adapters that the plan was built from: the
    kernels read A and B, and write the gradients, at the call's widths and the plan's
    ranks.  The gradients are looked at once for each plan built.  Paged adapters have
    no gradient calls: their page tables would be read as A and B."""
    if plan.paged:
        raise ValueError("the plan's adapters are paged; the gradient calls take whole matrices")
    if plan.made_for is None or plan.h.num_segments == 0:  # built without a Plan; no adapter is touched
        return
    if plan.made_for != (d_in, d_out, dtype):
        raise ValueError(f"a call of ({d_in}, {d_out}, {dtype}) on a plan of adapters of {plan.made_for}")
    if grads is None or (plan.grads_fit is not None and plan.grads_fit() is grads):
        return
    t = plan.segment_table()
    for i, r in zip(t["seg_adapter"].tolist(), t["seg_rank"].tolist()):
        for g, n in ((grads.A, r * d_in), (grads.B, r * d_out)):
            if i < len(g) and g[i] is not None and (g[i].numel() < n or g[i].get_device() != device):
                raise ValueError(f"a gradient of adapter {i} of {g[i].numel()} elements on {g[i].device}; {n} on the "
                                 "current device are wanted")
    plan.grads_fit = weakref.ref(grads)


def sgmv_backward(x, dy, plan: Plan, grads: Optional[GradPool], dx, ws, dtype: str, accumulate: bool = False,
                  stream=None):
    """Gradients of sgmv: dx[perm] += u A (dx None: not wanted), grads.A = u^T x,
    grads.B = dy^T v over each adapter's rows (added to them with accumulate;
    grads None: not wanted).  Widths, type and gradients are those of the pool that
    the plan was built from; others are refused, and so are plans of a PagedPool."""
    if x is not None or dx is not None:
        d_in = (dx if x is None else x).shape[-1]
    elif grads is not None:
        raise ValueError("x is None")
    else:
        return  # nothing is wanted
    tA, tB, n = (None, None, 0) if grads is None else (grads.addr_A_dev, grads.addr_B_dev, grads.n_adapters)
    device, (pdy, lddy, px, ldx, pdx, lddx) = _gradient_rows(
        dtype, plan.h.batch_tokens, (plan.dev, ws) if grads is None else (plan.dev, ws, tA, tB),
        ((dy, None), (x, d_in), (dx, d_in)))
    _fits_plan(plan, d_in, dy.shape[1], dtype, grads, device)
    _check(load().lora_sgmv_backward(_stream_handle(stream, device), DTYPES[dtype], px, ldx, d_in, pdy, lddy,
                                     dy.shape[1], plan.seg, _ptr(tA), _ptr(tB), n,
                                     LORA_GRAD_ACCUMULATE if accumulate else 0, pdx, lddx, ws.data_ptr(),
                                     ws.numel() * ws.element_size()),
           "lora_sgmv_backward")


def fused_linear_backward(x, W0, dy, plan: Plan, grads: Optional[GradPool], dx, ws, dtype: str = "bf16",
                          accumulate: bool = False, stream=None):
    """Gradients of fused_linear: dx = dy W0 + u A (overwritten, every row), and the
    adapters' gradients as in sgmv_backward (grads None: not wanted; x may then be None;
    what is refused is the same)."""
    d_out, d_in = W0.shape
    if not W0.is_contiguous():
        raise ValueError("W0 is contiguous [d_out, d_in]")
    tA, tB, n = (None, None, 0) if grads is None else (grads.addr_A_dev, grads.addr_B_dev, grads.n_adapters)
    device, (pdy, lddy, px, ldx, pdx, lddx) = _gradient_rows(
        dtype, plan.h.batch_tokens, (plan.dev, ws) if grads is None else (plan.dev, ws, tA, tB),
        ((dy, d_out), (x, d_in), (dx, d_in)))
    _, (pW0, _) = _gradient_rows(dtype, d_out, (), ((W0, d_in),))
    _fits_plan(plan, d_in, d_out, dtype, grads, device)
    _check(load().lora_fused_linear_backward(_stream_handle(stream, device), DTYPES[dtype], px, ldx, d_in, pW0, pdy,
                                             lddy, d_out, plan.seg, _ptr(tA), _ptr(tB), n,
                                             LORA_GRAD_ACCUMULATE if accumulate else 0, pdx, lddx, ws.data_ptr(),
                                             ws.numel() * ws.element_size()),
           "lora_fused_linear_backward")


def fused_linear_e4m3_block_backward(x, W0, w_scales, dy, plan: Plan, grads: Optional[GradPool], dx, ws,
                                     accumulate: bool = False, stream=None):
    """Gradients of fused_linear_e4m3_block: dx = Q(dy) W0 + u A (overwritten, every row; Q quantizes
    groups of 128 columns with scales of the base's type), and the adapters' gradients as in
    sgmv_backward (grads None: not wanted; x may then be None; what is refused is the same)."""
    d_out, d_in, pW, pws, kind = _block_base(W0, w_scales, _torch().cuda.current_device())
    tA, tB, n = (None, None, 0) if grads is None else (grads.addr_A_dev, grads.addr_B_dev, grads.n_adapters)
    device, (pdy, lddy, px, ldx, pdx, lddx) = _gradient_rows(
        "bf16", plan.h.batch_tokens, (plan.dev, ws) if grads is None else (plan.dev, ws, tA, tB),
        ((dy, d_out), (x, d_in), (dx, d_in)))
    _fits_plan(plan, d_in, d_out, "bf16", grads, device)
    _check(load().lora_fused_linear_e4m3_block_backward(
        _stream_handle(stream, device), px, ldx, d_in, pW, pws, kind, pdy, lddy,
        d_out, plan.seg, _ptr(tA), _ptr(tB), n, LORA_GRAD_ACCUMULATE if accumulate else 0, pdx, lddx, ws.data_ptr(),
        ws.numel() * ws.element_size()), "lora_fused_linear_e4m3_block_backward")


def adamw_hyper(n_groups: int, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0, step=1,
                seed=0, device="cuda"):
    """The device table of lora_adamw, int32 [n_groups, 8] (columns 0 .. 5 hold
    fp32 bits, 6 the step, 7 the seed).  Each argument is a number or one value
    for each group.  `hyper[:, 6] += 1` counts a step on the device."""
    torch = _torch()

    def column(v, dtype):
        t = torch.as_tensor(v, device=device)
        t = (t.to(torch.int64) & 0xFFFFFFFF).to(torch.int32) if dtype is torch.int32 else t.to(dtype)
        return t.expand(n_groups).contiguous().view(torch.int32)

    floats = (lr, beta1, beta2, eps, weight_decay, grad_scale)
    return torch.stack([*(column(v, torch.float32) for v in floats), column(step, torch.int32),
                        column(seed, torch.int32)], 1)


class AdamW:
    """AdamW over many tensors in one launch (lora_adamw): params are fp32 device
    tensors, grads fp32 or bf16 ones (all of one dtype), copies optional bf16
    tensors that receive the rounded parameters.  groups[i] is the entry of
    `hyper` (see adamw_hyper) that tensor i goes by.  state: "f32" or "8bit";
    m, v (and m_scale, v_scale for 8-bit states) are lists of state tensors, made
    here as zeros when not given.  stream: where the plan is uploaded.  The states
    and the plan are complete when the constructor returns (it waits for the current
    stream and for `stream`, so it is not for a captured region), so that steps may go
    to any stream; they are used until the steps given are done."""

    def __init__(self, params, grads, groups, hyper, state: str = "f32", copies=None, m=None, v=None, m_scale=None,
                 v_scale=None, stream=None):
        torch = _torch()
        if state not in ("f32", "8bit"):
            raise ValueError("state is 'f32' or '8bit'")
        if hyper.is_cuda and torch.cuda.is_current_stream_capturing():
            raise ValueError("AdamW is built outside of a captured region; its steps may be captured")
        eight, device = state == "8bit", params[0].device if params else hyper.device
        made = lambda given, size, dt: list(given) if given is not None else [  # noqa: E731
            torch.zeros(size(p.numel()), dtype=dt, device=p.device) for p in params]
        blocks = lambda n: (n + ADAM_BLOCK - 1) // ADAM_BLOCK  # noqa: E731
        # lists of its own: the plan holds addresses, so every tensor lives as long as this
        copies = None if copies is None else list(copies)
        self.params, self.grads, self.copies, self.hyper, self.state = list(params), list(grads), copies, hyper, state
        self.m = made(m, lambda n: n, torch.uint8 if eight else torch.float32)
        self.v = made(v, lambda n: n, torch.uint8 if eight else torch.float32)
        self.m_scale = made(m_scale, blocks, torch.uint8) if eight else None
        self.v_scale = made(v_scale, blocks, torch.uint8) if eight else None
        gdt = self.grads[0].dtype if self.grads else torch.float32
        if gdt not in (torch.float32, torch.bfloat16):
            raise ValueError("gradients are fp32 or bf16")
        if hyper.dtype != torch.int32 or hyper.dim() != 2 or hyper.shape[1] != 8 or not hyper.is_contiguous():
            raise ValueError("hyper is the int32 [n_groups, 8] table of adamw_hyper")
        if not hyper.is_cuda or hyper.device != device or hyper.get_device() != torch.cuda.current_device():
            raise ValueError("params and hyper are on the current device")
        n = len(self.params)
        sdt = torch.uint8 if eight else torch.float32
        lists = [("params", self.params, torch.float32, None), ("grads", self.grads, gdt, None),
                 ("m", self.m, sdt, None), ("v", self.v, sdt, None)]
        lists += [("copies", copies, torch.bfloat16, None)] if copies is not None else []
        lists += [("m_scale", self.m_scale, sdt, blocks), ("v_scale", self.v_scale, sdt, blocks)] if eight else []
        for name, ts, dt, size in lists:
            if len(ts) != n or len(groups) != n:
                raise ValueError(f"{name} and groups list one entry for each parameter")
            for t, p in zip(ts, self.params):
                want = size(p.numel()) if size else p.numel()
                if t is None or t.dtype != dt or t.numel() != want or not t.is_contiguous() or t.device != device:
                    raise ValueError(f"{name}: contiguous {dt} tensors of {want} elements on the device of hyper")
        arr = (LoraAdamTensor * max(n, 1))()
        for i, p in enumerate(self.params):
            arr[i] = LoraAdamTensor(_ptr(p), _ptr(self.grads[i]), _ptr(copies[i]) if copies is not None else 0,
                                    _ptr(self.m[i]), _ptr(self.v[i]), _ptr(self.m_scale[i]) if eight else 0,
                                    _ptr(self.v_scale[i]) if eight else 0, p.numel(), int(groups[i]), 0)
        lib = load()
        nbytes = int(lib.lora_adamw_plan_bytes(arr, n))
        self._host = torch.empty(max(nbytes, 16), dtype=torch.uint8, pin_memory=True)
        self._dev = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
        _check(lib.lora_adamw_plan(arr, n, hyper.shape[0], LORA_ADAM_8BIT if eight else LORA_ADAM_F32,
                                   LORA_BF16 if gdt == torch.bfloat16 else LORA_F32, _ptr(self._host), nbytes),
               "lora_adamw_plan")
        # zeros and the plan's memory belong to the current stream, the upload to `stream`,
        # the steps to others: each waits for the one before
        made_on = torch.cuda.current_stream()
        if stream is not None:
            made_on.synchronize()
        _check(lib.lora_adamw_upload(_ptr(self._host), _ptr(self._dev), nbytes, _stream_handle(stream)),
               "lora_adamw_upload")
        (stream or made_on).synchronize()
        self._fn, self._device = lib.lora_adamw, hyper.get_device()
        self._args = (_vp(_ptr(self._host)), _vp(_ptr(self._dev)), _vp(_ptr(hyper)), _i32(hyper.shape[0]))

    def step(self, stream=None):
        """One step of every tensor, with the numbers that `hyper` holds on the device."""
        if self._device != _torch().cuda.current_device():
            raise ValueError("the tensors are not on the current device")
        st = self._fn(_stream_handle(stream, self._device), *self._args)
        if st:
            _check(st, "lora_adamw")


def adamw_state_values(m, m_scale, v, v_scale, m_out, v_out, stream=None):
    """bf16 values of 8-bit states: flat code tensors (uint8), their scales (one
    for each 256 elements) and bf16 outputs; m or v may be None."""
    torch = _torch()
    if m is None and v is None:
        return
    n = (v if m is None else m).numel()
    sides = [s for s in ((m, m_scale, m_out), (v, v_scale, v_out)) if s[0] is not None]
    for side in sides:
        for t, dt, size in zip(side, (torch.uint8, torch.uint8, torch.bfloat16), (n, (n + ADAM_BLOCK - 1) // ADAM_BLOCK, n)):
            if t is None or t.dtype != dt or t.numel() < size or not t.is_contiguous():
                raise ValueError(f"contiguous codes (uint8) and values (bf16) of {n} elements, one scale for each {ADAM_BLOCK}")
    if any(t.get_device() < 0 or t.get_device() != torch.cuda.current_device() for side in sides for t in side):
        raise ValueError("the states are not on the current device")
    _check(load().lora_adam_state_values(_stream_handle(stream), n, _ptr(m), _ptr(m_scale), _ptr(v), _ptr(v_scale),
                                         _ptr(m_out), _ptr(v_out)), "lora_adam_state_values")


def v_pitch(max_rank: int) -> int:
    """Row pitch (fp32 elements) for v: max rank rounded up to a multiple of 4."""
    return max(4, (int(max_rank) + 3) // 4 * 4)
