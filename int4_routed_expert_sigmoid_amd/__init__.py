"""Python binding of libcoli_moe (one int4 routed-expert MoE layer, MI355X).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels (``csrc/``); this module turns torch tensors into device pointers and
the current torch stream into a ``hipStream_t``. The names follow the C ABI in
``include/coli_moe.h``. There is no CPU fallback: if the library is missing,
``lib()`` raises. Autograd records none of the calls: results of tensors that
require a gradient are detached, and the gradients that exist (``dispatch_bwd``,
``combine_bwd``, ``route_groups_bwd``, ``fp8_wgrad``, and ``fp8_matmul`` with transposed
matrices) are calls of their own.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
SO_PATH = os.path.join(HERE, "libcoli_moe.so")

COLI_OK, COLI_EINVAL, COLI_EUNSUPPORTED, COLI_EHIP, COLI_ENOMEM, COLI_EBUSY = 0, -1, -2, -3, -4, -5
PATH_AUTO, PATH_GEMV, PATH_MFMA = 0, 1, 2
F32, BF16, F16, MXFP4, FP8 = 0, 1, 2, 3, 4

EXPORTED = [
    "coli_last_error", "coli_version", "coli_expert_blob_layout", "coli_quantize_int4",
    "coli_quantize_expert", "coli_convert_fp8_int4", "coli_convert_fp8_expert",
    "coli_moe_router_logits", "coli_moe_route", "coli_moe_route_topp",
    "coli_moe_union_workspace_size", "coli_moe_union", "coli_moe_workspace_size",
    "coli_moe_expert_ffn", "coli_moe_layer_fwd", "coli_moe_layer_fwd_noalloc",
    "coli_expert_cache_create",
    "coli_expert_cache_destroy", "coli_expert_cache_ensure", "coli_expert_cache_wait",
    "coli_expert_cache_release", "coli_expert_cache_table", "coli_expert_cache_stats",
    "coli_expert_cache_reset", "coli_expert_cache_pin", "coli_expert_cache_usage",
    "coli_expert_cache_pin_hot", "coli_expert_cache_repin", "coli_expert_cache_prefetch",
    "coli_moe_lookahead", "coli_debug_fail_copies", "coli_debug_read_log",
    "coli_profile_enable", "coli_profile_clear",
    "coli_profile_summary", "coli_profile_rerun", "coli_read_probe",
    "coli_quantize_mxfp4", "coli_dequantize_mxfp4", "coli_mxfp4_blob_layout",
    "coli_quantize_mxfp4_expert", "coli_mxfp4_matmul", "coli_mxfp4_swiglu", "coli_debug_mxfp4_kernel",
    "coli_moe_union_inverse", "coli_moe_dispatch", "coli_moe_dispatch_mxfp4",
    "coli_moe_dispatch_bwd", "coli_moe_combine", "coli_moe_combine_bwd",
    "coli_moe_route_groups", "coli_moe_route_groups_bwd",
    "coli_quantize_fp8", "coli_quantize_fp8_matrix", "coli_quantize_fp8_columns", "coli_fp8_column_blocks",
    "coli_dequantize_fp8", "coli_dequantize_fp8_matrix", "coli_fp8_blob_layout", "coli_fp8_matmul", "coli_fp8_matmul_workspace_size", "coli_fp8_swiglu",
    "coli_fp8_swiglu_workspace_size", "coli_fp8_wgrad", "coli_fp8_wgrad_workspace_size",
    "coli_debug_fp8_kernel", "coli_moe_dispatch_fp8",
]


class ColiError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"coli status {code}: {msg}")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_routed", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("group", ctypes.c_int32),
                ("routed_scale", ctypes.c_float), ("topp", ctypes.c_float),
                ("wbits", ctypes.c_int32)]


class CacheCfg(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("slots_per_layer", ctypes.c_int32), ("blob_bytes", ctypes.c_size_t),
                ("d_arena", ctypes.c_void_p), ("h_pools", ctypes.c_void_p),
                ("copy_stream", ctypes.c_void_p)]


class CacheStats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_uint64), ("misses", ctypes.c_uint64),
                ("evictions", ctypes.c_uint64), ("bytes_h2d", ctypes.c_uint64),
                ("copy_ns", ctypes.c_uint64), ("lookups", ctypes.c_uint64),
                ("pin_hits", ctypes.c_uint64), ("pin_loads", ctypes.c_uint64),
                ("prefetches", ctypes.c_uint64), ("prefetch_hits", ctypes.c_uint64),
                ("repin_swaps", ctypes.c_uint64)]


_lock = threading.Lock()
_lib = None


def lib():
    """Load libcoli_moe.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(SO_PATH):
                raise ImportError(f"{SO_PATH} is missing: run __graft_entry__.build() first")
            L = ctypes.CDLL(SO_PATH)
            vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
            f32 = ctypes.c_float
            P = ctypes.POINTER
            for name in EXPORTED:
                getattr(L, name).restype = ctypes.c_int32
            L.coli_last_error.restype = ctypes.c_char_p
            L.coli_version.restype = ctypes.c_char_p
            L.coli_expert_blob_layout.argtypes = [P(Shape), P(sz), P(sz)]
            L.coli_quantize_int4.argtypes = [vp, i64, i64, i32, vp, vp, vp]
            L.coli_quantize_expert.argtypes = [P(Shape), vp, vp, vp, vp, vp]
            L.coli_convert_fp8_int4.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp]
            L.coli_convert_fp8_expert.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, vp, vp]
            L.coli_moe_router_logits.argtypes = [vp, vp, i32, i32, i32, vp, vp]
            L.coli_moe_route.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp]
            L.coli_moe_route_topp.argtypes = [vp, vp, i32, i32, i32, f32, vp, vp, vp]
            L.coli_moe_union_workspace_size.argtypes = [i32, i32, i32, P(sz)]
            L.coli_moe_union.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
            L.coli_moe_workspace_size.argtypes = [P(Shape), i32, i32, P(sz)]
            L.coli_moe_expert_ffn.argtypes = [P(Shape), vp, vp, i32, vp, vp, vp, vp, vp, i32, vp,
                                              sz, vp]
            L.coli_moe_layer_fwd.argtypes = [P(Shape), vp, i32, vp, vp, vp, vp, vp, vp, i32, vp,
                                             vp, vp, i32, vp, sz, vp]
            L.coli_moe_layer_fwd_noalloc.argtypes = [P(Shape), vp, i32, vp, vp, vp, vp, vp, vp, vp,
                                                     vp, i32, vp]
            L.coli_expert_cache_create.argtypes = [P(CacheCfg), P(vp)]
            L.coli_expert_cache_destroy.argtypes = [vp]
            L.coli_expert_cache_ensure.argtypes = [vp, i32, vp, i32, vp]
            L.coli_expert_cache_wait.argtypes = [vp, i32, vp]
            L.coli_expert_cache_release.argtypes = [vp, i32, vp]
            L.coli_expert_cache_table.argtypes = [vp, i32, P(vp)]
            L.coli_expert_cache_stats.argtypes = [vp, P(CacheStats)]
            L.coli_expert_cache_reset.argtypes = [vp]
            L.coli_expert_cache_pin.argtypes = [vp, i32, vp, i32]
            L.coli_expert_cache_usage.argtypes = [vp, vp]
            L.coli_expert_cache_pin_hot.argtypes = [vp, vp, i32]
            L.coli_expert_cache_repin.argtypes = [vp, i32, f32, f32, P(i32)]
            L.coli_expert_cache_prefetch.argtypes = [vp, i32, vp, i32, P(i32)]
            L.coli_moe_lookahead.argtypes = [P(Shape), vp, i32, vp, vp, vp, vp, i32, P(i32), vp,
                                             sz, vp]
            L.coli_debug_fail_copies.argtypes = [i32]
            L.coli_debug_read_log.argtypes = [vp, vp, i32]
            L.coli_profile_enable.argtypes = [i32]
            L.coli_profile_clear.argtypes = []
            L.coli_profile_summary.argtypes = [ctypes.c_char_p, P(i64), P(ctypes.c_double)]
            L.coli_profile_rerun.argtypes = [P(Shape), i32, vp, vp, i32, vp, sz, vp]
            L.coli_read_probe.argtypes = [vp, sz, i32, i32, i32, vp, sz, vp]
            L.coli_quantize_mxfp4.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp]
            L.coli_dequantize_mxfp4.argtypes = [vp, vp, i64, i64, vp, i32, i64, vp]
            L.coli_mxfp4_blob_layout.argtypes = [P(Shape), P(sz), P(sz)]
            L.coli_quantize_mxfp4_expert.argtypes = [P(Shape), vp, vp, vp, i32, vp, vp]
            L.coli_mxfp4_matmul.argtypes = [vp, vp, i32, i32, vp, i32, vp, sz, sz, i32, vp, i32, i64,
                                            vp]
            L.coli_mxfp4_swiglu.argtypes = [vp, vp, i32, i32, vp, i32, vp, sz, sz, i32, vp, vp, i32,
                                            i64, vp]
            L.coli_debug_mxfp4_kernel.argtypes = [i32, i32, i32, i32, i32, i32, P(i32)]
            L.coli_moe_union_inverse.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            L.coli_moe_dispatch.argtypes = [vp, i32, i32, i32, i32, i64, vp, vp, i64, vp]
            L.coli_moe_dispatch_mxfp4.argtypes = [vp, i32, i32, i32, i32, i64, vp, vp, vp, vp]
            L.coli_moe_dispatch_bwd.argtypes = [vp, i32, i64, i32, i32, i32, vp, vp, i32, i64, vp]
            L.coli_moe_combine.argtypes = [vp, i32, i64, i32, i32, i32, vp, vp, vp, i64, f32, vp, i32,
                                           i64, vp]
            L.coli_moe_combine_bwd.argtypes = [vp, i32, i64, vp, i32, i64, i32, i32, i32, vp, vp, f32,
                                               vp, i64, vp, vp]
            L.coli_moe_route_groups.argtypes = [vp, i32, vp, i32, i32, i32, i32, i32, i32, i32, i32, f32,
                                                vp, vp, vp, vp]
            L.coli_moe_route_groups_bwd.argtypes = [vp, vp, i32, vp, i32, i32, i32, i32, i32, f32, vp, vp,
                                                    i32, vp]
            L.coli_quantize_fp8.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp]
            L.coli_quantize_fp8_matrix.argtypes = [vp, i32, i32, i64, i64, i64, i64, vp, i64, vp, i64, vp,
                                                   i64, vp, i64, vp]
            L.coli_quantize_fp8_columns.argtypes = [vp, i32, i32, i32, i64, vp, i32, vp, i64, vp, vp, vp, vp]
            L.coli_fp8_column_blocks.argtypes = [i32, i32, P(i64)]
            L.coli_dequantize_fp8.argtypes = [vp, vp, i64, i64, i32, vp, i32, i64, vp]
            L.coli_dequantize_fp8_matrix.argtypes = [vp, i64, vp, i64, i32, i64, i64, vp, i32, i64, i64, vp]
            L.coli_fp8_blob_layout.argtypes = [P(Shape), P(sz), P(sz)]
            L.coli_fp8_matmul.argtypes = [vp, vp, i32, i32, vp, i32, vp, sz, sz, i32, vp, i32, i64, vp, sz, vp]
            L.coli_fp8_matmul_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, P(sz)]
            L.coli_fp8_swiglu.argtypes = [vp, vp, i32, i32, vp, i32, vp, sz, sz, sz, sz, i32, vp, vp, i32,
                                          i64, vp, sz, vp]
            L.coli_fp8_swiglu_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, P(sz)]
            L.coli_fp8_wgrad.argtypes = [vp, vp, vp, vp, i64, i32, vp, i32, i32, i32, i32, vp, i32, i64, vp, sz, vp]
            L.coli_fp8_wgrad_workspace_size.argtypes = [i32, i32, i32, i32, P(sz)]
            L.coli_debug_fp8_kernel.argtypes = [i32, i32, i32, i32, i32, i32, i32, P(i32)]
            L.coli_moe_dispatch_fp8.argtypes = [vp, i32, i32, i32, i32, i64, vp, vp, vp, vp]
            _lib = L
    return _lib


def _check(rc: int):
    if rc != COLI_OK:
        raise ColiError(rc, lib().coli_last_error().decode(errors="replace"))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, dtype, name):
    import torch
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@dataclass
class MoEShape:
    hidden: int
    inter: int
    n_routed: int
    n_shared: int = 1
    top_k: int = 8
    group: int = 0
    routed_scale: float = 1.0
    topp: float = 0.0
    wbits: int = 4

    def c(self) -> Shape:
        return Shape(self.hidden, self.inter, self.n_routed, self.n_shared, self.top_k, self.group,
                     self.routed_scale, self.topp, self.wbits)


def version() -> str:
    return lib().coli_version().decode()


def blob_layout(shape: MoEShape):
    """(offsets of gate_q, up_q, down_q, gate_s, up_s, down_s; blob bytes)."""
    off = (ctypes.c_size_t * 6)()
    nb = ctypes.c_size_t()
    _check(lib().coli_expert_blob_layout(ctypes.byref(shape.c()), off, ctypes.byref(nb)))
    return list(off), nb.value


def quantize_int4(w, group=0, q=None, s=None, stream=None):
    import torch
    _need(w, torch.float32, "w")
    rows, cols = w.shape
    if q is None:
        q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=w.device)
    if s is None:
        s = torch.empty((rows,) if group == 0 else (rows, cols // 64), dtype=torch.float32,
                        device=w.device)
    _check(lib().coli_quantize_int4(_ptr(w), rows, cols, group, _ptr(q), _ptr(s), _stream(stream)))
    return q, s


def quantize_expert(shape: MoEShape, gate, up, down, blob=None, stream=None):
    import torch
    for t, n in ((gate, "gate"), (up, "up"), (down, "down")):
        _need(t, torch.float32, n)
    if blob is None:
        blob = torch.empty(blob_layout(shape)[1], dtype=torch.uint8, device=gate.device)
    _check(lib().coli_quantize_expert(ctypes.byref(shape.c()), _ptr(gate), _ptr(up), _ptr(down),
                                      _ptr(blob), _stream(stream)))
    return blob


def convert_fp8_int4(w8, scale, group=0, q=None, s=None, stream=None):
    """FP8 e4m3 codes (uint8 [rows][cols]) with block scales (f32
    [ceil(rows/128)][ceil(cols/128)]) -> (q uint8 [rows][cols/2], s f32)."""
    import torch
    _need(w8, torch.uint8, "w8")
    _need(scale, torch.float32, "scale")
    rows, cols = w8.shape
    if scale.numel() != ((rows + 127) // 128) * ((cols + 127) // 128):
        raise ValueError("scale must hold one value per 128 x 128 block")
    if q is None:
        q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=w8.device)
    if s is None:
        shp = (rows,) if group == 0 else (rows, cols // group)
        s = torch.empty(shp, dtype=torch.float32, device=w8.device)
    _check(lib().coli_convert_fp8_int4(_ptr(w8), _ptr(scale), rows, cols, group, _ptr(q), _ptr(s),
                                       _stream(stream)))
    return q, s


def convert_fp8_expert(shape: MoEShape, gate8, gate_scale, up8, up_scale, down8, down_scale,
                       blob=None, stream=None):
    import torch
    for t, n in ((gate8, "gate8"), (up8, "up8"), (down8, "down8")):
        _need(t, torch.uint8, n)
    for t, n in ((gate_scale, "gate_scale"), (up_scale, "up_scale"), (down_scale, "down_scale")):
        _need(t, torch.float32, n)
    H, I = shape.hidden, shape.inter
    for t, sc, r, c in ((gate8, gate_scale, I, H), (up8, up_scale, I, H), (down8, down_scale, H, I)):
        if tuple(t.shape) != (r, c) or sc.numel() != ((r + 127) // 128) * ((c + 127) // 128):
            raise ValueError("FP8 matrix or scale shape does not match the layer shape")
    if blob is None:
        blob = torch.empty(blob_layout(shape)[1], dtype=torch.uint8, device=gate8.device)
    _check(lib().coli_convert_fp8_expert(ctypes.byref(shape.c()), _ptr(gate8), _ptr(gate_scale),
                                         _ptr(up8), _ptr(up_scale), _ptr(down8), _ptr(down_scale),
                                         _ptr(blob), _stream(stream)))
    return blob


def router_logits(wr, x, out=None, stream=None):
    import torch
    _need(wr, torch.float32, "wr")
    _need(x, torch.float32, "x")
    E, H = wr.shape
    T = x.shape[0]
    if out is None:
        out = torch.empty((T, E), dtype=torch.float32, device=x.device)
    _check(lib().coli_moe_router_logits(_ptr(wr), _ptr(x), T, H, E, _ptr(out), _stream(stream)))
    return out


def route(logits, bias, k, idx=None, w=None, stream=None, topp=None):
    """coli_moe_route, or coli_moe_route_topp when topp is given."""
    import torch
    _need(logits, torch.float32, "logits")
    _need(bias, torch.float32, "bias")
    T, E = logits.shape
    if idx is None:
        idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    if topp is None:
        _check(lib().coli_moe_route(_ptr(logits), _ptr(bias), T, E, k, _ptr(idx), _ptr(w),
                                    _stream(stream)))
    else:
        _check(lib().coli_moe_route_topp(_ptr(logits), _ptr(bias), T, E, k, float(topp), _ptr(idx),
                                         _ptr(w), _stream(stream)))
    return idx, w


def union(idx, E, stream=None):
    import torch
    _need(idx, torch.int32, "idx")
    T, k = idx.shape
    dev = idx.device
    nb = ctypes.c_size_t()
    _check(lib().coli_moe_union_workspace_size(T, k, E, ctypes.byref(nb)))
    ws = torch.empty(max(1, nb.value), dtype=torch.uint8, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(1, T * k), dtype=torch.int32, device=dev)
    unique = torch.empty(E, dtype=torch.int32, device=dev)
    n_unique = torch.empty(1, dtype=torch.int32, device=dev)
    _check(lib().coli_moe_union(_ptr(idx), T, k, E, _ptr(counts), _ptr(offsets), _ptr(perm),
                                _ptr(unique), _ptr(n_unique), _ptr(ws), nb.value, _stream(stream)))
    return counts, offsets, perm[: T * k], unique, n_unique


def workspace_size(shape: MoEShape, T: int, path: int = PATH_AUTO) -> int:
    nb = ctypes.c_size_t()
    _check(lib().coli_moe_workspace_size(ctypes.byref(shape.c()), T, path, ctypes.byref(nb)))
    return nb.value


def workspace(shape: MoEShape, T: int, path: int = PATH_AUTO, device="cuda"):
    """A workspace of the size coli_moe_workspace_size gives (no initialisation
    needed: every call writes what it reads)."""
    import torch
    return torch.empty(max(1, workspace_size(shape, T, path)), dtype=torch.uint8, device=device)


def blob_table(blobs, device="cuda"):
    """Device array of blob pointers from a list of device tensors (or ints)."""
    import torch
    ptrs = [b if isinstance(b, int) else b.data_ptr() for b in blobs]
    return torch.tensor(ptrs, dtype=torch.int64, device=device)


def expert_ffn(shape: MoEShape, table, x, offsets, perm, unique, n_unique, y_assign=None,
               path=PATH_AUTO, ws=None, stream=None):
    import torch
    _need(x, torch.float32, "x")
    T = x.shape[0]
    if y_assign is None:
        y_assign = torch.zeros((T * shape.top_k, shape.hidden), dtype=torch.float32,
                               device=x.device)
    if ws is None:
        ws = workspace(shape, T, path, x.device)
    _check(lib().coli_moe_expert_ffn(ctypes.byref(shape.c()), _ptr(table), _ptr(x), T,
                                     _ptr(offsets), _ptr(perm), _ptr(unique), _ptr(n_unique),
                                     _ptr(y_assign), path, _ptr(ws), ws.numel(), _stream(stream)))
    return y_assign


def layer_fwd(shape: MoEShape, x, table=None, shared_blob=None, logits=None, router_w=None,
              bias=None, cache=None, layer=0, y=None, idx_out=None, w_out=None, path=PATH_AUTO,
              ws=None, stream=None):
    import torch
    _need(x, torch.float32, "x")
    T = x.shape[0]
    if y is None:
        y = torch.empty((T, shape.hidden), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(shape, T, path, x.device)
    _check(lib().coli_moe_layer_fwd(ctypes.byref(shape.c()), _ptr(x), T, _ptr(logits),
                                    _ptr(router_w), _ptr(bias), _ptr(table), _ptr(shared_blob),
                                    None if cache is None else ctypes.c_void_p(cache.handle), layer,
                                    _ptr(y), _ptr(idx_out), _ptr(w_out), path, _ptr(ws), ws.numel(),
                                    _stream(stream)))
    return y


def layer_fwd_noalloc(shape: MoEShape, x, table, shared_blob=None, logits=None, router_w=None,
                      bias=None, y=None, idx_out=None, w_out=None, path=PATH_AUTO, stream=None):
    """coli_moe_layer_fwd_noalloc: the layer on the library's static scratch
    (no workspace, no cache). `y` must be given to allocate nothing here too."""
    import torch
    _need(x, torch.float32, "x")
    T = x.shape[0]
    if y is None:
        y = torch.empty((T, shape.hidden), dtype=torch.float32, device=x.device)
    _check(lib().coli_moe_layer_fwd_noalloc(ctypes.byref(shape.c()), _ptr(x), T, _ptr(logits),
                                            _ptr(router_w), _ptr(bias), _ptr(table),
                                            _ptr(shared_blob), _ptr(y), _ptr(idx_out), _ptr(w_out),
                                            path, _stream(stream)))
    return y


class LayerCall:
    """coli_moe_layer_fwd with every argument but x, y and idx_out fixed, for
    loops of same-shaped calls (one-token decode): the argument objects are
    built once, so each call costs little host time. Pointers are device
    addresses (ints); the caller keeps the tensors alive."""

    def __init__(self, shape: MoEShape, T, ws, table=None, shared_blob=None, logits=None,
                 router_w=None, bias=None, cache=None, layer=0, path=PATH_AUTO, stream=None):
        self._shape = shape.c()
        self._fn = lib().coli_moe_layer_fwd
        self._keep = (ws, table, shared_blob, logits, router_w, bias, cache)
        self._args = [ctypes.byref(self._shape), None, T, _ptr(logits), _ptr(router_w),
                      _ptr(bias), _ptr(table), _ptr(shared_blob),
                      None if cache is None else ctypes.c_void_p(cache.handle), layer, None, None,
                      None, path, _ptr(ws), ws.numel(), _stream(stream)]

    def __call__(self, x_ptr: int, y_ptr: int, idx_ptr: int = 0, w_ptr: int = 0):
        a = self._args
        a[1], a[10], a[11], a[12] = x_ptr, y_ptr, idx_ptr or None, w_ptr or None
        rc = self._fn(*a)
        if rc != COLI_OK:
            _check(rc)


def lookahead(shape: MoEShape, x, cache, layer, logits=None, router_w=None, bias=None, ws=None,
              stream=None) -> int:
    """coli_moe_lookahead: route x with `layer`'s router and prefetch its picks;
    returns the number of copies started."""
    import torch
    _need(x, torch.float32, "x")
    T = x.shape[0]
    if ws is None:
        ws = workspace(shape, T, PATH_AUTO, x.device)
    n = ctypes.c_int32()
    _check(lib().coli_moe_lookahead(ctypes.byref(shape.c()), _ptr(x), T, _ptr(logits),
                                    _ptr(router_w), _ptr(bias), ctypes.c_void_p(cache.handle),
                                    layer, ctypes.byref(n), _ptr(ws), ws.numel(), _stream(stream)))
    return n.value


def debug_fail_copies(n: int):
    """coli_debug_fail_copies: the next n expert-cache copies fail (COLI_EHIP)
    before anything is enqueued."""
    _check(lib().coli_debug_fail_copies(n))


def debug_read_log(count=None, records=None):
    """coli_debug_read_log: log the weight tiles the GEMV kernels stream.
    count: a zeroed 1-element int32/uint32 device tensor; records: an int32
    device tensor [capacity, 4]. No arguments: log off."""
    if count is None:
        _check(lib().coli_debug_read_log(None, None, 0))
        return
    cap = 0 if records is None else int(records.shape[0])
    _check(lib().coli_debug_read_log(_ptr(count), _ptr(records), cap))


def profile_enable(max_records: int):
    _check(lib().coli_profile_enable(max_records))


def profile_clear():
    _check(lib().coli_profile_clear())


def profile_summary(name: str):
    """(launches timed, total milliseconds) for kernel `name`."""
    n = ctypes.c_int64()
    ms = ctypes.c_double()
    _check(lib().coli_profile_summary(name.encode(), ctypes.byref(n), ctypes.byref(ms)))
    return n.value, ms.value


def profile_rerun(shape: MoEShape, T: int, table, shared_blob, which: int, ws, stream=None):
    """coli_profile_rerun: one more launch of the gate/up (which=0) or down (1)
    GEMV pass of the last layer call made with `ws`."""
    _check(lib().coli_profile_rerun(ctypes.byref(shape.c()), T, _ptr(table), _ptr(shared_blob),
                                    which, _ptr(ws), ws.numel(), _stream(stream)))


def read_probe(src, pattern: int, row_bytes: int, rows_per_wg: int, sink, stream=None,
               nbytes: int = None):
    """coli_read_probe: stream `nbytes` (default all) of the uint8 tensor `src`
    in a read-only pattern (0: contiguous chunks of row_bytes per workgroup;
    1: rows of row_bytes, rows_per_wg per workgroup), one word per wave to sink."""
    n = src.numel() if nbytes is None else nbytes
    _check(lib().coli_read_probe(_ptr(src), n, pattern, row_bytes, rows_per_wg, _ptr(sink),
                                 sink.numel() * sink.element_size(), _stream(stream)))


# ---------------------------------------------------------------- MXFP4 experts and token permutation
def _dtype_code(dtype) -> int:
    import torch
    if dtype == torch.bfloat16:
        return BF16
    if dtype == torch.float32:
        return F32
    if dtype == torch.float16:
        return F16
    raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")


def _rows(t, name, rows=None, cols=None, dtype=None):
    """(type code, row stride) of a 2-d device tensor whose columns follow each
    other; `rows` is a least number of rows, `cols` and `dtype` must be met."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-d")
    n, m = t.shape
    ld, step = t.stride()
    if step != 1 and m > 1:
        raise ValueError(f"{name} must have contiguous columns")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if (rows is not None and n < rows) or (cols is not None and m != cols):
        raise ValueError(f"{name} has shape {(n, m)}, expected ({rows}, {cols})")
    if ld < m:
        if n > 1:
            raise ValueError(f"{name} has rows that overlap")
        ld = m
    return _dtype_code(t.dtype), ld


def _mx(q, s, name):
    """(rows, cols) of an MXFP4 pair: codes uint8 [rows][cols/2], scales uint8 [rows][cols/32]."""
    import torch
    _need(q, torch.uint8, f"{name} codes")
    _need(s, torch.uint8, f"{name} scales")
    if q.dim() == 2 and s.dim() == 2:
        rows, half = q.shape
        if s.shape == (rows, half // 16) and half % 16 == 0:
            return rows, 2 * half
    raise ValueError(f"{name}: codes {tuple(q.shape)} and scales {tuple(s.shape)} do not match")


def _new(like, shape, dtype, stream, zero=False):
    """A new tensor on like's device that belongs to the stream the call runs on, so that its
    memory is neither still in use on another stream nor reused there while the call runs."""
    make = like.new_zeros if zero else like.new_empty
    if stream is None:
        return make(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype)


def _mx_out(q, s, rows, cols, like, name, stream):
    import torch
    if cols % 32:
        raise ValueError(f"{name}: the columns of MXFP4 rows must be a multiple of 32, got {cols}")
    fresh = q is None and s is None
    if q is None:
        q = _new(like, (rows, cols // 2), torch.uint8, stream)
    if s is None:
        s = _new(like, (rows, cols // 32), torch.uint8, stream)
    if fresh:
        return q, s
    if _mx(q, s, name) != (rows, cols):
        raise ValueError(f"{name}: codes must have shape ({rows}, {cols // 2})")
    return q, s


@functools.lru_cache(None)
def _device_call():
    """torch.cuda.current_device, or what it calls where this torch has that: 0.5 us less a call."""
    import torch
    return getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _enqueue(tensors, stream, fn, *args):
    """The library's call `fn`(*args, stream) on the tensors' device, on its current stream unless
    one is given. That one has to wait for the inputs, as for any work of another stream; their
    memory is not reused before it is done. (The raw current stream costs 0.2 us of host time, a
    Stream object 2.)"""
    import torch
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on devices {dev} and {t.get_device()}: one device is needed")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        if stream.device_index != dev:
            raise ValueError(f"tensors on device {dev}, stream on device {stream.device_index}")
        raw = stream.cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    call = getattr(_lib or lib(), fn)
    if dev == _device_call()():
        rc = call(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = call(*args, raw)
    if rc != COLI_OK:
        _check(rc)


def quantize_mxfp4(x, q=None, s=None, stream=None):
    """Rows x [rows][cols] (float32, bfloat16 or float16) -> (codes uint8
    [rows][cols/2], scales uint8 [rows][cols/32])."""
    code, ld = _rows(x, "x")
    rows, cols = x.shape
    q, s = _mx_out(q, s, rows, cols, x, "quantize_mxfp4", stream)
    _enqueue((x, q, s), stream, "coli_quantize_mxfp4", x.data_ptr(), code, rows, cols, ld,
             q.data_ptr(), s.data_ptr())
    return q, s


def dequantize_mxfp4(q, s, dtype=None, out=None, stream=None):
    """The values of MXFP4 rows, in `out`'s type, else `dtype` (default float32)."""
    import torch
    rows, cols = _mx(q, s, "dequantize_mxfp4")
    if out is None:
        out = _new(q, (rows, cols), dtype or torch.float32, stream)
    code, ld = _rows(out, "out", rows, cols, dtype)
    _enqueue((q, s, out), stream, "coli_dequantize_mxfp4", q.data_ptr(), s.data_ptr(), rows, cols,
             out.data_ptr(), code, ld)
    return out


def mxfp4_blob_layout(shape: MoEShape):
    """(offsets of the gate/up codes, down codes, gate/up scales, down scales; blob bytes)."""
    off = (ctypes.c_size_t * 4)()
    nb = ctypes.c_size_t()
    _check(lib().coli_mxfp4_blob_layout(ctypes.byref(shape.c()), off, ctypes.byref(nb)))
    return list(off), nb.value


def quantize_mxfp4_expert(shape: MoEShape, gate, up, down, blob=None, stream=None):
    """One expert's gate/up [inter][hidden] and down [hidden][inter] into an MXFP4 blob."""
    import torch
    H, I = shape.hidden, shape.inter
    nbytes = mxfp4_blob_layout(shape)[1]
    for t, n, want in ((gate, "gate", (I, H)), (up, "up", (I, H)), (down, "down", (H, I))):
        _need(t, gate.dtype, n)
        if tuple(t.shape) != want:
            raise ValueError(f"{n} must have shape {want}")
    if blob is None:
        blob = _new(gate, (nbytes,), torch.uint8, stream)
    _need(blob, torch.uint8, "blob")
    if blob.numel() < nbytes:
        raise ValueError(f"blob must hold {nbytes} bytes")
    _enqueue((gate, up, down, blob), stream, "coli_quantize_mxfp4_expert", ctypes.byref(shape.c()),
             gate.data_ptr(), up.data_ptr(), down.data_ptr(), _dtype_code(gate.dtype), blob.data_ptr())
    return blob


def _groups(table, offsets, rows, K, n, q_off, s_off):
    import torch
    _need(table, torch.int64, "table")
    _need(offsets, torch.int32, "offsets")
    if offsets is not None and offsets.numel() != table.numel() + 1:
        raise ValueError("offsets must hold one more value than the table")
    # what the C types would cut to other values
    E = table.numel()
    if max(rows, K, E) >= 2 ** 31 or not 0 < n < 2 ** 31 or (q_off | s_off) >> 63:
        raise ValueError(f"rows {rows}, columns {K}, matrices {E} and matrix rows {n} must be below 2^31, "
                         f"q_off {q_off} and s_off {s_off} below 2^63 and not negative")
    return E, None if offsets is None else offsets.data_ptr()


def mxfp4_matmul(a, a_s, table, n, q_off=0, s_off=0, offsets=None, dtype=None, out=None, stream=None):
    """out[r] = W_e(r) a[r] for MXFP4 rows (a, a_s) sorted by expert. table: device
    array (int64) of pointers to the experts' buffers, each with an MXFP4
    [n][K] matrix: codes at q_off, scales at s_off. offsets [E + 1] as union
    gives it (None: one matrix for every row). out in `dtype` (default float32); its
    rows outside the offsets are left as they are (undefined in a new one)."""
    import torch
    rows, K = _mx(a, a_s, "a")
    E, off = _groups(table, offsets, rows, K, n, q_off, s_off)
    if out is None:
        out = _new(a, (rows, n), dtype or torch.float32, stream)
    code, ld = _rows(out, "out", rows, n, dtype)
    _enqueue((a, a_s, table, offsets, out), stream, "coli_mxfp4_matmul", a.data_ptr(),
             a_s.data_ptr(), rows, K, off, E, table.data_ptr(), q_off, s_off, n, out.data_ptr(), code, ld)
    return out


def mxfp4_swiglu(a, a_s, table, inter, q_off=0, s_off=0, offsets=None, dtype=None, out=None,
                 stream=None):
    """h[r] = silu(G_e(r) a[r]) * (U_e(r) a[r]), arguments as mxfp4_matmul with the
    interleaved [2 inter][K] gate/up matrix (rows outside the offsets too). dtype
    "mxfp4" (or out a (codes, scales) pair): h as MXFP4 rows, returned as that pair."""
    import torch
    rows, K = _mx(a, a_s, "a")
    E, off = _groups(table, offsets, rows, K, inter, q_off, s_off)
    if dtype == "mxfp4" or isinstance(out, (tuple, list)):
        if dtype not in (None, "mxfp4"):
            raise ValueError(f"out is an MXFP4 pair, dtype {dtype}")
        q, s = _mx_out(*(out or (None, None)), rows, inter, a, "mxfp4_swiglu", stream)
        out, h, hs, code, ld = (q, s), q, s.data_ptr(), MXFP4, inter
    else:
        if out is None:
            out = _new(a, (rows, inter), dtype or torch.float32, stream)
        code, ld = _rows(out, "out", rows, inter, dtype)
        h, hs, s = out, None, None
    _enqueue((a, a_s, table, offsets, h, s), stream, "coli_mxfp4_swiglu", a.data_ptr(),
             a_s.data_ptr(), rows, K, off, E, table.data_ptr(), q_off, s_off, inter, h.data_ptr(), hs,
             code, ld)
    return out


MXFP4_KERNELS = ("few_rows_2", "few_rows_4", "tiles_short", "tiles_64", "tiles_128", "lines_128", "lines_256")


def debug_mxfp4_kernel(rows: int, K: int, E: int, N: int, grouped=True, aligned=True) -> str:
    """coli_debug_mxfp4_kernel: the kernel that a product of these sizes runs."""
    out = ctypes.c_int32()
    _check(lib().coli_debug_mxfp4_kernel(rows, K, E, N, int(grouped), int(aligned), ctypes.byref(out)))
    return MXFP4_KERNELS[out.value]


@functools.lru_cache(4096)
def _union_ws(T, k, E):
    nb = ctypes.c_size_t()
    _check(lib().coli_moe_union_workspace_size(T, k, E, ctypes.byref(nb)))
    return nb.value


def union_inverse(idx, E, stream=None):
    """union, with each assignment's place in the experts' order: (counts, offsets,
    perm, unique, n_unique, inv [T][k])."""
    import torch
    _need(idx, torch.int32, "idx")
    T, k = idx.shape
    n = T * k
    if n >= 2 ** 31 or E >= 2 ** 31:
        raise ValueError(f"idx must have fewer than 2^31 values, and E, {E}, be below 2^31")
    nb = _union_ws(T, k, E)
    buf = _new(idx, (3 * E + 2 + 2 * n + (nb + 3) // 4,), torch.int32, stream)
    counts, offsets, perm, unique, n_unique, inv, ws = buf.split_with_sizes(
        (E, E + 1, n, E, 1, n, (nb + 3) // 4))
    base = buf.data_ptr()
    at = [base + 4 * i for i in (0, E, 2 * E + 1, 2 * E + 1 + n, 3 * E + 1 + n, 3 * E + 2 + n,
                                 3 * E + 2 + 2 * n)]
    _enqueue((idx, buf), stream, "coli_moe_union_inverse", idx.data_ptr(), T, k, E, *at[:6], at[6],
             nb)
    return counts, offsets, perm, unique, n_unique, inv.view(T, k)


def _slots(inv, w=None):
    import torch
    _need(inv, torch.int32, "inv")
    _need(w, torch.float32, "w")
    if inv.dim() != 2 or (w is not None and w.shape != inv.shape):
        raise ValueError("inv must be [T][k], and w of the same shape")
    if inv.numel() >= 2 ** 31:
        raise ValueError("inv must have fewer than 2^31 values")
    return inv.shape


def dispatch(x, inv, out=None, stream=None):
    """out[inv[t, j]] = x[t]: the tokens' rows in the experts' order (rows of no
    slot are left as they are, undefined in a new out)."""
    T, k = _slots(inv)
    code, ld = _rows(x, "x", T)
    H = x.shape[1]
    if out is None:
        out = _new(x, (T * k, H), x.dtype, stream)
    ld_out = _rows(out, "out", T * k, H, x.dtype)[1]
    _enqueue((x, inv, out), stream, "coli_moe_dispatch", x.data_ptr(), code, T, k, H, ld,
             inv.data_ptr(), out.data_ptr(), ld_out)
    return out


def dispatch_mxfp4(x, inv, q=None, s=None, stream=None):
    """dispatch with the rows quantised on the way: (codes, scales) of T*k MXFP4 rows (those
    of no slot as there)."""
    T, k = _slots(inv)
    code, ld = _rows(x, "x", T)
    H = x.shape[1]
    q, s = _mx_out(q, s, T * k, H, x, "dispatch_mxfp4", stream)
    _enqueue((x, inv, q, s), stream, "coli_moe_dispatch_mxfp4", x.data_ptr(), code, T, k, H, ld,
             inv.data_ptr(), q.data_ptr(), s.data_ptr())
    return q, s


def dispatch_fp8(x, inv, q=None, s=None, stream=None):
    """dispatch with the rows quantised on the way: (codes, scales) of T*k FP8 rows (those of no
    slot as there)."""
    T, k = _slots(inv)
    code, ld = _rows(x, "x", T)
    H = x.shape[1]
    q, s = _fp8_out(q, s, T * k, H, x, "dispatch_fp8", stream)
    _enqueue((x, inv, q, s), stream, "coli_moe_dispatch_fp8", x.data_ptr(), code, T, k, H, ld,
             inv.data_ptr(), q.data_ptr(), s.data_ptr())
    return q, s


def dispatch_bwd(grad, inv, dtype=None, out=None, stream=None):
    """dispatch's gradient: out[t] = sum_j grad[inv[t, j]], in `dtype` (default grad's)."""
    T, k = _slots(inv)
    g_code, ld_g = _rows(grad, "grad", T * k)
    H = grad.shape[1]
    if out is None:
        out = _new(grad, (T, H), dtype or grad.dtype, stream)
    code, ld = _rows(out, "out", T, H, dtype)
    _enqueue((grad, inv, out), stream, "coli_moe_dispatch_bwd", grad.data_ptr(), g_code, ld_g, T, k,
             H, inv.data_ptr(), out.data_ptr(), code, ld)
    return out


def combine(rows, inv, w, shared=None, scale=1.0, dtype=None, out=None, stream=None):
    """out[t] = shared[t] + scale * sum_j w[t, j] * rows[inv[t, j]], in `dtype`
    (default: shared's type, else the rows'). out may be shared."""
    T, k = _slots(inv, w)
    r_code, ld_r = _rows(rows, "rows", T * k)
    H = rows.shape[1]
    if out is None:
        out = _new(rows, (T, H), dtype or (rows if shared is None else shared).dtype, stream)
    code, ld = _rows(out, "out", T, H, dtype)
    ld_s = ld if shared is None else _rows(shared, "shared", T, H, out.dtype)[1]
    _enqueue((rows, inv, w, shared, out), stream, "coli_moe_combine", rows.data_ptr(), r_code, ld_r,
             T, k, H, inv.data_ptr(), w.data_ptr(), None if shared is None else shared.data_ptr(), ld_s,
             scale, out.data_ptr(), code, ld)
    return out


def combine_bwd(grad, rows, inv, w, scale=1.0, rows_grad=None, w_grad=None, stream=None):
    """combine's gradients for the output gradient `grad` (which is shared's own
    gradient): (rows_grad in the rows' type and order, w_grad [T][k])."""
    T, k = _slots(inv, w)
    r_code, ld_r = _rows(rows, "rows", T * k)
    H = rows.shape[1]
    g_code, ld_g = _rows(grad, "grad", T, H)
    if rows_grad is None:
        rows_grad = _new(rows, rows.shape, rows.dtype, stream, zero=True)
    if w_grad is None:
        w_grad = _new(w, w.shape, w.dtype, stream)
    _slots(inv, w_grad)
    ld_rg = _rows(rows_grad, "rows_grad", T * k, H, rows.dtype)[1]
    _enqueue((grad, rows, inv, w, rows_grad, w_grad), stream, "coli_moe_combine_bwd",
             grad.data_ptr(), g_code, ld_g, rows.data_ptr(), r_code, ld_r, T, k, H, inv.data_ptr(),
             w.data_ptr(), scale, rows_grad.data_ptr(), ld_rg, w_grad.data_ptr())
    return rows_grad, w_grad


# ---------------------------------------------------------------- routing with groups
SCORES = {"sigmoid": 0, "softmax": 1}


def _score(score) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return SCORES[score]


def _token_rows(t, name, dtype=None, shape=None):
    """Type code of a contiguous 2-d device tensor."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be 2-d and contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if max(t.shape) >= 2 ** 31:
        raise ValueError(f"{name} must have fewer than 2^31 rows and columns")
    return None if dtype is not None else _dtype_code(t.dtype)


def _small(*numbers):
    """Refuses what a C int would cut to another value."""
    for n in numbers:
        if n >> 31 not in (0, -1):
            raise ValueError(f"{n} is no number of 32 bits")


def route_groups(logits, bias, k, score="sigmoid", groups=1, groups_kept=None, group_top=2, norm=True,
                 scale=1.0, with_scores=False, idx=None, w=None, scores=None, stream=None):
    """The k experts of every token and their weights, (idx int32 [T][k], w float32 [T][k]), for logits
    [T][E] (float32, bfloat16 or float16) and a selection bias float32 [E] (or None): sigmoid or softmax
    scores; the `groups_kept` (default all) best of `groups` groups by their largest key or the sum of
    their `group_top` = 2 largest; weights `scale` times the scores, which `norm` divides by their sum.
    Slots for which no expert is left have idx -1. with_scores (or scores given): also the scores,
    float32 [T][E]."""
    import torch
    if groups_kept is None:
        groups_kept = groups
    if (k | groups | groups_kept | group_top) >> 31:
        _small(k, groups, groups_kept, group_top)
    code = _token_rows(logits, "logits")
    T, E = logits.shape
    if bias is not None:
        _need(bias, torch.float32, "bias")
        if bias.numel() != E:
            raise ValueError(f"bias must have {E} values")
    if idx is None:
        idx = _new(logits, (T, k), torch.int32, stream)
    else:
        _token_rows(idx, "idx", torch.int32, (T, k))
    if w is None:
        w = _new(logits, (T, k), torch.float32, stream)
    else:
        _token_rows(w, "w", torch.float32, (T, k))
    if scores is not None:
        _token_rows(scores, "scores", torch.float32, (T, E))
    elif with_scores:
        scores = _new(logits, (T, E), torch.float32, stream)
    _enqueue((logits, bias, idx, w, scores), stream, "coli_moe_route_groups", logits.data_ptr(), code,
             None if bias is None else bias.data_ptr(), T, E, k, _score(score), groups, groups_kept, group_top,
             1 if norm else 0, scale, idx.data_ptr(), w.data_ptr(), None if scores is None else scores.data_ptr())
    return (idx, w) if scores is None else (idx, w, scores)


def route_groups_bwd(w_grad, logits, idx, score="sigmoid", norm=True, scale=1.0, scores_grad=None,
                     dtype=None, out=None, stream=None):
    """route_groups' gradient to the logits, [T][E] in `dtype` (default the logits'), from that of its
    weights and (optionally) that of its scores; score, norm and scale as there."""
    import torch
    code = _token_rows(logits, "logits")
    T, E = logits.shape
    _token_rows(idx, "idx", torch.int32)
    k = idx.shape[1]
    _token_rows(idx, "idx", torch.int32, (T, k))
    _token_rows(w_grad, "w_grad", torch.float32, (T, k))
    if scores_grad is not None:
        _token_rows(scores_grad, "scores_grad", torch.float32, (T, E))
    if out is None:
        out = _new(logits, (T, E), dtype or logits.dtype, stream)
    elif dtype is not None and out.dtype != dtype:
        raise ValueError(f"out must be {dtype}, got {out.dtype}")
    if tuple(out.shape) != (T, E):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(T, E)}")
    out_code = _token_rows(out, "out")
    _enqueue((w_grad, logits, idx, scores_grad, out), stream, "coli_moe_route_groups_bwd", w_grad.data_ptr(),
             logits.data_ptr(), code, idx.data_ptr(), T, E, k, _score(score), 1 if norm else 0, scale,
             None if scores_grad is None else scores_grad.data_ptr(), out.data_ptr(), out_code)
    return out


# ---------------------------------------------------------------- FP8 experts
FP8_KERNELS = ("few_rows_16", "few_rows_32", "lines_128", "lines_256")


def _blocks(n):
    return -(-n // 128)


def _fp8_rows(q, s, name):
    """(rows, cols) of FP8 rows: codes uint8 [rows][cols], scales float32 [rows][ceil(cols / 128)]."""
    import torch
    _need(q, torch.uint8, f"{name} codes")
    _need(s, torch.float32, f"{name} scales")
    shape = q.shape
    if len(shape) != 2 or s.shape != (shape[0], _blocks(shape[1])):
        raise ValueError(f"{name}: codes {tuple(shape)} and scales {tuple(s.shape)} do not match")
    return shape[0], shape[1]


def _fp8_out(q, s, rows, cols, like, name, stream):
    import torch
    fresh = q is None and s is None
    if q is None:
        q = _new(like, (rows, cols), torch.uint8, stream)
    if s is None:
        s = _new(like, (rows, _blocks(cols)), torch.float32, stream)
    if not fresh and _fp8_rows(q, s, name) != (rows, cols):
        raise ValueError(f"{name}: codes must have shape ({rows}, {cols})")
    return q, s


def quantize_fp8(x, q=None, s=None, stream=None):
    """Rows x [rows][cols] (float32, bfloat16 or float16) -> (codes uint8 [rows][cols], scales float32
    [rows][ceil(cols / 128)])."""
    code, ld = _rows(x, "x")
    rows, cols = x.shape
    q, s = _fp8_out(q, s, rows, cols, x, "quantize_fp8", stream)
    _enqueue((x, q, s), stream, "coli_quantize_fp8", x.data_ptr(), code, rows, cols, ld, q.data_ptr(),
             s.data_ptr())
    return q, s


def _fp8_matrices(q, s, lead, rows, cols, like, name, stream):
    """Outputs [..lead][rows][cols] and [..lead][blocks][blocks], each matrix without gaps; their strides in bytes."""
    import torch
    blocks = _blocks(rows), _blocks(cols)
    made = []
    for t, shape, dtype, part in ((q, (rows, cols), torch.uint8, "codes"), (s, blocks, torch.float32, "scales")):
        if t is None:
            made += _new(like, (*lead, *shape), dtype, stream), shape[0] * shape[1]
            continue
        if t.dtype != dtype or not t.is_cuda or t.shape != (*lead, *shape):
            raise ValueError(f"{name}: {part} must be a {dtype} device tensor of shape {(*lead, *shape)}")
        if not t.is_contiguous() and not (lead and t[0].is_contiguous()):
            raise ValueError(f"{name}: each matrix of the {part} must be contiguous")
        made += t, t.stride(0) if lead else shape[0] * shape[1]
    return made[0], made[2], made[1], 4 * made[3]


def quantize_fp8_matrix(x, transposed=False, q=None, s=None, qt=None, st=None, stream=None):
    """Matrices x [rows][cols] or [count][rows][cols] (float32, bfloat16 or float16) by blocks of 128 x 128
    -> (codes uint8 of x's shape, scales float32 [..][ceil(rows / 128)][ceil(cols / 128)]), with
    `transposed` (or qt, st given) followed by those of the transposed matrices. Given outputs may be
    views into experts' buffers: only a matrix itself has to be contiguous."""
    shape = x.shape
    if len(shape) not in (2, 3):
        raise ValueError("x must be [rows][cols] or [count][rows][cols]")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    lead, (rows, cols) = shape[:-2], shape[-2:]
    count, x_stride = (lead[0], x.stride(0)) if lead else (1, 0)
    code, ld = (_dtype_code(x.dtype), cols) if x.numel() == 0 else _rows(x[0] if lead else x, "x")
    if count >= 2 ** 31:
        raise ValueError("fewer than 2^31 matrices are needed")
    if count > 1 and x.numel() and x_stride < (rows - 1) * ld + cols:
        raise ValueError("x has matrices that overlap")
    name = "quantize_fp8_matrix"
    q, s, q_stride, s_stride = _fp8_matrices(q, s, lead, rows, cols, x, name, stream)
    if not transposed and qt is None and st is None:
        _enqueue((x, q, s), stream, "coli_quantize_fp8_matrix", x.data_ptr(), code, count, rows, cols, ld, x_stride,
                 q.data_ptr(), q_stride, s.data_ptr(), s_stride, None, 0, None, 0)
        return q, s
    qt, st, qt_stride, st_stride = _fp8_matrices(qt, st, lead, cols, rows, x, name, stream)
    _enqueue((x, q, s, qt, st), stream, "coli_quantize_fp8_matrix", x.data_ptr(), code, count, rows, cols, ld, x_stride,
             q.data_ptr(), q_stride, s.data_ptr(), s_stride, qt.data_ptr(), qt_stride, st.data_ptr(), st_stride)
    return q, s, qt, st


@functools.lru_cache(4096)
def fp8_column_blocks(rows: int, E: int) -> int:
    """The blocks of 128 rows of an expert that quantize_fp8_columns may need."""
    _small(rows, E)
    out = ctypes.c_int64()
    _check(lib().coli_fp8_column_blocks(rows, E, ctypes.byref(out)))
    return out.value


def quantize_fp8_columns(x, offsets=None, rows=False, qt=None, st=None, q=None, s=None, stream=None):
    """Rows x [rows][cols] sorted by expert -> (codes uint8 [blocks][cols][128], scale exponents uint8
    [blocks][cols]) over 128 of an expert's rows by one column, for fp8_wgrad; as many blocks as
    fp8_column_blocks says (or a given qt has). `rows` (or q, s given): also quantize_fp8's codes and
    scales, from the same pass."""
    import torch
    code, ld = _rows(x, "x")
    n, cols = x.shape
    _need(offsets, torch.int32, "offsets")
    E = 1 if offsets is None else offsets.numel() - 1
    if max(n, cols, E) >= 2 ** 31 or E < 1:
        raise ValueError(f"rows {n}, columns {cols} and experts {E} must be below 2^31, experts at least 1")
    blocks = fp8_column_blocks(n, E) if qt is None else qt.shape[0]
    fresh = qt is None and st is None
    if qt is None:
        qt = _new(x, (blocks, cols, 128), torch.uint8, stream)
    if st is None:
        st = _new(x, (blocks, cols), torch.uint8, stream)
    if not fresh:
        _fp8_columns(qt, st, "quantize_fp8_columns", cols)
    if rows or q is not None or s is not None:
        q, s = _fp8_out(q, s, n, cols, x, "quantize_fp8_columns", stream)
    _enqueue((x, offsets, qt, st, q, s), stream, "coli_quantize_fp8_columns", x.data_ptr(), code, n, cols, ld,
             None if offsets is None else offsets.data_ptr(), E, qt.data_ptr(), blocks, st.data_ptr(),
             None if q is None else q.data_ptr(), None if s is None else s.data_ptr())
    return (qt, st) if q is None else (qt, st, q, s)


def _rows_of_blocks(blocks, E):
    """The most rows over E experts that fit the blocks."""
    many = 128 * blocks + 127 - 127 * E
    return many if many >= E else min(blocks, E)


def _fp8_columns(qt, st, name, cols=None):
    """(blocks, cols) of columns: codes uint8 [blocks][cols][128], scale exponents uint8 [blocks][cols]."""
    import torch
    _need(qt, torch.uint8, f"{name} codes")
    _need(st, torch.uint8, f"{name} scales")
    shape = qt.shape
    if len(shape) != 3 or shape[2] != 128 or st.shape != shape[:2] or cols not in (None, shape[1]):
        raise ValueError(f"{name}: codes {tuple(shape)} and scales {tuple(st.shape)} do not match")
    return shape[0], shape[1]


def dequantize_fp8(q, s, dtype=None, out=None, stream=None):
    """The values of FP8 rows, or of matrices ([..][rows][cols] with a scale for each 128 x 128 block), in
    `out`'s type, else `dtype` (default float32)."""
    import torch
    shape, many = q.shape, q.dim() == 3
    if len(shape) not in (2, 3) or s.dim() != len(shape):
        raise ValueError("codes must be [rows][cols] or [count][rows][cols], and scales have as many dimensions")
    for t, kind, name in ((q, torch.uint8, "codes"), (s, torch.float32, "scales")):
        _need(t[0] if many and len(t) and not t.is_contiguous() else t, kind, name)
    lead, (rows, cols) = shape[:-2], shape[-2:]
    per_row = s.shape == (*lead, rows, _blocks(cols))
    if not per_row and s.shape != (*lead, _blocks(rows), _blocks(cols)):
        raise ValueError(f"codes {tuple(shape)} and scales {tuple(s.shape)} do not match")
    fresh = out is None
    if fresh:
        out = _new(q, shape, dtype or torch.float32, stream)
    elif out.shape != shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    if not many:
        parts = [(q, s, out)]
    elif per_row and q.is_contiguous() and s.is_contiguous() and out.is_contiguous():       # the rows of one long matrix
        parts = [(q.view(-1, cols), s.view(-1, s.shape[-1]), out.view(-1, cols))]
    elif not per_row and 0 < len(q) < 2 ** 31 and (fresh or len(q) == 1 or out.stride(0) >= (rows - 1) * out.stride(1) + cols) and (
            len(q) == 1 or q.stride(0) % 16 == 0):
        code, ld = (_dtype_code(out.dtype), cols) if fresh else _rows(out[0], "out", rows, cols, dtype)
        _enqueue((q, s, out), stream, "coli_dequantize_fp8_matrix", q.data_ptr(), q.stride(0), s.data_ptr(),
                 4 * s.stride(0), len(q), rows, cols, out.data_ptr(), code, ld, out.stride(0))
        return out
    else:
        parts = zip(q, s, out)
    for pq, ps, po in parts:
        code, ld = _rows(po, "out", pq.shape[0], cols, dtype)
        _enqueue((pq, ps, po), stream, "coli_dequantize_fp8", pq.data_ptr(), ps.data_ptr(), pq.shape[0], cols,
                 1 if per_row else 128, po.data_ptr(), code, ld)
    return out


def fp8_blob_layout(shape: MoEShape):
    """(offsets of the gate, up and down codes, then of their scales; blob bytes)."""
    off = (ctypes.c_size_t * 6)()
    nb = ctypes.c_size_t()
    _check(lib().coli_fp8_blob_layout(ctypes.byref(shape.c()), off, ctypes.byref(nb)))
    return list(off), nb.value


@functools.lru_cache(4096)
def _fp8_matmul_ws(rows, K, E, n, grouped, code):
    nb = ctypes.c_size_t()
    _check(lib().coli_fp8_matmul_workspace_size(rows, K, E, n, int(grouped), code, ctypes.byref(nb)))
    return nb.value


def fp8_matmul(a, a_s, table, n, q_off=0, s_off=0, offsets=None, dtype=None, out=None, stream=None):
    """out[r] = W_e(r) a[r] for FP8 rows (a, a_s) sorted by expert. table: device array (int64) of pointers
    to the experts' buffers, each with an FP8 [n][K] matrix: codes at q_off, scales at s_off. offsets [E + 1]
    as union gives it (None: one matrix for every row). out in `dtype` (default float32); its rows outside
    the offsets are left as they are (undefined in a new one). With the transposed matrices of
    quantize_fp8_matrix it is the product's gradient to its rows."""
    import torch
    rows, K = _fp8_rows(a, a_s, "a")
    E, off = _groups(table, offsets, rows, K, n, q_off, s_off)
    if out is None:
        out = _new(a, (rows, n), dtype or torch.float32, stream)
    code, ld = _rows(out, "out", rows, n, dtype)
    nb = _fp8_matmul_ws(rows, K, E, n, off is not None, code)
    ws = _new(a, (nb,), torch.uint8, stream) if nb else None
    _enqueue((a, a_s, table, offsets, out, ws), stream, "coli_fp8_matmul", a.data_ptr(), a_s.data_ptr(), rows, K,
             off, E, table.data_ptr(), q_off, s_off, n, out.data_ptr(), code, ld, None if ws is None else ws.data_ptr(), nb)
    return out


@functools.lru_cache(4096)
def _fp8_swiglu_ws(rows, K, E, inter, grouped, code):
    nb = ctypes.c_size_t()
    _check(lib().coli_fp8_swiglu_workspace_size(rows, K, E, inter, int(grouped), code, ctypes.byref(nb)))
    return nb.value


def fp8_swiglu(a, a_s, table, inter, q_off=0, s_off=0, up_q_off=None, up_s_off=None, offsets=None, dtype=None,
               out=None, stream=None):
    """h[r] = silu(G_e(r) a[r]) * (U_e(r) a[r]), arguments as fp8_matmul: the gate matrix [inter][K] at q_off
    and s_off, the up matrix at up_q_off and up_s_off (default: right behind gate's codes and scales).
    dtype "fp8" (or out a (codes, scales) pair): h as FP8 rows, returned as that pair."""
    import torch
    rows, K = _fp8_rows(a, a_s, "a")
    E, off = _groups(table, offsets, rows, K, inter, q_off, s_off)
    if up_q_off is None:
        up_q_off = q_off + inter * K
    if up_s_off is None:
        up_s_off = s_off + 4 * _blocks(inter) * _blocks(K)
    if (up_q_off | up_s_off) >> 63:
        raise ValueError(f"up_q_off {up_q_off} and up_s_off {up_s_off} must be below 2^63 and not negative")
    if dtype == "fp8" or isinstance(out, (tuple, list)):
        if dtype not in (None, "fp8"):
            raise ValueError(f"out is an FP8 pair, dtype {dtype}")
        q, s = _fp8_out(*(out or (None, None)), rows, inter, a, "fp8_swiglu", stream)
        out, h, hs, code, ld = (q, s), q, s.data_ptr(), FP8, inter
    else:
        if out is None:
            out = _new(a, (rows, inter), dtype or torch.float32, stream)
        code, ld = _rows(out, "out", rows, inter, dtype)
        h, hs, s = out, None, None
    nb = _fp8_swiglu_ws(rows, K, E, inter, off is not None, code)
    ws = _new(a, (nb,), torch.uint8, stream) if nb else None
    _enqueue((a, a_s, table, offsets, h, s, ws), stream, "coli_fp8_swiglu", a.data_ptr(), a_s.data_ptr(), rows, K,
             off, E, table.data_ptr(), q_off, s_off, up_q_off, up_s_off, inter, h.data_ptr(), hs, code, ld,
             None if ws is None else ws.data_ptr(), nb)
    return out


@functools.lru_cache(4096)
def _fp8_wgrad_ws(rows, E, n, K):
    nb = ctypes.c_size_t()
    _check(lib().coli_fp8_wgrad_workspace_size(rows, E, n, K, ctypes.byref(nb)))
    return nb.value


def fp8_wgrad(gt, gt_s, xt, xt_s, offsets=None, rows=None, dtype=None, out=None, accumulate=False, stream=None):
    """fp8_matmul's gradient to its matrices, out[e] = sum over the expert's rows of grad[r] x[r]^T, [E][n][K]
    in `dtype` (default float32), from quantize_fp8_columns of the output's gradient and of the rows, with
    the same offsets. rows (needed only without offsets, where there are more blocks than it takes): how
    many rows those had. accumulate: added to what `out` holds."""
    import torch
    blocks, n = _fp8_columns(gt, gt_s, "gt")
    x_blocks, K = _fp8_columns(xt, xt_s, "xt")
    if blocks != x_blocks:
        raise ValueError(f"gt has {blocks} blocks, xt {x_blocks}")
    _need(offsets, torch.int32, "offsets")
    E = 1 if offsets is None else offsets.numel() - 1
    if E < 1:
        raise ValueError("offsets must hold at least two values")
    if rows is None:
        rows = _rows_of_blocks(blocks, E)
    if max(n, K, rows, E) >= 2 ** 31 or rows < 0:
        raise ValueError("rows, columns and experts must be below 2^31")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = _new(gt, (E, n, K), dtype or torch.float32, stream)
        code, ld = _dtype_code(out.dtype), K
    else:
        if out.shape != (E, n, K) or not out.is_cuda:
            raise ValueError(f"out must be a device tensor of shape {(E, n, K)}")
        if E > 1 and n and out.stride(0) != n * out.stride(1):
            raise ValueError("out's matrices must follow each other without gaps")
        code, ld = _rows(out.view(E * n, K) if out.is_contiguous() else out[0], "out", n, K, dtype)
    nb = _fp8_wgrad_ws(rows, E, n, K)
    ws = _new(gt, (nb,), torch.uint8, stream) if nb else None
    _enqueue((gt, gt_s, xt, xt_s, offsets, out, ws), stream, "coli_fp8_wgrad", gt.data_ptr(), gt_s.data_ptr(),
             xt.data_ptr(), xt_s.data_ptr(), blocks, rows, None if offsets is None else offsets.data_ptr(), E, n, K,
             1 if accumulate else 0, out.data_ptr(), code, ld, None if ws is None else ws.data_ptr(), nb)
    return out


def debug_fp8_kernel(rows: int, K: int, E: int, N: int, grouped=True, swiglu=False, wide=False) -> str:
    """coli_debug_fp8_kernel: the kernel that a product of these sizes runs without a workspace (wide: exact products,
    of float32 results and of FP8 rows below 2^20 values)."""
    _small(rows, K, E, N)
    out = ctypes.c_int32()
    _check(lib().coli_debug_fp8_kernel(rows, K, E, N, bool(grouped), bool(swiglu), bool(wide), ctypes.byref(out)))
    return FP8_KERNELS[out.value]


class ExpertCache:
    """Per-layer LRU of expert blobs in an HBM arena in front of pinned host
    memory (coli_expert_cache_*). With arena and pool both None the cache only
    keeps the books (policy simulation, no GPU needed)."""

    def __init__(self, n_layers, n_experts, slots_per_layer, blob_bytes, arena=None, pools=None,
                 copy_stream=None):
        """pools: one pinned host tensor (n_experts * blob_bytes bytes) per layer, or
        one tensor holding all layers back to back."""
        ptrs = None
        if pools is not None:
            if not isinstance(pools, (list, tuple)):
                base = pools.data_ptr()
                layer_bytes = n_experts * blob_bytes
                pools_list = [base + l * layer_bytes for l in range(n_layers)]
            else:
                pools_list = [p if isinstance(p, int) else p.data_ptr() for p in pools]
            ptrs = (ctypes.c_void_p * n_layers)(*pools_list)
        self.cfg = CacheCfg(n_layers, n_experts, slots_per_layer, blob_bytes,
                            None if arena is None else arena.data_ptr(),
                            None if ptrs is None else ctypes.cast(ptrs, ctypes.c_void_p).value,
                            None if copy_stream is None else copy_stream.cuda_stream)
        self._keep = (arena, pools, copy_stream, ptrs)
        h = ctypes.c_void_p()
        _check(lib().coli_expert_cache_create(ctypes.byref(self.cfg), ctypes.byref(h)))
        self.handle = h.value
        self.n_experts = n_experts

    def close(self):
        if self.handle:
            lib().coli_expert_cache_destroy(ctypes.c_void_p(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def ensure(self, layer, ids):
        import numpy as np
        ids = np.ascontiguousarray(np.asarray(ids, dtype=np.int32))
        miss = np.zeros(len(ids), dtype=np.int32)
        _check(lib().coli_expert_cache_ensure(ctypes.c_void_p(self.handle), layer,
                                              ids.ctypes.data_as(ctypes.c_void_p), len(ids),
                                              miss.ctypes.data_as(ctypes.c_void_p)))
        return miss

    def _stream_arg(self, stream):
        # a bookkeeping-only cache records no events: no stream needed
        return None if self._keep[0] is None else _stream(stream)

    def wait(self, layer, stream=None):
        _check(lib().coli_expert_cache_wait(ctypes.c_void_p(self.handle), layer,
                                            self._stream_arg(stream)))

    def release(self, layer, stream=None):
        _check(lib().coli_expert_cache_release(ctypes.c_void_p(self.handle), layer,
                                               self._stream_arg(stream)))

    def pin(self, layer, ids):
        import numpy as np
        ids = np.ascontiguousarray(np.asarray(ids, dtype=np.int32))
        _check(lib().coli_expert_cache_pin(ctypes.c_void_p(self.handle), layer,
                                           ids.ctypes.data_as(ctypes.c_void_p), len(ids)))

    def usage(self):
        """Usage history, uint64 [n_layers][n_experts]."""
        import numpy as np
        out = np.zeros((self.cfg.n_layers, self.n_experts), dtype=np.uint64)
        _check(lib().coli_expert_cache_usage(ctypes.c_void_p(self.handle),
                                             out.ctypes.data_as(ctypes.c_void_p)))
        return out

    def pin_hot(self, per_layer, counts=None):
        import numpy as np
        c = None
        if counts is not None:
            c = np.ascontiguousarray(np.asarray(counts, dtype=np.uint64))
            assert c.shape == (self.cfg.n_layers, self.n_experts)
        _check(lib().coli_expert_cache_pin_hot(
            ctypes.c_void_p(self.handle), None if c is None else c.ctypes.data_as(ctypes.c_void_p),
            per_layer))

    def repin(self, max_swaps=4, hysteresis=0.25, decay=0.5) -> int:
        n = ctypes.c_int32()
        _check(lib().coli_expert_cache_repin(ctypes.c_void_p(self.handle), max_swaps, hysteresis,
                                             decay, ctypes.byref(n)))
        return n.value

    def prefetch(self, layer, ids) -> int:
        import numpy as np
        ids = np.ascontiguousarray(np.asarray(ids, dtype=np.int32))
        n = ctypes.c_int32()
        _check(lib().coli_expert_cache_prefetch(ctypes.c_void_p(self.handle), layer,
                                                ids.ctypes.data_as(ctypes.c_void_p), len(ids),
                                                ctypes.byref(n)))
        return n.value

    def table_ptr(self, layer) -> int:
        p = ctypes.c_void_p()
        _check(lib().coli_expert_cache_table(ctypes.c_void_p(self.handle), layer, ctypes.byref(p)))
        return p.value

    def stats(self) -> dict:
        s = CacheStats()
        _check(lib().coli_expert_cache_stats(ctypes.c_void_p(self.handle), ctypes.byref(s)))
        return {f: getattr(s, f) for f, _ in CacheStats._fields_}

    def reset(self):
        _check(lib().coli_expert_cache_reset(ctypes.c_void_p(self.handle)))
