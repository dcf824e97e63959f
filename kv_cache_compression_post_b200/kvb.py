"""Python binding of libkvb, the sm_100a KV-bank library (argument marshalling only).

Every function here has the name of the C entry point it calls (include/kvb.h)
and only converts arguments: torch tensors become device pointers, a torch
stream (or None = torch's current stream) becomes a cudaStream_t, a non-OK status
becomes a ``KvbError``.  All computation happens in the library's CUDA kernels;
importing this package fails if the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "KvbError", "kvb_config", "kvb_admit_stats", "make_config", "lib", "LIB_PATH", "Bank", "PAGES_PRESET",
    "KVB_BF16", "KVB_F32", "KVB_DENSITYKV", "KVB_FORCINGKV",
    "KVB_ORDER_DISTURBANCE", "KVB_ORDER_SOURCE", "KVB_BASELINES_FIXED", "KVB_BASELINES_REFRESH",
    "KVB_EVICT_THRESHOLD_RATIO", "KVB_EVICT_DENSEST", "KVB_EVICT_THRESHOLD_SOURCE",
    "KVB_BOTTOMK_FRAME", "KVB_BOTTOMK_CALL", "KVB_SIM_PER_LAYER", "KVB_SIM_FIRST_LAYER",
    "KVB_STORE_NATIVE", "KVB_STORE_FP8_E4M3",
    "kvb_workspace_size", "kvb_bank_create", "kvb_bank_destroy", "kvb_admit", "kvb_prune_hybrid",
    "kvb_attend", "kvb_read_stats", "kvb_bank_export", "kvb_bank_import", "kvb_device_status",
    "kvb_status_string", "kvb_launch_count", "kvb_trace_enable", "kvb_trace_read", "kvb_density_workspace_size", "kvb_density", "kvb_density_noalloc", "kvb_segment_cosine",
    "kvb_selftest_timeout", "kvb_admit_begin", "kvb_admit_finish",
    "KVB_ROPE_INTERLEAVED", "KVB_ROPE_HALVES", "kvb_rope", "rope",
    "kvb_q8_cache", "kvb_q8_workspace_size", "kvb_q8_append", "kvb_q8_attend", "kvb_q8_mass", "kvb_q8_evict", "Q8Cache",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkvb.so")

KVB_BF16, KVB_F32 = 0, 1
KVB_DENSITYKV, KVB_FORCINGKV = 0, 1
KVB_ORDER_DISTURBANCE, KVB_ORDER_SOURCE = 0, 1
KVB_BASELINES_FIXED, KVB_BASELINES_REFRESH = 0, 1
KVB_EVICT_THRESHOLD_RATIO, KVB_EVICT_DENSEST, KVB_EVICT_THRESHOLD_SOURCE = 0, 1, 2
KVB_BOTTOMK_FRAME, KVB_BOTTOMK_CALL = 0, 1
KVB_SIM_PER_LAYER, KVB_SIM_FIRST_LAYER = 0, 1
KVB_STORE_NATIVE, KVB_STORE_FP8_E4M3 = 0, 1
KVB_ROPE_INTERLEAVED, KVB_ROPE_HALVES = 0, 1

# The Soft-Riesz parameters the DensityKV pages select (§4 parameter sensitivity,
# App. E parameter sweeps: width sigma = 8, decay p = 2, regulariser eps fixed
# at 1) in this library's form phi = (||a - b||^2 / h + eps)^(-s/2): h = sigma^2.
# make_config(**PAGES_PRESET) uses them instead of the defaults (h = d, eps 1e-3).
PAGES_PRESET = dict(dist_scale=64.0, eps=1.0, s=2.0)

STATUS = {0: "KVB_OK", 1: "KVB_E_INVAL", 2: "KVB_E_WORKSPACE", 3: "KVB_E_CUDA", 4: "KVB_E_DEVICE_TIMEOUT",
          5: "KVB_E_DEVICE_BOUNDS", 6: "KVB_E_STATE", 7: "KVB_E_UNSUPPORTED"}


class KvbError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({kvb_status_string(status)})")


class kvb_config(ctypes.Structure):
    _fields_ = [
        ("method", ctypes.c_int), ("dtype", ctypes.c_int),
        ("layers", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("capacity", ctypes.c_int32), ("max_candidates", ctypes.c_int32),
        ("tau", ctypes.c_float), ("eps", ctypes.c_float), ("s", ctypes.c_float), ("dist_scale", ctypes.c_float),
        ("sync_heads", ctypes.c_int32),
        ("frame_h", ctypes.c_int32), ("frame_w", ctypes.c_int32), ("seg_h", ctypes.c_int32),
        ("seg_w", ctypes.c_int32), ("hist_frames", ctypes.c_int32), ("max_new_frames", ctypes.c_int32),
        ("retention", ctypes.c_float), ("max_queries", ctypes.c_int32),
        ("cand_order", ctypes.c_int32), ("baselines", ctypes.c_int32), ("evict_order", ctypes.c_int32),
        ("bottomk_scope", ctypes.c_int32), ("sim_source", ctypes.c_int32), ("storage", ctypes.c_int32),
    ]


class kvb_admit_stats(ctypes.Structure):
    _fields_ = [("admitted", ctypes.c_int32), ("feasible", ctypes.c_int32), ("mandatory", ctypes.c_int32),
                ("capacity_evicted", ctypes.c_int32), ("size", ctypes.c_int32), ("moved", ctypes.c_int32),
                ("near_ties", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def make_config(**kw) -> kvb_config:
    """kvb_config with the pages' defaults (tau 2, eps 1e-3, s 2, synchronised heads)."""
    c = kvb_config()
    defaults = dict(method=KVB_DENSITYKV, dtype=KVB_BF16, layers=1, heads=12, head_dim=128, capacity=9360,
                    max_candidates=4680, tau=2.0, eps=1e-3, s=2.0, dist_scale=0.0, sync_heads=1,
                    frame_h=0, frame_w=0, seg_h=4, seg_w=4, hist_frames=21, max_new_frames=3,
                    retention=0.7, max_queries=4680, cand_order=KVB_ORDER_DISTURBANCE,
                    baselines=KVB_BASELINES_FIXED, evict_order=KVB_EVICT_THRESHOLD_RATIO,
                    bottomk_scope=KVB_BOTTOMK_FRAME, sim_source=KVB_SIM_PER_LAYER, storage=KVB_STORE_NATIVE)
    defaults.update(kw)
    for k, v in defaults.items():
        setattr(c, k, v)
    return c


class kvb_trace_record(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char_p), ("ms", ctypes.c_float), ("device", ctypes.c_int32)]


class kvb_q8_cache(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("block", ctypes.c_int32), ("K", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("mass", ctypes.c_void_p), ("status", ctypes.c_void_p)]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m kv_cache_compression_post_b200.build`")

lib = ctypes.CDLL(LIB_PATH)

_vp, _i32, _f, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_i64, _q8 = ctypes.c_int64, ctypes.POINTER(kvb_q8_cache)
_SIGS = {
    "kvb_workspace_size": (_sz, [ctypes.POINTER(kvb_config)]),
    "kvb_bank_create": (ctypes.c_int, [ctypes.POINTER(kvb_config), _vp, _sz, _vp, ctypes.POINTER(_vp)]),
    "kvb_bank_destroy": (ctypes.c_int, [_vp]),
    "kvb_admit": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _i32, _vp]),
    "kvb_prune_hybrid": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp]),
    "kvb_attend": (ctypes.c_int, [_vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp]),
    "kvb_read_stats": (ctypes.c_int, [_vp, _i32, ctypes.POINTER(kvb_admit_stats), _vp]),
    "kvb_bank_export": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(_i32), _vp]),
    "kvb_bank_import": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp]),
    "kvb_device_status": (ctypes.c_int, [_vp, _vp]),
    "kvb_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kvb_launch_count": (ctypes.c_ulonglong, []),
    "kvb_trace_enable": (ctypes.c_int, [_i32]),
    "kvb_trace_read": (ctypes.c_int, [ctypes.POINTER(kvb_trace_record), _i32, ctypes.POINTER(_i32)]),
    "kvb_density_workspace_size": (_sz, [_i32, _i32, _i32, _i32, ctypes.c_int]),
    "kvb_density": (ctypes.c_int, [_vp, _i32, _vp, _i32, _i32, _i32, ctypes.c_int, _f, _f, _f, _i32, _vp, _vp,
                                   _sz, _vp]),
    "kvb_density_noalloc": (ctypes.c_int, [_vp, _i32, _vp, _i32, _i32, _i32, ctypes.c_int, _f, _f, _f, _i32, _vp,
                                           _vp, _vp]),
    "kvb_segment_cosine": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int, _vp,
                                          _vp]),
    "kvb_selftest_timeout": (ctypes.c_int, [_vp, _vp, ctypes.c_int64, _vp]),
    "kvb_admit_begin": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp]),
    "kvb_admit_finish": (ctypes.c_int, [_vp, _i32, _vp, _vp]),
    "kvb_rope": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, ctypes.c_int, ctypes.POINTER(_i32), _f, ctypes.c_int, _i32,
                                _i64, _i64, _vp, _i64, _i64, _vp]),
    "kvb_q8_workspace_size": (_sz, [_q8, _i32, ctypes.c_int]),
    "kvb_q8_append": (ctypes.c_int, [_q8, _vp, _i64, _i64, _vp, _i64, _i64, _i32, ctypes.c_int, _vp, _vp]),
    "kvb_q8_attend": (ctypes.c_int, [_q8, _vp, _i32, ctypes.c_int, _f, _vp, _vp, _vp, _sz, _vp]),
    "kvb_q8_mass": (ctypes.c_int, [_q8, _vp, _i32, ctypes.c_int, _f, _vp, _f, _vp, _vp, _sz, _vp]),
    "kvb_q8_evict": (ctypes.c_int, [_q8, _q8, _i32, _i32, _i32, _vp, _vp, _sz, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        import torch
        if torch.cuda.is_initialized():     # the current stream's handle, without a Stream object around it
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(st: int, where: str) -> None:
    if st != 0:
        raise KvbError(st, where)


def kvb_launch_count() -> int:
    return int(lib.kvb_launch_count())


def kvb_trace_enable(enable: bool) -> None:
    _check(lib.kvb_trace_enable(1 if enable else 0), "kvb_trace_enable")


def kvb_trace_read(max_records: int = 65536) -> list:
    """[(kernel name, device ms), ...] of the launches traced since the last read,
    in launch order (waits for their events)."""
    buf = (kvb_trace_record * max_records)()
    n = _i32(0)
    _check(lib.kvb_trace_read(buf, max_records, ctypes.byref(n)), "kvb_trace_read")
    return [(buf[i].kernel.decode(), float(buf[i].ms)) for i in range(min(n.value, max_records))]


def kvb_status_string(status: int) -> str:
    return lib.kvb_status_string(status).decode()


def kvb_workspace_size(cfg: kvb_config) -> int:
    return lib.kvb_workspace_size(ctypes.byref(cfg))


def kvb_bank_create(cfg: kvb_config, workspace, workspace_bytes: int, stream=None) -> int:
    out = _vp()
    _check(lib.kvb_bank_create(ctypes.byref(cfg), _ptr(workspace), workspace_bytes, _stream(stream),
                               ctypes.byref(out)), "kvb_bank_create")
    return out.value


def kvb_bank_destroy(bank: int) -> None:
    _check(lib.kvb_bank_destroy(bank), "kvb_bank_destroy")


def kvb_admit(bank: int, layer: int, candK, candV, cand_ids, N: int, stream=None) -> None:
    _check(lib.kvb_admit(bank, layer, _ptr(candK), _ptr(candV), _ptr(cand_ids), N, _stream(stream)), "kvb_admit")


def kvb_admit_begin(bank: int, layer: int, candK, candV, cand_ids, N: int, prefix_out, stream=None) -> None:
    _check(lib.kvb_admit_begin(bank, layer, _ptr(candK), _ptr(candV), _ptr(cand_ids), N, _ptr(prefix_out),
                               _stream(stream)), "kvb_admit_begin")


def kvb_admit_finish(bank: int, layer: int, prefix_bound=None, stream=None) -> None:
    _check(lib.kvb_admit_finish(bank, layer, _ptr(prefix_bound), _stream(stream)), "kvb_admit_finish")


def kvb_prune_hybrid(bank: int, layer: int, head_is_static, newK, newV, nextK, new_ids, n_frames: int,
                     stream=None) -> None:
    """head_is_static: host bytes / bytearray / numpy uint8 array of length H."""
    import numpy as np
    if isinstance(head_is_static, (bytes, bytearray)):
        arr = np.frombuffer(bytes(head_is_static), dtype=np.uint8).copy()
    else:
        arr = np.ascontiguousarray(np.asarray(head_is_static, dtype=np.uint8))
    _check(lib.kvb_prune_hybrid(bank, layer, arr.ctypes.data, _ptr(newK), _ptr(newV), _ptr(nextK),
                                _ptr(new_ids), n_frames, _stream(stream)), "kvb_prune_hybrid")


def kvb_attend(bank: int, layer: int, Q, Nq: int, sinkK, sinkV, Ls: int, winK, winV, Lw: int, O, lse=None,
               stream=None) -> None:
    _check(lib.kvb_attend(bank, layer, _ptr(Q), Nq, _ptr(sinkK), _ptr(sinkV), Ls, _ptr(winK), _ptr(winV), Lw,
                          _ptr(O), _ptr(lse), _stream(stream)), "kvb_attend")


def kvb_read_stats(bank: int, layer: int, heads: int, stream=None):
    arr = (kvb_admit_stats * heads)()
    _check(lib.kvb_read_stats(bank, layer, arr, _stream(stream)), "kvb_read_stats")
    return [dict(admitted=a.admitted, feasible=a.feasible, mandatory=a.mandatory,
                 capacity_evicted=a.capacity_evicted, size=a.size, moved=a.moved, near_ties=a.near_ties)
            for a in arr]


def kvb_bank_export(bank: int, layer: int, head: int, ids, rho, rho0, K, V, stream=None) -> int:
    n = _i32()
    _check(lib.kvb_bank_export(bank, layer, head, _ptr(ids), _ptr(rho), _ptr(rho0), _ptr(K), _ptr(V),
                               ctypes.byref(n), _stream(stream)), "kvb_bank_export")
    return n.value


def kvb_bank_import(bank: int, layer: int, head: int, ids, rho, rho0, K, V, size: int, stream=None) -> None:
    _check(lib.kvb_bank_import(bank, layer, head, _ptr(ids), _ptr(rho), _ptr(rho0), _ptr(K), _ptr(V), size,
                               _stream(stream)), "kvb_bank_import")


def kvb_device_status(bank: int, stream=None) -> int:
    return lib.kvb_device_status(bank, _stream(stream))


def kvb_density_workspace_size(heads: int, n_rows: int, n_cols: int, head_dim: int, dtype: int) -> int:
    return lib.kvb_density_workspace_size(heads, n_rows, n_cols, head_dim, dtype)


def kvb_density(rows, n_rows: int, cols, n_cols: int, heads: int, head_dim: int, dtype: int, dist_scale: float,
                eps: float, s: float, exclude_diagonal: int, out, workspace, workspace_bytes: int,
                stream=None) -> None:
    _check(lib.kvb_density(_ptr(rows), n_rows, _ptr(cols), n_cols, heads, head_dim, dtype, dist_scale, eps, s,
                           exclude_diagonal, _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)),
           "kvb_density")


def kvb_selftest_timeout(status, out, timeout_ns: int, stream=None) -> None:
    """Run the library's bounded mbarrier wait to expiry (see kvb.h): status is a
    device int32 word, out a device int64[4]."""
    _check(lib.kvb_selftest_timeout(_ptr(status), _ptr(out), int(timeout_ns), _stream(stream)), "kvb_selftest_timeout")


def kvb_density_noalloc(rows, n_rows: int, cols, n_cols: int, heads: int, head_dim: int, dtype: int,
                        dist_scale: float, eps: float, s: float, exclude_diagonal: int, out, status_out=None,
                        stream=None) -> None:
    """kvb_density without a workspace (scratch in a fixed device array of the library)."""
    _check(lib.kvb_density_noalloc(_ptr(rows), n_rows, _ptr(cols), n_cols, heads, head_dim, dtype, dist_scale, eps,
                                   s, exclude_diagonal, _ptr(out), _ptr(status_out), _stream(stream)),
           "kvb_density_noalloc")


def kvb_segment_cosine(K, nextK, heads: int, n_frames: int, frame_h: int, frame_w: int, seg_h: int, seg_w: int,
                       head_dim: int, dtype: int, sim, stream=None) -> None:
    _check(lib.kvb_segment_cosine(_ptr(K), _ptr(nextK), heads, n_frames, frame_h, frame_w, seg_h, seg_w, head_dim,
                                  dtype, _ptr(sim), _stream(stream)), "kvb_segment_cosine")


def kvb_rope(X, pos, heads: int, n_tokens: int, head_dim: int, dtype: int, axis_pairs, base: float, pairing: int,
             inverse: int, x_head_stride: int, x_token_stride: int, out, out_head_stride: int, out_token_stride: int,
             stream=None) -> None:
    """axis_pairs: three host integers."""
    _check(lib.kvb_rope(_ptr(X), _ptr(pos), heads, n_tokens, head_dim, dtype, (_i32 * 3)(*axis_pairs), base, pairing,
                        inverse, x_head_stride, x_token_stride, _ptr(out), out_head_stride, out_token_stride,
                        _stream(stream)), "kvb_rope")


def kvb_q8_workspace_size(cache: kvb_q8_cache, max_queries: int, dtype: int) -> int:
    return lib.kvb_q8_workspace_size(ctypes.byref(cache), max_queries, dtype)


def kvb_q8_append(cache: kvb_q8_cache, K, k_head_stride: int, k_token_stride: int, V, v_head_stride: int,
                  v_token_stride: int, n: int, dtype: int, start=None, stream=None) -> None:
    _check(lib.kvb_q8_append(ctypes.byref(cache), _ptr(K), k_head_stride, k_token_stride, _ptr(V), v_head_stride,
                             v_token_stride, n, dtype, _ptr(start), _stream(stream)), "kvb_q8_append")


def kvb_q8_attend(cache: kvb_q8_cache, Q, Nq: int, dtype: int, scale: float, O, lse, workspace, workspace_bytes: int,
                  stream=None) -> None:
    _check(lib.kvb_q8_attend(ctypes.byref(cache), _ptr(Q), Nq, dtype, scale, _ptr(O), _ptr(lse), _ptr(workspace),
                             workspace_bytes, _stream(stream)), "kvb_q8_attend")


def kvb_q8_mass(cache: kvb_q8_cache, Q, Nq: int, dtype: int, scale: float, lse, decay: float, prev, workspace,
                workspace_bytes: int, stream=None) -> None:
    _check(lib.kvb_q8_mass(ctypes.byref(cache), _ptr(Q), Nq, dtype, scale, _ptr(lse), decay, _ptr(prev),
                           _ptr(workspace), workspace_bytes, _stream(stream)), "kvb_q8_mass")


def kvb_q8_evict(src: kvb_q8_cache, dst: kvb_q8_cache, budget: int, sink: int, recent: int, kept, workspace,
                 workspace_bytes: int, stream=None) -> None:
    _check(lib.kvb_q8_evict(ctypes.byref(src), ctypes.byref(dst), budget, sink, recent, _ptr(kept), _ptr(workspace),
                            workspace_bytes, _stream(stream)), "kvb_q8_evict")


def _tensor_dtype(x, where: str) -> int:
    import torch
    if x.dtype is torch.bfloat16:
        return KVB_BF16
    if x.dtype is torch.float32:
        return KVB_F32
    raise KvbError(1, where)


def _device(device, where: str) -> int:
    """The current device's ordinal, which has to be `device` where that is given: a kernel
    runs on the current device, and its tensors have to lie there."""
    import torch
    if not torch.cuda.is_initialized():
        raise KvbError(1, where)
    now = torch._C._cuda_getDevice()
    if device is not None and now != device:
        raise KvbError(1, where)
    return now


def _rows(x, shape, dtype, device: int, where: str):
    """The head and token strides of a [heads][n][d] tensor of a call, in any order of its
    rows: its shape, type and device are checked, and that a row is contiguous.  The
    stride of a dimension of one row says nothing and counts as 0."""
    if x.shape != shape or x.dtype is not dtype or x.get_device() != device:
        raise KvbError(1, where)
    h, n, e = x.stride()
    if e != 1 and shape[2] != 1:
        raise KvbError(1, where)
    return (h if shape[0] > 1 else 0), (n if shape[1] > 1 else 0)


def _whole(x, shape, dtype, device: int, where: str) -> int:
    """The address of a contiguous tensor of a call, checked (None passes, as 0)."""
    if x is None:
        return 0
    if x.shape != shape or x.dtype is not dtype or x.get_device() != device or not x.is_contiguous():
        raise KvbError(1, where)
    return x.data_ptr()


def rope(X, pos, out, axis_pairs, base: float = 10000.0, pairing: int = KVB_ROPE_INTERLEAVED, inverse: bool = False,
         stream=None) -> None:
    """kvb_rope on [heads][tokens][d] views of any row order (``x.transpose(0, 1)`` of a
    token-major tensor, say), both of one type; pos int32 [tokens][3]."""
    import torch
    dtype = _tensor_dtype(X, "kvb_rope")
    dev = _device(None, "kvb_rope")
    if X.dim() != 3 or len(axis_pairs) != 3:
        raise KvbError(1, "kvb_rope")
    shape = X.shape
    xh, xt = _rows(X, shape, X.dtype, dev, "kvb_rope")
    oh, ot = _rows(out, shape, X.dtype, dev, "kvb_rope")
    st = lib.kvb_rope(X.data_ptr(), _whole(pos, (shape[1], 3), torch.int32, dev, "kvb_rope"), shape[0], shape[1], shape[2],
                      dtype, (_i32 * 3)(*axis_pairs), base, pairing, 1 if inverse else 0, xh, xt, out.data_ptr(), oh,
                      ot, _stream(stream))
    if st:
        raise KvbError(st, "kvb_rope")


class Q8Cache:
    """A kvb_q8_cache over torch tensors of the current device, with the workspace for up
    to ``max_queries`` rows per head.  Tensors not given are allocated; lengths, weights
    and the status word then start at zero.  Calls on one cache share its workspace, so
    order them on one stream.

    Marshalling only: every method calls the C entry point named in its docstring, on the
    tensors' addresses after checking their shapes, types and layouts."""

    def __init__(self, heads: int, head_dim: int, capacity: int, block: int = 64, dtype: int = KVB_BF16,
                 max_queries: int = 1, with_mass: bool = False, K=None, V=None, k_scale=None, v_scale=None, len=None,
                 mass=None):
        import torch

        def own(x, shape, dt, make):
            if x is None:
                return make(shape, dtype=dt, device="cuda")
            _whole(x, shape, dt, self.device, "kvb_q8_cache")
            return x

        torch.cuda.init()
        self.device = _device(None, "kvb_q8_cache")
        if block not in (16, 32, 64, 128) or capacity % block:
            raise KvbError(1, "kvb_q8_cache")
        self.heads, self.head_dim, self.capacity, self.block = heads, head_dim, capacity, block
        self.dtype, self.max_queries = dtype, max_queries
        self.torch_dtype = torch.float32 if dtype == KVB_F32 else torch.bfloat16
        self.K = own(K, (heads, capacity, head_dim), torch.uint8, torch.empty)
        self.V = own(V, (heads, capacity, head_dim), torch.uint8, torch.empty)
        self.k_scale = own(k_scale, (heads, capacity // block), torch.float32, torch.empty)
        self.v_scale = own(v_scale, (heads, capacity // block), torch.float32, torch.empty)
        self.len = own(len, (heads,), torch.int32, torch.zeros)
        self.mass = own(mass, (heads, capacity), torch.float32, torch.zeros) if mass is not None or with_mass else None
        self.status_word = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.c = kvb_q8_cache(heads, head_dim, capacity, block, self.K.data_ptr(), self.V.data_ptr(),
                              self.k_scale.data_ptr(), self.v_scale.data_ptr(), self.len.data_ptr(), _ptr(self.mass),
                              self.status_word.data_ptr())
        self._ref = ctypes.byref(self.c)
        self.nbytes = kvb_q8_workspace_size(self.c, max_queries, dtype)
        if self.nbytes == 0:
            raise KvbError(1, "kvb_q8_workspace_size")
        self._buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device="cuda")
        self.ws = (self._buf.data_ptr() + 255) & ~255

    def append(self, K, V, start=None, stream=None) -> None:
        """kvb_q8_append: K, V [heads][n][d] in any row order; start int32 [heads] or None."""
        import torch
        dev = _device(self.device, "kvb_q8_append")
        shape = (self.heads, K.shape[1] if K.dim() == 3 else -1, self.head_dim)
        kh, kt = _rows(K, shape, self.torch_dtype, dev, "kvb_q8_append")
        vh, vt = _rows(V, shape, self.torch_dtype, dev, "kvb_q8_append")
        st = lib.kvb_q8_append(self._ref, K.data_ptr(), kh, kt, V.data_ptr(), vh, vt, shape[1], self.dtype,
                               _whole(start, (self.heads,), torch.int32, dev, "kvb_q8_append"), _stream(stream))
        if st:
            raise KvbError(st, "kvb_q8_append")

    def attend(self, Q, O, lse=None, scale: float = 0.0, stream=None) -> None:
        """kvb_q8_attend: Q, O [heads][Nq][d], lse f32 [heads][Nq] or None."""
        import torch
        dev = _device(self.device, "kvb_q8_attend")
        n = Q.shape[1] if Q.dim() == 3 else 0
        shape = (self.heads, n, self.head_dim)
        st = lib.kvb_q8_attend(self._ref, _whole(Q, shape, self.torch_dtype, dev, "kvb_q8_attend"), n, self.dtype, scale,
                               _whole(O, shape, self.torch_dtype, dev, "kvb_q8_attend"),
                               _whole(lse, (self.heads, n), torch.float32, dev, "kvb_q8_attend"), self.ws, self.nbytes,
                               _stream(stream))
        if st:
            raise KvbError(st, "kvb_q8_attend")

    def accumulate(self, Q, lse, decay: float = 1.0, prev=None, scale: float = 0.0, stream=None) -> None:
        """kvb_q8_mass: ``mass`` = decay * prev + the weights of these queries; prev None is
        the present ``mass``."""
        import torch
        dev = _device(self.device, "kvb_q8_mass")
        n = Q.shape[1] if Q.dim() == 3 else 0
        st = lib.kvb_q8_mass(self._ref, _whole(Q, (self.heads, n, self.head_dim), self.torch_dtype, dev, "kvb_q8_mass"), n,
                             self.dtype, scale, _whole(lse, (self.heads, n), torch.float32, dev, "kvb_q8_mass"), decay,
                             _whole(self.mass if prev is None else prev, (self.heads, self.capacity), torch.float32, dev,
                                    "kvb_q8_mass"), self.ws, self.nbytes, _stream(stream))
        if st:
            raise KvbError(st, "kvb_q8_mass")

    def evict(self, to: "Q8Cache", budget: int, sink: int = 0, recent: int = 0, kept=None, stream=None) -> None:
        """kvb_q8_evict into another cache of the device; kept int32 [heads][budget] or None."""
        import torch
        dev = _device(self.device, "kvb_q8_evict")
        if to.device != dev:
            raise KvbError(1, "kvb_q8_evict")
        st = lib.kvb_q8_evict(self._ref, to._ref, budget, sink, recent,
                              _whole(kept, (self.heads, budget), torch.int32, dev, "kvb_q8_evict"), self.ws, self.nbytes,
                              _stream(stream))
        if st:
            raise KvbError(st, "kvb_q8_evict")

    def status(self) -> int:
        """The status word (synchronises)."""
        return int(self.status_word.item())


class Bank:
    """A kvb bank whose workspace is a torch uint8 tensor on the current device.

    Marshalling only: every method calls the C entry point of the same name."""

    def __init__(self, cfg: kvb_config, stream=None):
        import torch
        self.cfg = cfg
        self.nbytes = kvb_workspace_size(cfg)
        if self.nbytes == 0:
            raise KvbError(1, "kvb_workspace_size")
        self._buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device="cuda")
        self.ws = (self._buf.data_ptr() + 255) & ~255
        self.handle = kvb_bank_create(cfg, self.ws, self.nbytes, stream)

    def close(self):
        if getattr(self, "handle", None):
            kvb_bank_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def admit(self, layer, candK, candV, cand_ids, stream=None):
        kvb_admit(self.handle, layer, candK, candV, cand_ids, cand_ids.shape[0], stream)

    def admit_begin(self, layer, candK, candV, cand_ids, prefix_out, stream=None):
        kvb_admit_begin(self.handle, layer, candK, candV, cand_ids, cand_ids.shape[0], prefix_out, stream)
        # the library reads the candidates again in kvb_admit_finish: keep them alive
        self._pending = (candK, candV, cand_ids)

    def admit_finish(self, layer, prefix_bound=None, stream=None):
        kvb_admit_finish(self.handle, layer, prefix_bound, stream)
        self._pending = None

    def prune_hybrid(self, layer, head_is_static, newK, newV, nextK, new_ids, n_frames, stream=None):
        kvb_prune_hybrid(self.handle, layer, head_is_static, newK, newV, nextK, new_ids, n_frames, stream)

    def attend(self, layer, Q, sinkK, sinkV, winK, winV, O, lse=None, stream=None):
        kvb_attend(self.handle, layer, Q, Q.shape[1], sinkK, sinkV, sinkK.shape[1], winK, winV, winK.shape[1],
                   O, lse, stream)

    def stats(self, layer, stream=None):
        return kvb_read_stats(self.handle, layer, self.cfg.heads, stream)

    def status(self, stream=None) -> int:
        return kvb_device_status(self.handle, stream)

    def export(self, layer, head, stream=None):
        """(ids, rho, rho0, K, V) torch tensors of one (layer, head) bank or history."""
        import torch
        cap = self.cfg.capacity if self.cfg.method == KVB_DENSITYKV else \
            self.cfg.hist_frames * self.cfg.frame_h * self.cfg.frame_w
        dt = torch.bfloat16 if self.cfg.dtype == KVB_BF16 else torch.float32
        ids = torch.empty(cap, dtype=torch.int32, device="cuda")
        rho = torch.zeros(cap, dtype=torch.float32, device="cuda")
        rho0 = torch.zeros(cap, dtype=torch.float32, device="cuda")
        K = torch.empty(cap, self.cfg.head_dim, dtype=dt, device="cuda")
        V = torch.empty(cap, self.cfg.head_dim, dtype=dt, device="cuda")
        n = kvb_bank_export(self.handle, layer, head, ids, rho, rho0, K, V, stream)
        return ids[:n], rho[:n], rho0[:n], K[:n], V[:n]

    def import_(self, layer, head, ids, rho, rho0, K, V, stream=None):
        kvb_bank_import(self.handle, layer, head, ids, rho, rho0, K, V, int(ids.shape[0]), stream)
