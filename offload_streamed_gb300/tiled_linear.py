"""Python binding of ``libtiled_linear.so`` (the C ABI in ``include/tiled_linear.h``).

Argument marshalling only: every step of the forward / backward path runs in
the library's CUDA kernels and copy streams.  There is no fallback: if the
shared library is missing or fails to load, every entry point raises.

Module-level functions carry the C names and take plain integers (pointers,
sizes, stream handles).  ``TiledLinear`` and ``PinnedBuffer`` wrap them for
PyTorch callers: PyTorch provides device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import _build

(TL_OK, TL_ERR_INVALID, TL_ERR_NOT_PINNED, TL_ERR_WORKSPACE, TL_ERR_CUDA, TL_ERR_TIMEOUT, TL_ERR_STATE,
 TL_ERR_IO) = range(8)
STATUS_NAMES = {0: "TL_OK", 1: "TL_ERR_INVALID", 2: "TL_ERR_NOT_PINNED", 3: "TL_ERR_WORKSPACE",
                4: "TL_ERR_CUDA", 5: "TL_ERR_TIMEOUT", 6: "TL_ERR_STATE", 7: "TL_ERR_IO"}


class TiledLinearError(RuntimeError):
    def __init__(self, status: int, where: str, message: str = ""):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}"
                         + (f" ({message})" if message else ""))


class tl_stats(ctypes.Structure):
    _fields_ = [
        ("n_tiles", ctypes.c_int32), ("depth", ctypes.c_int32),
        ("fwd_valid", ctypes.c_int32), ("bwd_valid", ctypes.c_int32),
        ("fwd_total_ms", ctypes.c_float), ("fwd_gemm_ms", ctypes.c_float), ("fwd_h2d_ms", ctypes.c_float),
        ("bwd_total_ms", ctypes.c_float), ("bwd_dw_gemm_ms", ctypes.c_float),
        ("bwd_dx_gemm_ms", ctypes.c_float), ("bwd_h2d_ms", ctypes.c_float), ("bwd_d2h_ms", ctypes.c_float),
        ("fwd_wait_ms", ctypes.c_float), ("bwd_wait_ms", ctypes.c_float),
        ("fwd_h2d_bytes", ctypes.c_int64), ("bwd_h2d_bytes", ctypes.c_int64), ("bwd_d2h_bytes", ctypes.c_int64),
        ("fwd_launches", ctypes.c_int32), ("bwd_launches", ctypes.c_int32),
        ("fwd_calls", ctypes.c_int64), ("bwd_calls", ctypes.c_int64),
        ("sum_fwd_total_ms", ctypes.c_double), ("sum_fwd_gemm_ms", ctypes.c_double),
        ("sum_fwd_h2d_ms", ctypes.c_double), ("sum_bwd_total_ms", ctypes.c_double),
        ("sum_bwd_dw_gemm_ms", ctypes.c_double), ("sum_bwd_dx_gemm_ms", ctypes.c_double),
        ("sum_bwd_h2d_ms", ctypes.c_double), ("sum_bwd_d2h_ms", ctypes.c_double),
        ("sum_bwd_gemm_ms", ctypes.c_double), ("bwd_gemm_ms", ctypes.c_float), ("staging_slots", ctypes.c_int32),
        ("bwd_reused_tiles", ctypes.c_int32),
        ("fwd_timed_calls", ctypes.c_int64), ("bwd_timed_calls", ctypes.c_int64), ("timing_every", ctypes.c_int32),
        ("fwd_h2d_max_ms", ctypes.c_float),
    ]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class tl_file_stats(ctypes.Structure):
    _fields_ = [("read_bytes", ctypes.c_int64), ("write_bytes", ctypes.c_int64),
                ("read_seconds", ctypes.c_double), ("write_seconds", ctypes.c_double),
                ("fetch_wait_seconds", ctypes.c_double), ("writeback_wait_seconds", ctypes.c_double),
                ("host_slots", ctypes.c_int32), ("io_threads", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


TL_TRACE_FWD_GEMM, TL_TRACE_DW_GEMM, TL_TRACE_DX_GEMM, TL_TRACE_H2D, TL_TRACE_D2H = range(5)
TRACE_KINDS = {0: "fwd_gemm", 1: "dw_gemm", 2: "dx_gemm", 3: "h2d", 4: "d2h"}


class tl_trace_event(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("tile", ctypes.c_int32),
                ("start_ms", ctypes.c_float), ("end_ms", ctypes.c_float)]


class tl_adam_config(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("threads", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def lib_path() -> str:
    return _build.LIB


def load():
    """Load the shared library (it must have been built: ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(path)
        i64, i32, sz, vp, st = ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
        L.tiled_linear_workspace_bytes.argtypes = [i64, i64, i32, i32]
        L.tiled_linear_workspace_bytes.restype = sz
        for name in ("tiled_linear_create", "tiled_linear_create_tilemajor"):
            fn = getattr(L, name)
            fn.argtypes = [ctypes.POINTER(vp), i64, i64, i32, i32, vp, vp, vp, sz, ctypes.c_int]
            fn.restype = st
        L.tiled_linear_create_file.argtypes = [ctypes.POINTER(vp), i64, i64, i32, i32, ctypes.c_char_p,
                                               ctypes.c_char_p, i32, i32, vp, sz, ctypes.c_int]
        L.tiled_linear_create_file.restype = st
        L.tiled_linear_file_sync.argtypes = [vp]
        L.tiled_linear_file_sync.restype = st
        L.tiled_linear_file_stats.argtypes = [vp, vp]
        L.tiled_linear_file_stats.restype = st
        L.tiled_linear_forward.argtypes = [vp, i64, vp, vp, vp]
        L.tiled_linear_forward.restype = st
        L.tiled_linear_backward.argtypes = [vp, i64, vp, vp, vp, vp]
        L.tiled_linear_backward.restype = st
        L.tiled_linear_destroy.argtypes = [vp]
        L.tiled_linear_destroy.restype = st
        L.tiled_linear_last_error.argtypes = [vp]
        L.tiled_linear_last_error.restype = ctypes.c_char_p
        L.tiled_linear_get_stats.argtypes = [vp, vp]
        L.tiled_linear_get_stats.restype = st
        L.tiled_linear_get_trace.argtypes = [vp, i32, vp, i32, ctypes.POINTER(i32)]
        L.tiled_linear_get_trace.restype = st
        L.tiled_linear_reset_stats.argtypes = [vp]
        L.tiled_linear_reset_stats.restype = st
        L.tiled_linear_set_tile_reuse.argtypes = [vp, i32]
        L.tiled_linear_set_tile_reuse.restype = st
        L.tiled_linear_set_timing.argtypes = [vp, i32]
        L.tiled_linear_set_timing.restype = st
        L.tiled_linear_set_stall_allowance.argtypes = [vp, ctypes.c_double]
        L.tiled_linear_set_stall_allowance.restype = st
        L.tiled_linear_adam_update.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, vp]
        L.tiled_linear_adam_update.restype = st
        L.tiled_linear_optimizer_create.argtypes = [ctypes.POINTER(vp), vp, vp, vp, vp, vp, vp]
        L.tiled_linear_optimizer_create.restype = st
        for name in ("tiled_linear_optimizer_accumulate", "tiled_linear_optimizer_step",
                     "tiled_linear_optimizer_wait", "tiled_linear_optimizer_destroy"):
            getattr(L, name).argtypes = [vp]
            getattr(L, name).restype = st
        L.tiled_linear_optimizer_stats.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_double)]
        L.tiled_linear_optimizer_stats.restype = st
        L.tiled_linear_chain_workspace_bytes.argtypes = [i32, vp, vp, i32]
        L.tiled_linear_chain_workspace_bytes.restype = sz
        L.tiled_linear_chain_create.argtypes = [ctypes.POINTER(vp), i32, vp, vp, i32, vp, vp, vp, sz, ctypes.c_int]
        L.tiled_linear_chain_create.restype = st
        L.tiled_linear_chain_forward.argtypes = [vp, i64, vp, vp, vp]
        L.tiled_linear_chain_forward.restype = st
        L.tiled_linear_chain_scratch_bytes.argtypes = [i64, i32, vp]
        L.tiled_linear_chain_scratch_bytes.restype = sz
        L.tiled_linear_chain_backward.argtypes = [vp, i64, vp, vp, vp, vp, vp, sz, vp]
        L.tiled_linear_chain_backward.restype = st
        L.tiled_linear_gemm_forward.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp]
        L.tiled_linear_gemm_forward.restype = st
        L.tiled_linear_gemm_dw.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp]
        L.tiled_linear_gemm_dw.restype = st
        L.tiled_linear_gemm_dx.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, i32, vp, vp]
        L.tiled_linear_gemm_dx.restype = st
        L.tiled_linear_gemm_dx_bf16.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp]
        L.tiled_linear_gemm_dx_bf16.restype = st
        L.tiled_linear_selftest_timeout.argtypes = [vp, sz, i64, vp]
        L.tiled_linear_selftest_timeout.restype = st
        L.tiled_linear_forward_static.argtypes = [i64, i64, i64, i32, vp, vp, vp, vp, vp]
        L.tiled_linear_forward_static.restype = st
        L.tiled_linear_operator_error_word.argtypes = [ctypes.POINTER(vp)]
        L.tiled_linear_operator_error_word.restype = st
        L.tiled_linear_norm_forward.argtypes = [i64, i64, i32, vp, i64, i32, vp, vp, ctypes.c_float, vp, i64, vp,
                                                vp, vp, vp]
        L.tiled_linear_norm_forward.restype = st
        L.tiled_linear_norm_backward_workspace_bytes.argtypes = [i64, i64]
        L.tiled_linear_norm_backward_workspace_bytes.restype = sz
        L.tiled_linear_norm_backward.argtypes = [i64, i64, i32, vp, i64, vp, i64, vp, vp, i32, vp, vp, i64, vp, vp,
                                                 vp, sz, vp, vp]
        L.tiled_linear_norm_backward.restype = st
        L.tiled_linear_fp8_quantize.argtypes = [i64, i64, i32, vp, i64, i32] + [vp, i64, vp] * 3 + [vp]
        L.tiled_linear_fp8_quantize.restype = st
        for name in ("tiled_linear_fp8_gemm_forward", "tiled_linear_fp8_gemm_dx", "tiled_linear_fp8_gemm_dw"):
            getattr(L, name).argtypes = [i64, i64, i64] + [i32, vp, i64, vp] * 2 + [vp, i64, vp, vp]
            getattr(L, name).restype = st
        for name in ("tiled_linear_fp8_linear_workspace_bytes", "tiled_linear_fp8_linear_backward_workspace_bytes"):
            getattr(L, name).argtypes = [i64, i64, i64]
            getattr(L, name).restype = sz
        L.tiled_linear_fp8_linear.argtypes = [i64, i64, i64, i32, vp, i64, i32, vp, i64, vp, vp, i64, vp, sz, vp, vp]
        L.tiled_linear_fp8_linear.restype = st
        L.tiled_linear_fp8_linear_backward.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, i32, vp, i64, vp, vp, i64,
                                                       vp, i64, vp, sz, vp, vp]
        L.tiled_linear_fp8_linear_backward.restype = st
        L.tiled_linear_orthogonalize_workspace_bytes.argtypes = [i64, i64, i64]
        L.tiled_linear_orthogonalize_workspace_bytes.restype = sz
        L.tiled_linear_orthogonalize.argtypes = [i64, i64, i64, i32, vp, i64, i64, i32] + [ctypes.c_float] * 5 + \
            [vp, i64, i64, vp, sz, vp, vp]
        L.tiled_linear_orthogonalize.restype = st
        L.tiled_linear_route_workspace_bytes.argtypes = [i64, i64, i64]
        L.tiled_linear_route_workspace_bytes.restype = sz
        L.tiled_linear_group_rows.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, sz, vp]
        L.tiled_linear_route.argtypes = [i64, i64, i64, i32, vp, i64, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.tiled_linear_route_backward.argtypes = [i64, i64, i64, i32, vp, i64, vp, vp, i32, vp, i64, vp]
        L.tiled_linear_combine.argtypes = [i64, i64, i64, i64, i32, vp, i64, vp, vp, vp, i64, vp]
        L.tiled_linear_combine_backward.argtypes = [i64, i64, i64, i64, i32, vp, i64, vp, vp, i64, vp, vp, i64, vp, vp]
        L.tiled_linear_grouped_workspace_bytes.argtypes = [i64, i64]
        L.tiled_linear_grouped_workspace_bytes.restype = sz
        L.tiled_linear_grouped_forward.argtypes = [i64, i64, i64, i64, i32, vp, i64, i64, vp, vp, i64, i64, vp, vp, i64, vp, sz, vp, vp]
        L.tiled_linear_grouped_dx.argtypes = [i64, i64, i64, i64, i32, vp, i64, vp, i64, i64, vp, vp, i64, vp, vp]
        L.tiled_linear_grouped_dw.argtypes = [i64, i64, i64, i64, i32, vp, i64, i64, vp, vp, i64, vp, vp, i64, i64, vp, sz, vp, vp]
        L.tiled_linear_adapter_workspace_bytes.argtypes = [i64, i64, i64]
        L.tiled_linear_adapter_workspace_bytes.restype = sz
        L.tiled_linear_adapter_forward.argtypes = [i64] * 5 + [i32, vp, i64, vp, i64, i64, vp, i64, i64, vp, vp, ctypes.c_float,
                                                               i32, vp, i64, vp, i64, vp, i64, vp, sz, vp, vp]
        L.tiled_linear_adapter_backward.argtypes = [i64] * 5 + [i32, vp, i64, vp, i64, vp, i64, vp, i64, i64, vp, i64, i64, vp,
                                                                vp, ctypes.c_float, i32, vp, i64, vp, i64, vp, i64, i64, vp,
                                                                i64, i64, vp, sz, vp, vp]
        for name in ("group_rows", "route", "route_backward", "combine", "combine_backward", "grouped_forward", "grouped_dx",
                     "grouped_dw", "adapter_forward", "adapter_backward"):
            getattr(L, "tiled_linear_" + name).restype = st
        L.tiled_linear_host_alloc.argtypes = [sz, ctypes.POINTER(vp)]
        L.tiled_linear_host_alloc.restype = st
        L.tiled_linear_host_free.argtypes = [vp]
        L.tiled_linear_host_free.restype = st
        L.tiled_linear_version.restype = ctypes.c_char_p
        _lib = L
        return L


def _check(status: int, where: str, handle=None):
    if status != TL_OK:
        raise TiledLinearError(status, where, tiled_linear_last_error(handle))


# --- the C ABI, name for name ----------------------------------------------

def tiled_linear_workspace_bytes(K: int, M: int, N: int, d: int) -> int:
    return int(load().tiled_linear_workspace_bytes(K, M, N, d))


def tiled_linear_create(K, M, N, d, w_host, dw_host, workspace_dev, workspace_bytes, device,
                        tile_major: bool = False) -> int:
    """Returns the handle (an integer).  ``tile_major`` selects
    ``tiled_linear_create_tilemajor``."""
    h = ctypes.c_void_p()
    fn = load().tiled_linear_create_tilemajor if tile_major else load().tiled_linear_create
    _check(fn(ctypes.byref(h), K, M, N, d, w_host, dw_host, workspace_dev, workspace_bytes, device),
           "tiled_linear_create")
    return h.value


def tiled_linear_create_tilemajor(K, M, N, d, w_host, dw_host, workspace_dev, workspace_bytes,
                                  device) -> int:
    return tiled_linear_create(K, M, N, d, w_host, dw_host, workspace_dev, workspace_bytes, device,
                               tile_major=True)


def tiled_linear_create_file(K, M, N, d, w_path: str, dw_path: str, host_slots: int, io_threads: int,
                             workspace_dev, workspace_bytes, device) -> int:
    """W and dW in files (tile-major), streamed through pinned host slots."""
    h = ctypes.c_void_p()
    _check(load().tiled_linear_create_file(ctypes.byref(h), K, M, N, d, os.fsencode(w_path), os.fsencode(dw_path),
                                           host_slots, io_threads, workspace_dev, workspace_bytes, device),
           "tiled_linear_create_file")
    return h.value


def tiled_linear_file_sync(h: int) -> None:
    _check(load().tiled_linear_file_sync(h), "tiled_linear_file_sync", h)


def tiled_linear_file_stats(h: int) -> dict:
    s = tl_file_stats()
    _check(load().tiled_linear_file_stats(h, ctypes.byref(s)), "tiled_linear_file_stats", h)
    return s.as_dict()


def tiled_linear_forward(h: int, T: int, x_dev: int, y_dev: int, stream: int) -> None:
    _check(load().tiled_linear_forward(h, T, x_dev, y_dev, stream), "tiled_linear_forward", h)


def tiled_linear_backward(h: int, T: int, x_dev: int, dy_dev: int, dx_dev: int, stream: int) -> None:
    _check(load().tiled_linear_backward(h, T, x_dev, dy_dev, dx_dev, stream), "tiled_linear_backward", h)


def tiled_linear_destroy(h: int) -> int:
    return int(load().tiled_linear_destroy(h))


def tiled_linear_last_error(h=None) -> str:
    msg = load().tiled_linear_last_error(h)
    return msg.decode(errors="replace") if msg else ""


def tiled_linear_get_stats(h: int) -> dict:
    s = tl_stats()
    _check(load().tiled_linear_get_stats(h, ctypes.byref(s)), "tiled_linear_get_stats", h)
    return s.as_dict()


def tiled_linear_get_trace(h: int, backward: bool) -> list:
    """The last timed forward / backward call's launches and copies: a list of
    {"kind", "tile", "start_ms", "end_ms"} (see include/tiled_linear.h)."""
    n = ctypes.c_int32(0)
    _check(load().tiled_linear_get_trace(h, 1 if backward else 0, None, 0, ctypes.byref(n)),
           "tiled_linear_get_trace", h)
    buf = (tl_trace_event * max(n.value, 1))()
    _check(load().tiled_linear_get_trace(h, 1 if backward else 0, buf, n.value, ctypes.byref(n)),
           "tiled_linear_get_trace", h)
    return [{"kind": TRACE_KINDS[e.kind], "tile": e.tile, "start_ms": e.start_ms, "end_ms": e.end_ms}
            for e in buf[:n.value]]


def tiled_linear_reset_stats(h: int) -> None:
    _check(load().tiled_linear_reset_stats(h), "tiled_linear_reset_stats", h)


def tiled_linear_set_timing(h: int, every: int) -> None:
    _check(load().tiled_linear_set_timing(h, int(every)), "tiled_linear_set_timing", h)


def tiled_linear_set_tile_reuse(h: int, enable: bool) -> None:
    _check(load().tiled_linear_set_tile_reuse(h, 1 if enable else 0), "tiled_linear_set_tile_reuse", h)


def tiled_linear_set_stall_allowance(h: int, ms: float) -> None:
    _check(load().tiled_linear_set_stall_allowance(h, float(ms)), "tiled_linear_set_stall_allowance", h)


def _i64s(v):
    return (ctypes.c_int64 * len(v))(*[int(a) for a in v])


def _i32s(v):
    return (ctypes.c_int32 * len(v))(*[int(a) for a in v])


def _ptrs(v):
    return (ctypes.c_void_p * len(v))(*[int(a) if a else None for a in v])


def tiled_linear_chain_workspace_bytes(L: int, dims, n_tiles, d: int) -> int:
    return int(load().tiled_linear_chain_workspace_bytes(L, _i64s(dims), _i32s(n_tiles), d))


def tiled_linear_chain_create(L, dims, n_tiles, d, w_hosts, dw_hosts, workspace_dev, workspace_bytes,
                              device) -> int:
    h = ctypes.c_void_p()
    _check(load().tiled_linear_chain_create(ctypes.byref(h), L, _i64s(dims), _i32s(n_tiles), d,
                                            _ptrs(w_hosts), _ptrs(dw_hosts), workspace_dev, workspace_bytes,
                                            device), "tiled_linear_chain_create")
    return h.value


def tiled_linear_chain_forward(h: int, T: int, x_dev: int, y_devs, stream: int) -> None:
    _check(load().tiled_linear_chain_forward(h, T, x_dev, _ptrs(y_devs), stream), "tiled_linear_chain_forward", h)


def tiled_linear_chain_scratch_bytes(T: int, L: int, dims) -> int:
    return int(load().tiled_linear_chain_scratch_bytes(T, L, _i64s(dims)))


def tiled_linear_chain_backward(h: int, T: int, x_dev: int, y_devs, dy_dev: int, dx_dev: int, scratch_dev: int,
                                scratch_bytes: int, stream: int) -> None:
    _check(load().tiled_linear_chain_backward(h, T, x_dev, _ptrs(y_devs) if y_devs is not None else None, dy_dev,
                                              dx_dev, scratch_dev, scratch_bytes, stream),
           "tiled_linear_chain_backward", h)


def adam_config(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, threads=0) -> tl_adam_config:
    return tl_adam_config(lr, beta1, beta2, eps, weight_decay, threads)


def tiled_linear_adam_update(cfg: tl_adam_config, step: int, n: int, master: int, m: int, v: int, grad_acc: int,
                             grad_bf16: int, w_bf16: int) -> None:
    _check(load().tiled_linear_adam_update(ctypes.byref(cfg), step, n, master, m, v, grad_acc or None, grad_bf16,
                                           w_bf16), "tiled_linear_adam_update")


def tiled_linear_optimizer_create(h: int, cfg: tl_adam_config, masters, ms, vs, accs=None) -> int:
    o = ctypes.c_void_p()
    _check(load().tiled_linear_optimizer_create(ctypes.byref(o), h, ctypes.byref(cfg), _ptrs(masters), _ptrs(ms),
                                                _ptrs(vs), _ptrs(accs) if accs else None),
           "tiled_linear_optimizer_create", h)
    return o.value


def tiled_linear_optimizer_accumulate(o: int, h=None) -> None:
    _check(load().tiled_linear_optimizer_accumulate(o), "tiled_linear_optimizer_accumulate", h)


def tiled_linear_optimizer_step(o: int, h=None) -> None:
    _check(load().tiled_linear_optimizer_step(o), "tiled_linear_optimizer_step", h)


def tiled_linear_optimizer_wait(o: int, h=None) -> None:
    _check(load().tiled_linear_optimizer_wait(o), "tiled_linear_optimizer_wait", h)


def tiled_linear_optimizer_stats(o: int) -> tuple:
    steps, busy = ctypes.c_int64(), ctypes.c_double()
    _check(load().tiled_linear_optimizer_stats(o, ctypes.byref(steps), ctypes.byref(busy)),
           "tiled_linear_optimizer_stats")
    return steps.value, busy.value


def tiled_linear_optimizer_destroy(o: int) -> int:
    return int(load().tiled_linear_optimizer_destroy(o))


def tiled_linear_gemm_forward(T, K, n, x, ldx, w, ldw, y, ldy, err, stream) -> None:
    _check(load().tiled_linear_gemm_forward(T, K, n, x, ldx, w, ldw, y, ldy, err, stream),
           "tiled_linear_gemm_forward")


def tiled_linear_gemm_dw(T, K, n, x, ldx, dy, lddy, dw, lddw, err, stream) -> None:
    _check(load().tiled_linear_gemm_dw(T, K, n, x, ldx, dy, lddy, dw, lddw, err, stream),
           "tiled_linear_gemm_dw")


def tiled_linear_gemm_dx(T, K, n, dy, lddy, w, ldw, dx, lddx, accumulate, err, stream) -> None:
    _check(load().tiled_linear_gemm_dx(T, K, n, dy, lddy, w, ldw, dx, lddx, int(accumulate), err, stream),
           "tiled_linear_gemm_dx")


def tiled_linear_gemm_dx_bf16(T, K, n, dy, lddy, w, ldw, addend, ld_add, dx, lddx, err, stream) -> None:
    _check(load().tiled_linear_gemm_dx_bf16(T, K, n, dy, lddy, w, ldw, addend, ld_add, dx, lddx, err, stream),
           "tiled_linear_gemm_dx_bf16")


def tiled_linear_selftest_timeout(scratch_dev: int, scratch_bytes: int, timeout_ns: int, stream: int) -> None:
    """Run the kernels' failure path once (see the header); the error bits
    land in the first int32 of scratch_dev."""
    _check(load().tiled_linear_selftest_timeout(scratch_dev, scratch_bytes, timeout_ns, stream),
           "tiled_linear_selftest_timeout")


def tiled_linear_forward_static(T, K, M, N, w_host, x_dev, y_dev, status_host, stream) -> None:
    """Forward with no device allocation (scratch in a static device array);
    see the header for its limit and ordering rules."""
    st = load().tiled_linear_forward_static(T, K, M, N, w_host, x_dev, y_dev, status_host, stream)
    if st != TL_OK:
        raise TiledLinearError(st, "tiled_linear_forward_static")


def tiled_linear_operator_error_word() -> int:
    p = ctypes.c_void_p()
    _check(load().tiled_linear_operator_error_word(ctypes.byref(p)), "tiled_linear_operator_error_word")
    return p.value


def tiled_linear_norm_forward(rows, cols, type, x, ldx, param_type, weight, bias, eps, y, ldy, mean, rstd, err,
                              stream) -> None:
    _check(load().tiled_linear_norm_forward(rows, cols, type, x, ldx, param_type, weight, bias, eps, y, ldy, mean,
                                            rstd, err, stream), "tiled_linear_norm_forward")


def tiled_linear_norm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return int(load().tiled_linear_norm_backward_workspace_bytes(rows, cols))


def tiled_linear_norm_backward(rows, cols, type, dy, lddy, x, ldx, mean, rstd, param_type, weight, dx, lddx, dweight,
                               dbias, workspace, workspace_bytes, err, stream) -> None:
    _check(load().tiled_linear_norm_backward(rows, cols, type, dy, lddy, x, ldx, mean, rstd, param_type, weight, dx,
                                             lddx, dweight, dbias, workspace, workspace_bytes, err, stream),
           "tiled_linear_norm_backward")


def tiled_linear_fp8_quantize(rows, cols, type, x, ldx, format, row_q, ld_row, row_scale, col_q, ld_col, col_scale,
                              tile_q, ld_tile, tile_scale, stream) -> None:
    _check(load().tiled_linear_fp8_quantize(rows, cols, type, x, ldx, format, row_q, ld_row, row_scale, col_q, ld_col,
                                            col_scale, tile_q, ld_tile, tile_scale, stream),
           "tiled_linear_fp8_quantize")


def tiled_linear_fp8_gemm_forward(T, K, n, x_format, x_q, ldx, x_scale, w_format, w_q, ldw, w_scale, y, ldy, err,
                                  stream) -> None:
    _check(load().tiled_linear_fp8_gemm_forward(T, K, n, x_format, x_q, ldx, x_scale, w_format, w_q, ldw, w_scale, y,
                                                ldy, err, stream), "tiled_linear_fp8_gemm_forward")


def tiled_linear_fp8_gemm_dx(T, K, n, dy_format, dy_q, lddy, dy_scale, w_format, w_q, ldw, w_scale, dx, lddx, err,
                             stream) -> None:
    _check(load().tiled_linear_fp8_gemm_dx(T, K, n, dy_format, dy_q, lddy, dy_scale, w_format, w_q, ldw, w_scale, dx,
                                           lddx, err, stream), "tiled_linear_fp8_gemm_dx")


def tiled_linear_fp8_gemm_dw(T, K, n, x_format, x_q, ldx, x_scale, dy_format, dy_q, lddy, dy_scale, dw, lddw, err,
                             stream) -> None:
    _check(load().tiled_linear_fp8_gemm_dw(T, K, n, x_format, x_q, ldx, x_scale, dy_format, dy_q, lddy, dy_scale, dw,
                                           lddw, err, stream), "tiled_linear_fp8_gemm_dw")


def tiled_linear_fp8_linear_workspace_bytes(T: int, K: int, n: int) -> int:
    return int(load().tiled_linear_fp8_linear_workspace_bytes(T, K, n))


def tiled_linear_fp8_linear(T, K, n, type, x, ldx, w_format, w_q, ldw, w_scale, y, ldy, workspace, workspace_bytes, err,
                            stream) -> None:
    _check(load().tiled_linear_fp8_linear(T, K, n, type, x, ldx, w_format, w_q, ldw, w_scale, y, ldy, workspace,
                                          workspace_bytes, err, stream), "tiled_linear_fp8_linear")


def tiled_linear_fp8_linear_backward_workspace_bytes(T: int, K: int, n: int) -> int:
    return int(load().tiled_linear_fp8_linear_backward_workspace_bytes(T, K, n))


def tiled_linear_fp8_linear_backward(T, K, n, type, x, ldx, dy, lddy, w_format, w_q, ldw, w_scale, dx, lddx, dw, lddw,
                                     workspace, workspace_bytes, err, stream) -> None:
    _check(load().tiled_linear_fp8_linear_backward(T, K, n, type, x, ldx, dy, lddy, w_format, w_q, ldw, w_scale, dx,
                                                   lddx, dw, lddw, workspace, workspace_bytes, err, stream),
           "tiled_linear_fp8_linear_backward")


def tiled_linear_orthogonalize_workspace_bytes(batch: int, rows: int, cols: int) -> int:
    return int(load().tiled_linear_orthogonalize_workspace_bytes(batch, rows, cols))


def tiled_linear_orthogonalize(batch, rows, cols, type, g, ldg, g_apart, steps, a, b, c, eps, scale, out, ldo, o_apart,
                               workspace, workspace_bytes, err, stream) -> None:
    _check(load().tiled_linear_orthogonalize(batch, rows, cols, type, g, ldg, g_apart, steps, a, b, c, eps, scale, out,
                                             ldo, o_apart, workspace, workspace_bytes, err, stream),
           "tiled_linear_orthogonalize")


def tiled_linear_route_workspace_bytes(T: int, k: int, groups: int) -> int:
    return int(load().tiled_linear_route_workspace_bytes(T, k, groups))


def tiled_linear_group_rows(T, k, groups, ids, slots, rows, offsets, workspace, workspace_bytes, stream) -> None:
    _check(load().tiled_linear_group_rows(T, k, groups, ids, slots, rows, offsets, workspace, workspace_bytes, stream),
           "tiled_linear_group_rows")


def tiled_linear_route(T, experts, k, type, logits, ld, normalize, weights, ids, slots, rows, offsets,
                       workspace, workspace_bytes, stream) -> None:
    _check(load().tiled_linear_route(T, experts, k, type, logits, ld, normalize, weights, ids, slots, rows, offsets,
                                     workspace, workspace_bytes, stream),
           "tiled_linear_route")


def tiled_linear_route_backward(T, experts, k, type, logits, ld, ids, dweights, normalize, dlogits, lddl,
                                stream) -> None:
    _check(load().tiled_linear_route_backward(T, experts, k, type, logits, ld, ids, dweights, normalize, dlogits,
                                              lddl, stream),
           "tiled_linear_route_backward")


def tiled_linear_combine(T, k, cols, rows, type, y, ldy, slots, weights, out, ldout, stream) -> None:
    _check(load().tiled_linear_combine(T, k, cols, rows, type, y, ldy, slots, weights, out, ldout, stream),
           "tiled_linear_combine")


def tiled_linear_combine_backward(T, k, cols, rows, type, dout, lddout, slots, y, ldy, weights, dy, lddy,
                                  dweights, stream) -> None:
    _check(load().tiled_linear_combine_backward(T, k, cols, rows, type, dout, lddout, slots, y, ldy, weights, dy,
                                                lddy, dweights, stream),
           "tiled_linear_combine_backward")


def tiled_linear_grouped_workspace_bytes(R: int, K: int) -> int:
    return int(load().tiled_linear_grouped_workspace_bytes(R, K))


def tiled_linear_grouped_forward(R, K, n, groups, type, x, ldx, x_rows, rows, w, ldw, w_apart, offsets, y,
                                 ldy, workspace, workspace_bytes, err, stream) -> None:
    _check(load().tiled_linear_grouped_forward(R, K, n, groups, type, x, ldx, x_rows, rows, w, ldw, w_apart, offsets,
                                               y, ldy, workspace, workspace_bytes, err, stream),
           "tiled_linear_grouped_forward")


def tiled_linear_grouped_dx(R, K, n, groups, type, dy, lddy, w, ldw, w_apart, offsets, dx, lddx, err, stream) -> None:
    _check(load().tiled_linear_grouped_dx(R, K, n, groups, type, dy, lddy, w, ldw, w_apart, offsets, dx, lddx, err,
                                          stream),
           "tiled_linear_grouped_dx")


def tiled_linear_grouped_dw(R, K, n, groups, type, x, ldx, x_rows, rows, dy, lddy, offsets, dw, lddw,
                            dw_apart, workspace, workspace_bytes, err, stream) -> None:
    _check(load().tiled_linear_grouped_dw(R, K, n, groups, type, x, ldx, x_rows, rows, dy, lddy, offsets, dw, lddw,
                                          dw_apart, workspace, workspace_bytes, err, stream),
           "tiled_linear_grouped_dw")


def tiled_linear_adapter_workspace_bytes(T: int, r: int, adapters: int) -> int:
    return int(load().tiled_linear_adapter_workspace_bytes(T, r, adapters))


def tiled_linear_adapter_forward(T, K, n, r, adapters, type, x, ldx, a, lda, a_apart, b, ldb, b_apart, ids,
                                 scale_dev, scale, base_type, base, ldbase, y, ldy, h, ldh, workspace,
                                 workspace_bytes, err, stream) -> None:
    _check(load().tiled_linear_adapter_forward(T, K, n, r, adapters, type, x, ldx, a, lda, a_apart, b, ldb, b_apart,
                                               ids, scale_dev, scale, base_type, base, ldbase, y, ldy, h, ldh,
                                               workspace, workspace_bytes, err, stream),
           "tiled_linear_adapter_forward")


def tiled_linear_adapter_backward(T, K, n, r, adapters, type, x, ldx, h, ldh, dy, lddy, a, lda, a_apart, b,
                                  ldb, b_apart, ids, scale_dev, scale, base_type, base, ldbase, dx, lddx,
                                  da, ldda, da_apart, db, lddb, db_apart, workspace, workspace_bytes, err,
                                  stream) -> None:
    _check(load().tiled_linear_adapter_backward(T, K, n, r, adapters, type, x, ldx, h, ldh, dy, lddy, a, lda, a_apart,
                                                b, ldb, b_apart, ids, scale_dev, scale, base_type, base, ldbase, dx,
                                                lddx, da, ldda, da_apart, db, lddb, db_apart, workspace,
                                                workspace_bytes, err, stream),
           "tiled_linear_adapter_backward")


def tiled_linear_host_alloc(nbytes: int) -> int:
    p = ctypes.c_void_p()
    _check(load().tiled_linear_host_alloc(nbytes, ctypes.byref(p)), "tiled_linear_host_alloc")
    return p.value


def tiled_linear_host_free(p: int) -> None:
    _check(load().tiled_linear_host_free(p), "tiled_linear_host_free")


def tiled_linear_version() -> str:
    return load().tiled_linear_version().decode()


# --- PyTorch convenience wrappers --------------------------------------------

def _stream_handle(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def host_tensor(ptr: int, numel: int, dtype=None):
    """Wrap ``numel`` elements of host memory at ``ptr`` as a CPU tensor (no
    copy; the memory stays owned by whoever allocated it)."""
    import torch
    dtype = dtype or torch.bfloat16
    itemsize = torch.empty((), dtype=dtype).element_size()
    buf = (ctypes.c_uint8 * (numel * itemsize)).from_address(ptr)
    return torch.frombuffer(buf, dtype=torch.uint8).view(dtype)


class PinnedBuffer:
    """Page-locked host memory from ``tiled_linear_host_alloc``, viewed as a
    CPU tensor of ``dtype``.  Freed by ``close()`` (or garbage collection)."""

    def __init__(self, numel: int, dtype=None):
        import torch
        self.dtype = dtype or torch.bfloat16
        self.numel = int(numel)
        itemsize = torch.empty((), dtype=self.dtype).element_size()
        self.nbytes = self.numel * itemsize
        self.ptr = tiled_linear_host_alloc(max(self.nbytes, 16))
        self.tensor = host_tensor(self.ptr, self.numel, self.dtype)

    def close(self):
        if self.ptr:
            self.tensor = None
            tiled_linear_host_free(self.ptr)
            self.ptr = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class TiledLinear:
    """Y = X.W with W [K, M] in pinned host memory, streamed in N output tiles
    through a depth-d device ring (see ``include/tiled_linear.h``).

    w_host / dw_host: pinned host buffers (``PinnedBuffer`` or a pinned CPU
    tensor) of K*M bf16 each, tile-major [N][K][M/N] when ``tile_major`` else
    row-major [K][M].  The workspace is a device uint8 tensor owned here.

    d = -1 (automatic depth): the workspace holds as many ring and staging
    slots as ``auto_workspace_bytes`` allows (default: half of the device's
    free memory), at most N of each."""

    def __init__(self, K: int, M: int, N: int, d: int, w_host, dw_host, *, tile_major: bool = True,
                 device=None, auto_workspace_bytes: int | None = None):
        import torch
        self.K, self.M, self.N, self.d = int(K), int(M), int(N), int(d)
        self.Mi = self.M // self.N
        self.tile_major = bool(tile_major)
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None else
                                   torch.device(device).index or 0)
        wb = tiled_linear_workspace_bytes(self.K, self.M, self.N, self.d)
        if wb == 0:
            raise TiledLinearError(TL_ERR_INVALID, "tiled_linear_workspace_bytes",
                                   f"invalid shape K={K} M={M} N={N} d={d}")
        if self.d < 0:
            least = tiled_linear_workspace_bytes(self.K, self.M, self.N, min(1, self.N - 1))
            budget = auto_workspace_bytes
            if budget is None:
                budget = torch.cuda.mem_get_info(self.device)[0] // 2
            wb = max(least, min(wb, int(budget)))
        self.workspace = torch.empty(wb, dtype=torch.uint8, device=self.device)
        self._w, self._dw = w_host, dw_host
        wp = w_host.ptr if isinstance(w_host, PinnedBuffer) else w_host.data_ptr()
        dwp = dw_host.ptr if isinstance(dw_host, PinnedBuffer) else dw_host.data_ptr()
        self.handle = tiled_linear_create(self.K, self.M, self.N, self.d, wp, dwp,
                                          self.workspace.data_ptr(), wb, self.device.index,
                                          tile_major=self.tile_major)

    def forward(self, x, y=None, stream=None):
        import torch
        T = x.shape[0]
        if y is None:
            y = torch.empty(T, self.M, dtype=torch.bfloat16, device=self.device)
        tiled_linear_forward(self.handle, T, x.data_ptr(), y.data_ptr(), _stream_handle(stream))
        return y

    def backward(self, x, dy, dx=None, stream=None):
        import torch
        T = x.shape[0]
        if dx is None:
            dx = torch.empty(T, self.K, dtype=torch.float32, device=self.device)
        tiled_linear_backward(self.handle, T, x.data_ptr(), dy.data_ptr(), dx.data_ptr(),
                              _stream_handle(stream))
        return dx

    def stats(self) -> dict:
        return tiled_linear_get_stats(self.handle)

    def reset_stats(self) -> None:
        tiled_linear_reset_stats(self.handle)

    def trace(self, backward: bool) -> list:
        """Launch and copy timeline of the last timed forward / backward call."""
        return tiled_linear_get_trace(self.handle, backward)

    def set_tile_reuse(self, enable: bool = True) -> None:
        """Let backward calls take the tiles still resident from the calls
        before them (W must not change in between)."""
        tiled_linear_set_tile_reuse(self.handle, enable)

    def set_timing(self, every: int) -> None:
        """Record per-launch / per-copy timing events on every `every`-th call."""
        tiled_linear_set_timing(self.handle, every)

    def set_stall_allowance(self, ms: float) -> None:
        """Automatic depth: host-link stall (ms) the ring is sized to ride out."""
        tiled_linear_set_stall_allowance(self.handle, ms)

    def close(self) -> int:
        st = TL_OK
        if self.handle:
            st = tiled_linear_destroy(self.handle)
            self.handle = 0
        return st

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class TiledLinearFile(TiledLinear):
    """A ``TiledLinear`` whose W and dW live in files (tile-major [N][K][M/N]
    bf16), one storage tier below host memory: reader threads stream the
    tiles into pinned host slots with direct I/O, ahead of the host->device
    copies, and writer threads store dW.  ``sync()`` waits until the dW of the
    backward calls made so far is in ``dw_path``."""

    def __init__(self, K: int, M: int, N: int, d: int, w_path: str, dw_path: str, *, host_slots: int = 4,
                 io_threads: int = 4, device=None):
        import torch
        self.K, self.M, self.N, self.d = int(K), int(M), int(N), int(d)
        self.Mi = self.M // self.N
        self.tile_major = True
        self.w_path, self.dw_path = str(w_path), str(dw_path)
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None else
                                   torch.device(device).index or 0)
        self.handle = 0
        wb = tiled_linear_workspace_bytes(self.K, self.M, self.N, self.d)
        if wb == 0:
            raise TiledLinearError(TL_ERR_INVALID, "tiled_linear_workspace_bytes",
                                   f"invalid shape K={K} M={M} N={N} d={d}")
        self.workspace = torch.empty(wb, dtype=torch.uint8, device=self.device)
        self.handle = tiled_linear_create_file(self.K, self.M, self.N, self.d, self.w_path, self.dw_path,
                                               int(host_slots), int(io_threads), self.workspace.data_ptr(), wb,
                                               self.device.index)

    def sync(self) -> None:
        """Wait for the device, then for the writers: dW is in ``dw_path``."""
        import torch
        torch.cuda.synchronize(self.device)
        tiled_linear_file_sync(self.handle)

    def file_stats(self) -> dict:
        return tiled_linear_file_stats(self.handle)


class TiledLinearChain:
    """A chain of tiled linear operators (see the chain section of
    ``include/tiled_linear.h``): operator l maps dims[l] -> dims[l+1] with its
    W_l in n_tiles[l] column tiles, tile-major in pinned host memory.  One
    ring and one prefetcher serve the whole chain."""

    def __init__(self, dims, n_tiles, d: int, w_hosts, dw_hosts, device=None):
        import torch
        self.dims = [int(v) for v in dims]
        self.n_tiles = [int(v) for v in n_tiles]
        self.L = len(self.n_tiles)
        if len(self.dims) != self.L + 1:
            raise ValueError("dims needs one entry more than n_tiles")
        self.d = int(d)
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None else
                                   torch.device(device).index or 0)
        wb = tiled_linear_chain_workspace_bytes(self.L, self.dims, self.n_tiles, self.d)
        if wb == 0:
            raise TiledLinearError(TL_ERR_INVALID, "tiled_linear_chain_workspace_bytes",
                                   f"invalid chain dims={self.dims} n_tiles={self.n_tiles} d={d}")
        self.workspace = torch.empty(wb, dtype=torch.uint8, device=self.device)
        self._w, self._dw = list(w_hosts), list(dw_hosts)
        ptr = lambda b: b.ptr if isinstance(b, PinnedBuffer) else b.data_ptr()
        self.handle = tiled_linear_chain_create(self.L, self.dims, self.n_tiles, self.d,
                                                [ptr(b) for b in self._w], [ptr(b) for b in self._dw],
                                                self.workspace.data_ptr(), wb, self.device.index)
        self._scratch = None

    def forward(self, x, ys=None, stream=None):
        """Returns the list of every operator's output (keep it for backward)."""
        import torch
        T = x.shape[0]
        if ys is None:
            ys = [torch.empty(T, self.dims[l + 1], dtype=torch.bfloat16, device=self.device)
                  for l in range(self.L)]
        tiled_linear_chain_forward(self.handle, T, x.data_ptr(), [y.data_ptr() for y in ys],
                                   _stream_handle(stream))
        return ys

    def backward(self, x, ys, dy, dx=None, stream=None):
        import torch
        T = x.shape[0]
        if dx is None:
            dx = torch.empty(T, self.dims[0], dtype=torch.float32, device=self.device)
        need = tiled_linear_chain_scratch_bytes(T, self.L, self.dims)
        if need and (self._scratch is None or self._scratch.numel() < need):
            self._scratch = torch.empty(need, dtype=torch.uint8, device=self.device)
        sp = self._scratch.data_ptr() if need else 0
        tiled_linear_chain_backward(self.handle, T, x.data_ptr(), [y.data_ptr() for y in ys] if ys else None,
                                    dy.data_ptr(), dx.data_ptr(), sp, need, _stream_handle(stream))
        return dx

    def stats(self) -> dict:
        return tiled_linear_get_stats(self.handle)

    def reset_stats(self) -> None:
        tiled_linear_reset_stats(self.handle)

    def trace(self, backward: bool) -> list:
        """Launch and copy timeline of the last timed forward / backward call."""
        return tiled_linear_get_trace(self.handle, backward)

    def set_tile_reuse(self, enable: bool = True) -> None:
        tiled_linear_set_tile_reuse(self.handle, enable)

    def close(self) -> int:
        st = TL_OK
        if self.handle:
            st = tiled_linear_destroy(self.handle)
            self.handle = 0
        return st

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HostAdam:
    """The Adam step on the host CPU for a ``TiledLinear`` or
    ``TiledLinearChain`` (see the optimizer section of
    ``include/tiled_linear.h``).  Keeps fp32 master weights (initialised from
    the op's host W), first and second moments, and optionally an fp32
    gradient accumulator, in the layout of each operator's host W.  After a
    backward call, ``step()`` (or ``accumulate()``) returns at once; the update
    overlaps the GPU, and the op's next calls wait for the tiles they read."""

    def __init__(self, op, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, threads=0,
                 accumulate=False):
        import torch
        self.op = op
        self.handle = 0
        if getattr(op, "_w", None) is None:
            raise TiledLinearError(TL_ERR_INVALID, "HostAdam", "the host optimizer needs W and dW in host memory")
        ws = op._w if isinstance(op._w, list) else [op._w]
        hosts = [b.tensor if isinstance(b, PinnedBuffer) else b for b in ws]
        self.master = [h.view(-1).float() for h in hosts]
        self.m = [torch.zeros_like(a) for a in self.master]
        self.v = [torch.zeros_like(a) for a in self.master]
        self.acc = [torch.zeros_like(a) for a in self.master] if accumulate else None
        self.cfg = adam_config(lr, beta1, beta2, eps, weight_decay, threads)
        ptr = lambda ts: [t.data_ptr() for t in ts]
        self.handle = tiled_linear_optimizer_create(op.handle, self.cfg, ptr(self.master), ptr(self.m), ptr(self.v),
                                                    ptr(self.acc) if self.acc else None)

    def step(self) -> None:
        tiled_linear_optimizer_step(self.handle, self.op.handle)

    def accumulate(self) -> None:
        tiled_linear_optimizer_accumulate(self.handle, self.op.handle)

    def wait(self) -> None:
        tiled_linear_optimizer_wait(self.handle, self.op.handle)

    def stats(self) -> dict:
        steps, busy = tiled_linear_optimizer_stats(self.handle)
        return {"steps": steps, "busy_seconds": busy}

    def close(self) -> int:
        st = TL_OK
        if self.handle:
            st = tiled_linear_optimizer_destroy(self.handle)
            self.handle = 0
        return st

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --- operators around the product ---------------------------------------------
# Functions of torch tensors: device-resident, enqueued on the current stream,
# with outputs and workspaces from torch's allocator on that stream.  They take
# no gradient through autograd: each backward is a function of its own.  Inputs are
# matrices of contiguous rows, any distance apart that keeps them from overlapping.
# Results of the 8-bit products and of orthogonalize have rows on 16-byte
# boundaries: where the width is no multiple of 8 they are views with gaps between
# the rows (.contiguous() packs them).

TL_TYPE_BF16, TL_TYPE_F16, TL_TYPE_F32 = range(3)
_torch = None
_types = {}


def _t():
    """torch, imported by the first call that needs it."""
    global _torch
    if _torch is None:
        import torch
        _types.update({torch.bfloat16: TL_TYPE_BF16, torch.float16: TL_TYPE_F16, torch.float32: TL_TYPE_F32})
        _torch = torch
    return _torch


def _refuse(where: str, why: str):
    raise TiledLinearError(TL_ERR_INVALID, where, why)


def _type_of(t, where: str) -> int:
    got = _types.get(t.dtype)
    if got is None:
        _refuse(where, f"dtype {t.dtype}: bfloat16, float16 or float32 is wanted")
    return got


def _ld(t, where: str, name: str) -> int:
    """Leading dimension of a device matrix whose rows are contiguous (that of
    a single row is its length)."""
    if not t.is_cuda:
        _refuse(where, f"{name} is not on a CUDA device")
    if t.dim() != 2:
        _refuse(where, f"{name} has {t.dim()} dimensions: a matrix is wanted")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        _refuse(where, f"the rows of {name} are not contiguous")
    if rows > 1 and ld < cols:
        _refuse(where, f"the rows of {name} overlap")
    return ld if rows > 1 else cols


def _vector(t, n: int, device, where: str, name: str) -> None:
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1) or t.device != device:
        _refuse(where, f"{name} must be a contiguous vector of {n} on the matrix's device")


def _stream_of(device, where: str) -> int:
    """The current stream, which is one of `device`."""
    torch = _torch
    if torch.cuda.current_device() != device.index:
        _refuse(where, f"the tensors are on {device}: make it the current device")
    return torch._C._cuda_getCurrentRawStream(device.index)


_err_words = {}


class _Word:
    """One int32 at an address, as torch takes memory that is not its own."""

    def __init__(self, address: int):
        self.__cuda_array_interface__ = {"shape": (1,), "typestr": "<i4", "data": (address, False), "version": 2}


def _err_word(device) -> int:
    """Device address of the error word that this process's calls on `device` share:
    the library's own, so that a first call may be captured in a graph."""
    got = _err_words.get(device.index)
    if got is None:
        with _torch.cuda.device(device):
            at = tiled_linear_operator_error_word()
            word = _torch.as_tensor(_Word(at), device=device)
        got = _err_words.setdefault(device.index, (word, at))
    return got[1]


def check_operators(device=None) -> None:
    """Wait for the device and raise TL_ERR_TIMEOUT if a kernel of the functions
    below has given up one of its bounded waits since the last check.  The results of
    one call at least since then are not valid, and which is not known."""
    torch = _t()
    index = None if device is None else torch.device(device).index
    if index is None:  # "cuda" is the current device, too
        index = torch.cuda.current_device()
    if index in _err_words:
        torch.cuda.synchronize(index)
        bits = int(_err_words[index][0][0])
        if bits:
            _err_words[index][0].zero_()
            torch.cuda.synchronize(index)  # before any stream's next call
            raise TiledLinearError(TL_ERR_TIMEOUT, "check_operators", f"error word {bits:#x}")


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """(y, mean, rstd): layer norm over the columns of x [rows, cols] (bf16, fp16 or
    fp32; any stride of rows that do not overlap).  weight, bias: [cols], both of one of those types, or
    None for ones / zeros.  mean and rstd are fp32 [rows], for the backward."""
    torch, where = _t(), "layer_norm"
    ldx, (rows, cols), device = _ld(x, where, "x"), x.shape, x.device
    ptype, wp, bp = TL_TYPE_F32, None, None
    if weight is not None:
        _vector(weight, cols, device, where, "weight")
        ptype, wp = _type_of(weight, where), weight.data_ptr()
    if bias is not None:
        _vector(bias, cols, device, where, "bias")
        if weight is not None and weight.dtype != bias.dtype:
            _refuse(where, "weight and bias differ in dtype")
        ptype, bp = _type_of(bias, where), bias.data_ptr()
    kind, stream = _type_of(x, where), _stream_of(device, where)
    y = torch.empty((rows, cols), dtype=x.dtype, device=device)
    mean = torch.empty(rows, dtype=torch.float32, device=device)
    rstd = torch.empty(rows, dtype=torch.float32, device=device)
    tiled_linear_norm_forward(rows, cols, kind, x.data_ptr(), ldx, ptype, wp, bp, eps, y.data_ptr(), cols,
                              mean.data_ptr(), rstd.data_ptr(), _err_word(device), stream)
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias) of ``layer_norm``: dx like x, dweight and dbias fp32
    [cols] (the derivative by a weight of ones where there is none)."""
    torch, where = _t(), "layer_norm_backward"
    ldx, (rows, cols), device = _ld(x, where, "x"), x.shape, x.device
    lddy = _ld(dy, where, "dy")
    if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != device:
        _refuse(where, "dy and x differ in shape, dtype or device")
    ptype, wp = TL_TYPE_F32, None
    if weight is not None:
        _vector(weight, cols, device, where, "weight")
        ptype, wp = _type_of(weight, where), weight.data_ptr()
    for v, name in ((mean, "mean"), (rstd, "rstd")):
        _vector(v, rows, device, where, name)
        if v.dtype != torch.float32:
            _refuse(where, f"{name} must be float32")
    kind, stream = _type_of(x, where), _stream_of(device, where)
    dx = torch.empty((rows, cols), dtype=x.dtype, device=device)
    dweight = torch.empty(cols, dtype=torch.float32, device=device)
    dbias = torch.empty(cols, dtype=torch.float32, device=device)
    need = tiled_linear_norm_backward_workspace_bytes(rows, cols)
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    tiled_linear_norm_backward(rows, cols, kind, dy.data_ptr(), lddy, x.data_ptr(), ldx, mean.data_ptr(),
                               rstd.data_ptr(), ptype, wp, dx.data_ptr(), cols, dweight.data_ptr(), dbias.data_ptr(),
                               ws.data_ptr(), need, _err_word(device), stream)
    return dx, dweight, dbias


TL_FP8_E4M3, TL_FP8_E5M2 = range(2)
FP8_BLOCK = 128


def _up(n: int, to: int) -> int:
    return -(-n // to) * to


def _fp8_format(t, where: str, name: str) -> int:
    torch = _torch
    if t.dtype == torch.float8_e4m3fn:
        return TL_FP8_E4M3
    if t.dtype == torch.float8_e5m2:
        return TL_FP8_E5M2
    _refuse(where, f"{name} has dtype {t.dtype}: float8_e4m3fn or float8_e5m2 is wanted")


def _fp8_scales(rows: int, cols: int, form: str) -> tuple:
    """Shape of a form's scales."""
    if form == "row":
        return -(-cols // (4 * FP8_BLOCK)), rows, 4
    if form == "col":
        return -(-rows // (4 * FP8_BLOCK)), cols, 4
    if form == "tile":
        return -(-rows // FP8_BLOCK), -(-cols // FP8_BLOCK)
    _refuse("fp8_quantize", f"form {form!r}: 'row', 'col' or 'tile' is wanted")


def fp8_quantize(x, *forms: str, format: str = "e4m3"):
    """x [rows, cols] (bf16, fp16 or fp32) in 8 bits: (q, scale) for one form, a
    tuple of such pairs for several, all from one reading of x.

    forms: "row" (a scale for 128 columns of a row), "col" (128 rows of a column),
    "tile" (128 x 128).  q: float8_e4m3fn or (format="e5m2") float8_e5m2
    [rows, cols], rows on 16-byte boundaries; scale: uint8, q stands for
    q * 2^(scale - 127).  A tile's scale is scale[row // 128, col // 128]; the row
    form's is scale[col // 512, row, col // 128 % 4] and the col form's
    scale[row // 512, col, row // 128 % 4], as the products take them."""
    torch, where = _t(), "fp8_quantize"
    ldx, (rows, cols), device = _ld(x, where, "x"), x.shape, x.device
    kind, stream = _type_of(x, where), _stream_of(device, where)
    if cols < 1 or not forms or len(set(forms)) < len(forms):
        _refuse(where, "x needs a column, and at least one form, each named once")
    if format not in ("e4m3", "e5m2"):
        _refuse(where, f"format {format!r}: 'e4m3' or 'e5m2' is wanted")
    dtype = torch.float8_e4m3fn if format == "e4m3" else torch.float8_e5m2
    ldq, out, args = _up(cols, 16), [], {}
    for form in forms:
        scale = torch.empty(_fp8_scales(rows, cols, form), dtype=torch.uint8, device=device)
        q = torch.empty((rows, ldq), dtype=dtype, device=device)
        args[form] = (q.data_ptr(), ldq, scale.data_ptr())
        out.append((q if ldq == cols else q[:, :cols], scale))
    none = (None, 0, None)
    tiled_linear_fp8_quantize(rows, cols, kind, x.data_ptr(), ldx, 0 if format == "e4m3" else 1,
                              *args.get("row", none), *args.get("col", none), *args.get("tile", none), stream)
    return out[0] if len(forms) == 1 else tuple(out)


def _fp8_operand(q, scale, form: str, where: str, name: str):
    """(format, pointer, ld, scale pointer) of a matrix in 8 bits."""
    fmt, ld = _fp8_format(q, where, name), _ld(q, where, name)
    rows, cols = q.shape
    shape = _fp8_scales(rows, cols, form)
    if scale.dtype != _torch.uint8 or scale.shape != shape or scale.device != q.device or not scale.is_contiguous():
        _refuse(where, f"the scales of {name} must be contiguous uint8 {list(shape)} on its device")
    if rows == 1:
        ld = _up(cols, 16)  # one row: there is no second for it to lead to
    return fmt, q.data_ptr(), ld, scale.data_ptr()


def _fp8_result(x, rows: int, cols: int):
    ld = _up(cols, 8)
    out = _torch.empty((rows, ld), dtype=_torch.bfloat16, device=x.device)
    return (out if ld == cols else out[:, :cols]), ld


def _weight_shape(q, where: str):
    if q.dim() != 2 or 0 in q.shape:
        _refuse(where, "the weight must be a matrix [K, n] with K, n >= 1")
    return q.shape


def fp8_matmul(x, w):
    """y [T, n] bf16 = x [T, K] . w [K, n], x = (q, scale) in the row form and
    w = (q, scale) in the tile form."""
    _t()
    where, (xq, xs), (wq, ws) = "fp8_matmul", x, w
    K, n = _weight_shape(wq, where)
    if xq.dim() != 2 or xq.shape[1] != K or xq.device != wq.device:
        _refuse(where, "x and the weight do not fit each other")
    T = xq.shape[0]
    y, ldy = _fp8_result(xq, T, n)
    tiled_linear_fp8_gemm_forward(T, K, n, *_fp8_operand(xq, xs, "row", where, "x"),
                                  *_fp8_operand(wq, ws, "tile", where, "the weight"), y.data_ptr(), ldy,
                                  _err_word(xq.device), _stream_of(xq.device, where))
    return y


def fp8_matmul_dx(dy, w):
    """dx [T, K] bf16 = dy [T, n] . w [K, n]^T, dy in the row form, w in the tile form."""
    _t()
    where, (dyq, dys), (wq, ws) = "fp8_matmul_dx", dy, w
    K, n = _weight_shape(wq, where)
    if dyq.dim() != 2 or dyq.shape[1] != n or dyq.device != wq.device:
        _refuse(where, "dy and the weight do not fit each other")
    T = dyq.shape[0]
    dx, lddx = _fp8_result(dyq, T, K)
    tiled_linear_fp8_gemm_dx(T, K, n, *_fp8_operand(dyq, dys, "row", where, "dy"),
                             *_fp8_operand(wq, ws, "tile", where, "the weight"), dx.data_ptr(), lddx,
                             _err_word(dyq.device), _stream_of(dyq.device, where))
    return dx


def fp8_matmul_dw(x, dy):
    """dw [K, n] bf16 = x [T, K]^T . dy [T, n], both in the col form."""
    _t()
    where, (xq, xs), (dyq, dys) = "fp8_matmul_dw", x, dy
    if xq.dim() != 2 or dyq.dim() != 2 or xq.shape[0] != dyq.shape[0] or xq.device != dyq.device \
            or 0 in (xq.shape[1], dyq.shape[1]):
        _refuse(where, "x and dy do not fit each other")
    (T, K), n = xq.shape, dyq.shape[1]
    dw, lddw = _fp8_result(xq, K, n)
    tiled_linear_fp8_gemm_dw(T, K, n, *_fp8_operand(xq, xs, "col", where, "x"),
                             *_fp8_operand(dyq, dys, "col", where, "dy"), dw.data_ptr(), lddw, _err_word(xq.device),
                             _stream_of(xq.device, where))
    return dw


def fp8_linear(x, wq, ws):
    """y [T, n] bf16 = x [T, K] . w with w in 8 bits (``fp8_quantize(w, "tile")``);
    x (bf16, fp16 or fp32) is quantised on the way, with a scale for each 128
    columns of a row.  (y's rows have gaps where n is no multiple of 8, as dx's and dw's.)"""
    torch, where = _t(), "fp8_linear"
    ldx, T, device, (K, n) = _ld(x, where, "x"), x.shape[0], x.device, _weight_shape(wq, where)
    if x.shape[1] != K or device != wq.device:
        _refuse(where, "x and the weight do not fit each other")
    kind, stream, w = _type_of(x, where), _stream_of(device, where), _fp8_operand(wq, ws, "tile", where, "the weight")
    y, ldy = _fp8_result(x, T, n)
    need = tiled_linear_fp8_linear_workspace_bytes(T, K, n)
    work = torch.empty(need, dtype=torch.uint8, device=device)
    tiled_linear_fp8_linear(T, K, n, kind, x.data_ptr(), ldx, *w, y.data_ptr(), ldy, work.data_ptr(), need,
                            _err_word(device), stream)
    return y


def fp8_linear_backward(x, dy, wq, ws):
    """(dx [T, K], dw [K, n]) bf16 of ``fp8_linear`` for dy [T, n], as products in 8
    bits: dy . w^T with dy's rows in blocks of 128, x^T . dy with blocks of 128
    tokens.  (The derivative passes through the rounding to 8 bits.)"""
    torch, where = _t(), "fp8_linear_backward"
    ldx, lddy, T, device, (K, n) = _ld(x, where, "x"), _ld(dy, where, "dy"), x.shape[0], x.device, _weight_shape(wq, where)
    if x.shape[1] != K or dy.shape != (T, n) or dy.dtype != x.dtype or device != wq.device or dy.device != device:
        _refuse(where, "x, dy and the weight do not fit each other")
    kind, stream, w = _type_of(x, where), _stream_of(device, where), _fp8_operand(wq, ws, "tile", where, "the weight")
    (dx, lddx), (dw, lddw) = _fp8_result(x, T, K), _fp8_result(x, K, n)
    need = tiled_linear_fp8_linear_backward_workspace_bytes(T, K, n)
    work = torch.empty(need, dtype=torch.uint8, device=device)
    tiled_linear_fp8_linear_backward(T, K, n, kind, x.data_ptr(), ldx, dy.data_ptr(), lddy, *w, dx.data_ptr(), lddx,
                                     dw.data_ptr(), lddw, work.data_ptr(), need, _err_word(device), stream)
    return dx, dw


def orthogonalize(g, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, scale: float = 1.0):
    """bf16 scale * X, X the matrix g (or each matrix of g [batch, rows, cols]; bf16,
    fp16 or fp32) after `steps` Newton-Schulz steps X = a X + (b P + c P^2) X,
    P = X X^T, from g / (|g|_F + eps): its singular values drawn to about one.  (The
    rows of the result have gaps where cols is no multiple of 8.)"""
    torch, where = _t(), "orthogonalize"
    if not g.is_cuda or g.dim() not in (2, 3):
        _refuse(where, "g must be a matrix or a stack of matrices on a CUDA device")
    device = g.device
    kind, stream = _type_of(g, where), _stream_of(device, where)
    stack = g if g.dim() == 3 else g.unsqueeze(0)
    batch, rows, cols = stack.shape
    if rows < 1 or cols < 1:
        _refuse(where, "the matrices have no elements")
    apart, ldg, step = stack.stride()
    if (cols > 1 and step != 1) or (rows > 1 and ldg < cols):
        _refuse(where, "the rows of g are not contiguous")
    ldg = ldg if rows > 1 else cols
    ldo = _up(cols, 8)
    out = torch.empty((batch, rows, ldo), dtype=torch.bfloat16, device=device)
    need = tiled_linear_orthogonalize_workspace_bytes(batch, rows, cols)
    work = torch.empty(need, dtype=torch.uint8, device=device)
    a, b, c = coefficients
    tiled_linear_orthogonalize(batch, rows, cols, kind, stack.data_ptr(), ldg, apart if batch > 1 else 0, steps, a, b, c,
                               eps, scale, out.data_ptr(), ldo, rows * ldo, work.data_ptr(), need, _err_word(device),
                               stream)
    out = out if ldo == cols else out[:, :, :cols]
    return out if g.dim() == 3 else out[0]


# --- a linear layer whose weight depends on the row ----------------------------
# The router's experts and the adapters of many requests.  Functions of torch tensors
# like the ones above.  Matrices of bf16 or fp16 are taken as they lie where their
# rows start on 16-byte boundaries, and are copied into such rows first where they
# do not (a weight that is used often is better kept in them).  Results whose width is no
# multiple of 8 are views with gaps between the rows.

def _half_type(t, where: str, name: str) -> int:
    kind = _types.get(t.dtype)
    if kind not in (TL_TYPE_BF16, TL_TYPE_F16):
        _refuse(where, f"{name} has dtype {t.dtype}: bfloat16 or float16 is wanted")
    return kind


def _int32(t, shape, device, where: str, name: str) -> int:
    if t.dtype != _torch.int32 or tuple(t.shape) != tuple(shape) or t.device != device or not t.is_contiguous():
        _refuse(where, f"{name} must be contiguous int32 {list(shape)} on the matrix's device")
    return t.data_ptr()


def _matrix16(t, where: str, name: str):
    """(tensor to keep, pointer, ld) of a matrix in rows on 16-byte boundaries."""
    ld = _ld(t, where, name)
    rows, cols = t.shape
    if rows <= 1:
        ld = _up(cols, 8)
    if t.data_ptr() % 16 or ld % 8:
        ld = _up(cols, 8)
        kept = _torch.empty((rows, ld), dtype=t.dtype, device=t.device)
        kept[:, :cols].copy_(t)
        t = kept
    return t, t.data_ptr(), ld


def _stack16(t, where: str, name: str):
    """(tensor to keep, pointer, ld, distance) of a stack of matrices, likewise."""
    if not t.is_cuda or t.dim() != 3 or 0 in t.shape:
        _refuse(where, f"{name} must be a stack of matrices with elements on a CUDA device")
    count, rows, cols = t.shape
    apart, ld, step = t.stride()
    if cols > 1 and step != 1:
        _refuse(where, f"the rows of {name} are not contiguous")
    if rows == 1:
        ld = _up(cols, 8)
    if count == 1:
        apart = rows * ld
    if ld < cols or apart < (rows - 1) * ld + cols:
        _refuse(where, f"the rows or matrices of {name} overlap")
    if t.data_ptr() % 16 or ld % 8 or apart % 8:
        ld = _up(cols, 8)
        kept = _torch.empty((count, rows, ld), dtype=t.dtype, device=t.device)
        kept[:, :, :cols].copy_(t)
        t, apart = kept, rows * ld
    return t, t.data_ptr(), ld, apart


def _result16(shape, like):
    """An empty result in rows on 16-byte boundaries, and its ld."""
    ld = _up(shape[-1], 8)
    out = _torch.empty((*shape[:-1], ld), dtype=like.dtype, device=like.device)
    return (out if ld == shape[-1] else out[..., :shape[-1]]), ld


def _grouping(T: int, k: int, groups: int, device):
    """Empty slots, rows and offsets, and the workspace of the grouping."""
    torch = _torch
    need = tiled_linear_route_workspace_bytes(T, k, groups)
    return (torch.empty((T, k), dtype=torch.int32, device=device), torch.empty(T * k, dtype=torch.int32, device=device),
            torch.empty(groups + 1, dtype=torch.int32, device=device), torch.empty(need, dtype=torch.uint8, device=device), need)


def group_rows(ids, groups: int):
    """(slots, rows, offsets): the order by group of the entries ids [T, k] (int32; an id
    outside 0..groups-1 is of no group).  Places offsets[g]..offsets[g + 1] - 1 hold
    group g's entries in the order they have in ids, rows[place] is an entry's t and
    slots [T, k] its place (-1 of no group; those entries' rows come last)."""
    where, _ = "group_rows", _t()
    if not ids.is_cuda or ids.dim() != 2:
        _refuse(where, "ids must be a matrix on a CUDA device")
    (T, k), device = ids.shape, ids.device
    if groups < 1:
        _refuse(where, "groups must be 1..1024")
    ip, stream = _int32(ids, ids.shape, device, where, "ids"), _stream_of(device, where)
    slots, rows, offsets, work, need = _grouping(T, k, groups, device)
    tiled_linear_group_rows(T, k, groups, ip, slots.data_ptr(), rows.data_ptr(), offsets.data_ptr(), work.data_ptr(), need, stream)
    return slots, rows, offsets


def route(logits, k: int, normalize: bool = True):
    """(weights, ids, slots, rows, offsets): the k experts with the largest of each token's
    logits [T, experts] (bf16, fp16 or fp32), largest first, the lowest index first among
    equals; their weights (fp32 [T, k]), a softmax over the k (normalize) or over all
    experts; and the entries' order by expert as ``group_rows`` gives it.  A logit of
    -inf or NaN is never chosen: where too few are left, ids are -1 and weights 0."""
    torch, where = _t(), "route"
    ld, (T, experts), device = _ld(logits, where, "logits"), logits.shape, logits.device
    kind, stream = _type_of(logits, where), _stream_of(device, where)
    if not 1 <= k <= experts:
        _refuse(where, f"k must be 1..{experts}")
    weights = torch.empty((T, k), dtype=torch.float32, device=device)
    ids = torch.empty((T, k), dtype=torch.int32, device=device)
    slots, rows, offsets, work, need = _grouping(T, k, experts, device)
    tiled_linear_route(T, experts, k, kind, logits.data_ptr(), ld, int(normalize), weights.data_ptr(), ids.data_ptr(),
                       slots.data_ptr(), rows.data_ptr(), offsets.data_ptr(), work.data_ptr(), need, stream)
    return weights, ids, slots, rows, offsets


def route_backward(dweights, logits, ids, normalize: bool = True):
    """dlogits (like logits) of ``route``'s weights for dweights [T, k] (fp32), with its
    ids [T, k]; the choice itself has no derivative."""
    torch, where = _t(), "route_backward"
    ld, (T, experts), device = _ld(logits, where, "logits"), logits.shape, logits.device
    kind, stream = _type_of(logits, where), _stream_of(device, where)
    if ids.dim() != 2 or ids.shape[0] != T:
        _refuse(where, "ids and logits do not fit each other")
    k, ip = ids.shape[1], _int32(ids, ids.shape, device, where, "ids")
    if dweights.shape != ids.shape or dweights.dtype != torch.float32 or dweights.device != device or not dweights.is_contiguous():
        _refuse(where, "dweights must be contiguous float32, as ids")
    out = torch.empty((T, experts), dtype=logits.dtype, device=device)
    tiled_linear_route_backward(T, experts, k, kind, logits.data_ptr(), ld, ip, dweights.data_ptr(), int(normalize), out.data_ptr(),
                                experts, stream)
    return out


def _combine_args(slots, weights, device, where: str):
    if slots.dim() != 2:
        _refuse(where, "slots must be a matrix")
    sp, wp = _int32(slots, slots.shape, device, where, "slots"), None
    if weights is not None:
        if weights.shape != slots.shape or weights.dtype != _torch.float32 or weights.device != device or not weights.is_contiguous():
            _refuse(where, "weights must be contiguous float32, as slots")
        wp = weights.data_ptr()
    return sp, wp


def combine(y, slots, weights=None):
    """out [T, cols] = sum over j of weights[t, j] y[slots[t, j]] for y [rows, cols] (bf16,
    fp16 or fp32), slots [T, k] as ``route`` gives them (-1 adds nothing) and weights
    fp32 [T, k], None for ones (which gives the gradient of rows picked up by ``rows``)."""
    torch, where = _t(), "combine"
    ldy, (rows, cols), device = _ld(y, where, "y"), y.shape, y.device
    kind, stream = _type_of(y, where), _stream_of(device, where)
    sp, wp = _combine_args(slots, weights, device, where)
    T, k = slots.shape
    out = torch.empty((T, cols), dtype=y.dtype, device=device)
    tiled_linear_combine(T, k, cols, rows, kind, y.data_ptr(), ldy, sp, wp, out.data_ptr(), cols, stream)
    return out


def combine_backward(dout, slots, y=None, weights=None):
    """(dy, dweights) of ``combine`` for dout [T, cols]: dy [rows, cols], rows as y's (T k without
    y), of which those that no slot names are left unset; dweights fp32 [T, k], None without y."""
    torch, where = _t(), "combine_backward"
    ldd, (T, cols), device = _ld(dout, where, "dout"), dout.shape, dout.device
    kind, stream = _type_of(dout, where), _stream_of(device, where)
    sp, wp = _combine_args(slots, weights, device, where)
    if slots.shape[0] != T:
        _refuse(where, "slots and dout do not fit each other")
    k, yp, ldy, dweights = slots.shape[1], None, 0, None
    rows = T * k
    if y is not None:
        ldy, rows = _ld(y, where, "y"), y.shape[0]
        if y.shape[1] != cols or y.dtype != dout.dtype or y.device != device:
            _refuse(where, "y and dout differ in columns, dtype or device")
        yp, dweights = y.data_ptr(), torch.empty((T, k), dtype=torch.float32, device=device)
    dy = torch.empty((rows, cols), dtype=dout.dtype, device=device)
    tiled_linear_combine_backward(T, k, cols, rows, kind, dout.data_ptr(), ldd, sp, yp, ldy, wp, dy.data_ptr(), cols,
                                  None if dweights is None else dweights.data_ptr(), stream)
    return dy, dweights


def _grouped_args(x, w, offsets, rows, where: str):
    kind, (xk, xp, ldx) = _half_type(x, where, "x"), _matrix16(x, where, "x")
    wk, wp, ldw, apart = _stack16(w, where, "the weight")
    groups, K, n = w.shape
    if x.shape[1] != K or w.dtype != x.dtype or w.device != x.device:
        _refuse(where, "x and the weight do not fit each other")
    op, rp, R = _int32(offsets, (groups + 1,), x.device, where, "offsets"), None, x.shape[0]
    if rows is not None:
        R = rows.shape[0] if rows.dim() == 1 else -1
        rp = _int32(rows, (R,), x.device, where, "rows")
        if R > 0 and x.shape[0] == 0:
            _refuse(where, "x has no rows")
    return kind, (xk, wk), (xp, ldx, x.shape[0], rp), (wp, ldw, apart), op, (R, K, n, groups)


def _grouped_work(R: int, K: int, rows, device):
    """The workspace for sorted rows and its size, where there are rows to sort."""
    if rows is None:
        return None, None, 0
    need = tiled_linear_grouped_workspace_bytes(R, K)
    work = _torch.empty(need, dtype=_torch.uint8, device=device)
    return work, work.data_ptr(), need


def grouped_linear(x, w, offsets, rows=None):
    """y [R, n]: y[p] = x[p] . w[g] for the places p = offsets[g]..offsets[g + 1] - 1 of each
    group g, with w [groups, K, n] and x [R, K] (both bf16 or fp16), or x[rows[p]] for
    x [tokens, K] and rows [R] (``route``'s).  offsets: int32 [groups + 1] on the
    device, groups of any size; rows of y in no group are left unset."""
    where, _ = "grouped_linear", _t()
    kind, kept, xa, wa, op, (R, K, n, groups) = _grouped_args(x, w, offsets, rows, where)
    stream = _stream_of(x.device, where)
    (y, ldy), (work, *ws) = _result16((R, n), x), _grouped_work(R, K, rows, x.device)
    tiled_linear_grouped_forward(R, K, n, groups, kind, *xa, *wa, op, y.data_ptr(), ldy, *ws, _err_word(x.device), stream)
    return y


def grouped_linear_backward(x, dy, w, offsets, rows=None):
    """(dx [R, K], dw [groups, K, n]) of ``grouped_linear`` for dy [R, n]: dx[p] = dy[p] . w[g]^T
    (with rows, the gradient by x is ``combine(dx, slots)``), dw[g] = the sum over g's
    places of x^T dy, zeros where there are none."""
    where, _ = "grouped_linear_backward", _t()
    kind, kept, xa, wa, op, (R, K, n, groups) = _grouped_args(x, w, offsets, rows, where)
    dk, dp, lddy = _matrix16(dy, where, "dy")
    if dy.shape != (R, n) or dy.dtype != x.dtype or dy.device != x.device:
        _refuse(where, "x, dy and the weight do not fit each other")
    stream, err = _stream_of(x.device, where), _err_word(x.device)
    (dx, lddx), (dw, lddw), (work, *ws) = _result16((R, K), x), _result16((groups, K, n), x), _grouped_work(R, K, rows, x.device)
    tiled_linear_grouped_dx(R, K, n, groups, kind, dp, lddy, *wa, op, dx.data_ptr(), lddx, err, stream)
    tiled_linear_grouped_dw(R, K, n, groups, kind, *xa, dp, lddy, op, dw.data_ptr(), lddw, K * lddw, *ws, err, stream)
    return dx, dw


def _adapter_args(x, a, b, ids, scale, where: str):
    kind, (xk, xp, ldx) = _half_type(x, where, "x"), _matrix16(x, where, "x")
    (ak, ap, lda, a_apart), (bk, bp, ldb, b_apart) = _stack16(a, where, "a"), _stack16(b, where, "b")
    adapters, K, r = a.shape
    if x.shape[1] != K or b.shape[:2] != (adapters, r) or any(t.dtype != x.dtype or t.device != x.device for t in (a, b)):
        _refuse(where, "x, a and b do not fit each other")
    ip, sp, s = _int32(ids, (x.shape[0],), x.device, where, "ids"), None, 1.0
    if _torch.is_tensor(scale):
        _vector(scale, adapters, x.device, where, "scale")
        if scale.dtype != _torch.float32:
            _refuse(where, "scale must be float32")
        sp = scale.data_ptr()
    else:
        s = float(scale)
    return kind, (xk, ak, bk), (xp, ldx), (ap, lda, a_apart), (bp, ldb, b_apart), ip, (sp, s), (x.shape[0], K, b.shape[2], r, adapters)


def _adapter_base(base, shape, like, where: str):
    if base is None:
        return TL_TYPE_F32, None, 0
    if base.shape != shape or base.device != like.device or base.dtype not in (like.dtype, _torch.float32):
        _refuse(where, f"base must be {list(shape)} of x's dtype or float32 on its device")
    return _type_of(base, where), base.data_ptr(), _ld(base, where, "base")


def _adapter_work(T: int, r: int, adapters: int, device):
    need = tiled_linear_adapter_workspace_bytes(T, r, adapters)
    return _torch.empty(need, dtype=_torch.uint8, device=device), need


def adapter_linear(x, a, b, ids, base=None, scale=1.0):
    """(y, h): y[t] = base[t] + s h[t] . b[ids[t]], h[t] = x[t] . a[ids[t]], for x [T, K], a
    [adapters, K, r] and b [adapters, r, n] (bf16 or fp16, r up to 128), ids int32 [T] on
    the device (one outside 0..adapters-1: no adapter, h = 0 and y = base).  base
    [T, n] (x's dtype or fp32; None for zeros) is the shared projection's result,
    streamed, in 8 bits or any other; scale: one number, or fp32 [adapters].  h, kept
    for the backward, is rounded to x's dtype (infinite where it leaves it), y is made
    from the one before that."""
    where, _ = "adapter_linear", _t()
    kind, kept, xa, aa, ba, ip, sa, (T, K, n, r, adapters) = _adapter_args(x, a, b, ids, scale, where)
    bt, bp, ldbase = _adapter_base(base, (T, n), x, where)
    stream, (work, need) = _stream_of(x.device, where), _adapter_work(T, r, adapters, x.device)
    (y, ldy), (h, ldh) = _result16((T, n), x), _result16((T, r), x)
    tiled_linear_adapter_forward(T, K, n, r, adapters, kind, *xa, *aa, *ba, ip, *sa, bt, bp, ldbase, y.data_ptr(), ldy,
                                 h.data_ptr(), ldh, work.data_ptr(), need, _err_word(x.device), stream)
    return y, h


def adapter_linear_backward(x, h, dy, a, b, ids, base=None, scale=1.0):
    """(dx [T, K], da, db) of ``adapter_linear`` for dy [T, n]: with dh = s dy . b^T, dx = base +
    dh . a^T (base [T, K], x's dtype or fp32: the gradient through the shared projection),
    da and db like a and b, zeros for adapters without rows."""
    where, _ = "adapter_linear_backward", _t()
    kind, kept, xa, aa, ba, ip, sa, (T, K, n, r, adapters) = _adapter_args(x, a, b, ids, scale, where)
    (hk, hp, ldh), (dk, dp, lddy) = _matrix16(h, where, "h"), _matrix16(dy, where, "dy")
    if h.shape != (T, r) or dy.shape != (T, n) or any(t.dtype != x.dtype or t.device != x.device for t in (h, dy)):
        _refuse(where, "x, h and dy do not fit each other")
    bt, bp, ldbase = _adapter_base(base, (T, K), x, where)
    stream, (work, need) = _stream_of(x.device, where), _adapter_work(T, r, adapters, x.device)
    (dx, lddx), (da, ldda), (db, lddb) = _result16((T, K), x), _result16((adapters, K, r), x), _result16((adapters, r, n), x)
    tiled_linear_adapter_backward(T, K, n, r, adapters, kind, *xa, hp, ldh, dp, lddy, *aa, *ba, ip, *sa, bt, bp, ldbase,
                                  dx.data_ptr(), lddx, da.data_ptr(), ldda, K * ldda, db.data_ptr(), lddb, r * lddb,
                                  work.data_ptr(), need, _err_word(x.device), stream)
    return dx, da, db
