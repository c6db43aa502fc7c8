"""Submanifold sparse convolution on AMD MI355X (gfx950).

A thin Python binding over the C ABI of ``libspconv.so`` (declared in
``include/spconv.h``).  It only marshals arguments: PyTorch tensors supply
device memory and the current HIP stream; every step of the map build and the
forward runs in the library's HIP kernels.  There is no CPU fallback: if the
library is missing, every entry point raises.

The raw C functions are exposed under their C names (``spconv_build_map``,
``spconv_forward``, ...) through :func:`lib`; :func:`build_map` and
:func:`forward` wrap them for torch tensors.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# SPCONV_LIB_PATH names another build of the same library (the tests' host-only
# sanitizer build); by default the in-tree libspconv.so.
LIB_PATH = os.environ.get("SPCONV_LIB_PATH") or os.path.join(_HERE, "libspconv.so")

STATUS = {
    0: "SPCONV_OK",
    1: "SPCONV_ERR_INVALID_ARG",
    2: "SPCONV_ERR_DUPLICATE_COORD",
    3: "SPCONV_ERR_COORD_RANGE",
    4: "SPCONV_ERR_UNSUPPORTED",
    5: "SPCONV_ERR_OUT_OF_MEMORY",
    6: "SPCONV_ERR_DEVICE",
}
DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2}

# Every symbol include/spconv.h declares.
EXPORTED = (
    "spconv_abi_version", "spconv_build_map", "spconv_build_map_async", "spconv_map_wait",
    "spconv_map_info", "spconv_map_counts", "spconv_map_lists", "spconv_forward",
    "spconv_forward_noalloc", "spconv_backward_data", "spconv_backward_weights", "spconv_build_map_strided",
    "spconv_map_transpose", "spconv_map_geometry", "spconv_map_out_coords", "spconv_group_plan", "spconv_group_plan_counts",
    "spconv_forward_grouped", "spconv_select_dataflow", "spconv_map_free", "spconv_status_string",
    "spconv_last_error", "spconv_weights_prepare", "spconv_forward_prepared", "spconv_weights_free",
    "spconv_attention_forward", "spconv_attention_backward", "spconv_norm_rotary_forward", "spconv_norm_rotary_backward",
    "spconv_rotary_table", "spconv_attention_workspace", "spconv_attention_forward_noalloc", "spconv_attention_backward_noalloc",
    "spconv_norm_rotary_workspace", "spconv_norm_rotary_backward_noalloc",
)
MAP_KINDS = {0: "submanifold", 1: "strided", 2: "transposed"}
DATAFLOWS = {0: "fused", 1: "grouped"}


class spconv_dataflow(ctypes.Structure):
    """Mirror of the C struct spconv_dataflow."""
    _fields_ = [("kind", ctypes.c_int32), ("groups", ctypes.c_int32), ("epsilon", ctypes.c_double),
                ("S", ctypes.c_double), ("ms", ctypes.c_float), ("fused_ms", ctypes.c_float),
                ("candidates", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class spconv_attention(ctypes.Structure):
    """Mirror of the C struct spconv_attention."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v")]
                + [(n, ctypes.c_int64) for n in ("q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride",
                                                 "v_row_stride", "v_head_stride")]
                + [(n, ctypes.c_void_p) for n in ("cu_q", "cu_k")]
                + [(n, ctypes.c_int64) for n in ("total_q", "total_k")]
                + [(n, ctypes.c_int32) for n in ("batch", "heads", "kv_heads", "head_dim", "left", "right")]
                + [("scale", ctypes.c_float), ("dtype", ctypes.c_int32)])


class spconv_attention_gradients(ctypes.Structure):
    """Mirror of the C struct spconv_attention_gradients."""
    _fields_ = [f for n in ("grad_out", "grad_q", "grad_k", "grad_v")
                for f in ((n, ctypes.c_void_p), (n + "_row_stride", ctypes.c_int64), (n + "_head_stride", ctypes.c_int64))]


class spconv_norm_rotary(ctypes.Structure):
    """Mirror of the C struct spconv_norm_rotary."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k")]
                + [(n, ctypes.c_int64) for n in ("q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride")]
                + [(n, ctypes.c_void_p) for n in ("q_weight", "k_weight", "table", "positions")]
                + [(n, ctypes.c_int64) for n in ("position_row_stride", "rows")]
                + [(n, ctypes.c_int32) for n in ("q_heads", "k_heads", "head_dim", "rotary_dim", "axes", "extent",
                                                 "interleaved")]
                + [("eps", ctypes.c_float), ("dtype", ctypes.c_int32)])


class spconv_norm_rotary_gradients(ctypes.Structure):
    """Mirror of the C struct spconv_norm_rotary_gradients."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("grad_q_out", "grad_k_out")]
                + [(n, ctypes.c_int64) for n in ("grad_q_out_row_stride", "grad_q_out_head_stride",
                                                 "grad_k_out_row_stride", "grad_k_out_head_stride")]
                + [(n, ctypes.c_void_p) for n in ("grad_q", "grad_k")]
                + [(n, ctypes.c_int64) for n in ("grad_q_row_stride", "grad_q_head_stride", "grad_k_row_stride",
                                                 "grad_k_head_stride")]
                + [(n, ctypes.c_void_p) for n in ("grad_q_weight", "grad_k_weight")])


_LIB: Optional[ctypes.CDLL] = None


class SpconvError(RuntimeError):
    """A non-OK status from the C ABI."""

    def __init__(self, status: int, detail: str):
        self.status = status
        self.name = STATUS.get(status, f"status {status}")
        super().__init__(f"{self.name}: {detail}")


def lib() -> ctypes.CDLL:
    """The loaded ``libspconv.so`` with argument types declared."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc for gfx950) first")
    # torch ships its own HIP runtime under the same soname (libamdhip64.so.7).
    # Loading torch first makes the library bind to that one runtime, so
    # torch's stream handles and allocations are valid in both.
    _torch()
    L = ctypes.CDLL(LIB_PATH)
    runtimes = _mapped_hip_runtimes()
    if len(runtimes) > 1:
        raise RuntimeError(f"two HIP runtimes are mapped in this process: {runtimes}")
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.spconv_abi_version.argtypes, L.spconv_abi_version.restype = [], i32
    L.spconv_build_map.argtypes = [vp, i64, i32, vp, ctypes.POINTER(vp)]
    L.spconv_build_map.restype = ctypes.c_int
    L.spconv_build_map_async.argtypes = [vp, i64, i32, vp, ctypes.POINTER(vp)]
    L.spconv_build_map_async.restype = ctypes.c_int
    L.spconv_map_wait.argtypes, L.spconv_map_wait.restype = [vp], ctypes.c_int
    L.spconv_map_info.argtypes = [vp, ctypes.POINTER(i32), ctypes.POINTER(i64), ctypes.POINTER(i64)]
    L.spconv_map_info.restype = ctypes.c_int
    L.spconv_map_counts.argtypes = [vp, vp, vp]
    L.spconv_map_counts.restype = ctypes.c_int
    L.spconv_map_lists.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp)]
    L.spconv_map_lists.restype = ctypes.c_int
    L.spconv_forward.argtypes = [vp, vp, vp, i32, i32, ctypes.c_int, vp, vp]
    L.spconv_forward.restype = ctypes.c_int
    L.spconv_forward_noalloc.argtypes = L.spconv_forward.argtypes
    L.spconv_forward_noalloc.restype = ctypes.c_int
    L.spconv_weights_prepare.argtypes = [vp, i32, i32, i32, ctypes.c_int, vp, ctypes.POINTER(vp)]
    L.spconv_weights_prepare.restype = ctypes.c_int
    L.spconv_forward_prepared.argtypes = [vp, vp, vp, vp, vp]
    L.spconv_forward_prepared.restype = ctypes.c_int
    L.spconv_weights_free.argtypes, L.spconv_weights_free.restype = [vp], None
    L.spconv_backward_data.argtypes = L.spconv_forward.argtypes
    L.spconv_backward_data.restype = ctypes.c_int
    L.spconv_backward_weights.argtypes = L.spconv_forward.argtypes
    L.spconv_backward_weights.restype = ctypes.c_int
    L.spconv_build_map_strided.argtypes = [vp, i64, i32, i32, vp, ctypes.POINTER(vp)]
    L.spconv_build_map_strided.restype = ctypes.c_int
    L.spconv_map_transpose.argtypes = [vp, vp, ctypes.POINTER(vp)]
    L.spconv_map_transpose.restype = ctypes.c_int
    L.spconv_map_geometry.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i32),
                                      ctypes.POINTER(i32)]
    L.spconv_map_geometry.restype = ctypes.c_int
    L.spconv_map_out_coords.argtypes = [vp, ctypes.POINTER(vp)]
    L.spconv_map_out_coords.restype = ctypes.c_int
    f64, pi32 = ctypes.c_double, ctypes.POINTER(i32)
    L.spconv_group_plan.argtypes = [vp, f64, f64, i32, pi32, pi32, pi32, pi32, ctypes.POINTER(i64)]
    L.spconv_group_plan.restype = ctypes.c_int
    L.spconv_group_plan_counts.argtypes = [ctypes.POINTER(i64), i32, i32, f64, f64, i32, pi32, pi32, pi32, pi32,
                                           ctypes.POINTER(i64)]
    L.spconv_group_plan_counts.restype = ctypes.c_int
    L.spconv_forward_grouped.argtypes = [vp, vp, vp, i32, i32, ctypes.c_int, f64, f64, vp, vp]
    L.spconv_forward_grouped.restype = ctypes.c_int
    L.spconv_select_dataflow.argtypes = [vp, vp, vp, i32, i32, ctypes.c_int, ctypes.POINTER(f64), i32,
                                         ctypes.POINTER(f64), i32, i32, vp, vp, ctypes.POINTER(spconv_dataflow)]
    L.spconv_select_dataflow.restype = ctypes.c_int
    # struct arguments as void*: a ctypes struct by reference, or packed bytes
    L.spconv_attention_forward.argtypes = [vp, vp, vp, vp]
    L.spconv_attention_forward.restype = ctypes.c_int
    L.spconv_attention_backward.argtypes = [vp, vp, vp, vp, vp]
    L.spconv_attention_backward.restype = ctypes.c_int
    L.spconv_norm_rotary_forward.argtypes = [vp, vp, i64, i64, vp, i64, i64, vp]
    L.spconv_norm_rotary_forward.restype = ctypes.c_int
    L.spconv_norm_rotary_backward.argtypes = [vp, vp, vp]
    L.spconv_norm_rotary_backward.restype = ctypes.c_int
    L.spconv_attention_workspace.argtypes = [vp, vp, vp]
    L.spconv_attention_workspace.restype = ctypes.c_int
    L.spconv_attention_forward_noalloc.argtypes = [vp, vp, vp, vp, ctypes.c_uint64, vp]
    L.spconv_attention_forward_noalloc.restype = ctypes.c_int
    L.spconv_attention_backward_noalloc.argtypes = [vp, vp, vp, vp, vp, ctypes.c_uint64, vp]
    L.spconv_attention_backward_noalloc.restype = ctypes.c_int
    L.spconv_norm_rotary_workspace.argtypes = [i32, vp]
    L.spconv_norm_rotary_workspace.restype = ctypes.c_int
    L.spconv_norm_rotary_backward_noalloc.argtypes = [vp, vp, vp, ctypes.c_uint64, vp]
    L.spconv_norm_rotary_backward_noalloc.restype = ctypes.c_int
    L.spconv_rotary_table.argtypes = [vp, i32, i32, f64, f64, vp]
    L.spconv_rotary_table.restype = ctypes.c_int
    L.spconv_map_free.argtypes, L.spconv_map_free.restype = [vp], None
    L.spconv_status_string.argtypes, L.spconv_status_string.restype = [ctypes.c_int], ctypes.c_char_p
    L.spconv_last_error.argtypes, L.spconv_last_error.restype = [], ctypes.c_char_p
    # the runtime's own copy routine, resolved through the library's dependencies
    L.hipMemcpyAsync.argtypes = [vp, vp, ctypes.c_size_t, ctypes.c_int, vp]
    L.hipMemcpyAsync.restype = ctypes.c_int
    _LIB = L
    return L


def _mapped_hip_runtimes():
    try:
        with open("/proc/self/maps") as f:
            return sorted({l.split()[-1] for l in f if "libamdhip64" in l})
    except OSError:
        return []


def _check(status: int) -> None:
    if status != 0:
        raise SpconvError(status, lib().spconv_last_error().decode(errors="replace"))


# ------------------------------------------------------------------ raw C names


def spconv_abi_version() -> int:
    return int(lib().spconv_abi_version())


def spconv_build_map(d_coords: int, n: int, kernel_size: int, hip_stream: int) -> int:
    """Raw call: returns the map handle (int) or raises SpconvError."""
    h = ctypes.c_void_p()
    _check(lib().spconv_build_map(d_coords, n, kernel_size, hip_stream, ctypes.byref(h)))
    return int(h.value)


def spconv_build_map_async(d_coords: int, n: int, kernel_size: int, hip_stream: int) -> int:
    """Raw call: enqueues the build and returns the map handle (int); device
    errors surface in spconv_map_wait / spconv_map_info / spconv_map_counts."""
    h = ctypes.c_void_p()
    _check(lib().spconv_build_map_async(d_coords, n, kernel_size, hip_stream, ctypes.byref(h)))
    return int(h.value)


def spconv_map_wait(handle: int) -> None:
    _check(lib().spconv_map_wait(handle))


def spconv_map_info(handle: int) -> Tuple[int, int, int]:
    K, n, e = ctypes.c_int32(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().spconv_map_info(handle, ctypes.byref(K), ctypes.byref(n), ctypes.byref(e)))
    return K.value, n.value, e.value


def spconv_map_counts(handle: int, kernel_volume: int) -> Tuple[np.ndarray, np.ndarray]:
    counts = np.zeros(kernel_volume, np.int64)
    offsets = np.zeros(kernel_volume + 1, np.int64)
    _check(lib().spconv_map_counts(handle, counts.ctypes.data, offsets.ctypes.data))
    return counts, offsets


def spconv_map_lists(handle: int) -> Tuple[int, int]:
    a, b = ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib().spconv_map_lists(handle, ctypes.byref(a), ctypes.byref(b)))
    return int(a.value or 0), int(b.value or 0)


def spconv_forward(d_feats: int, d_weights: int, handle: int, c_in: int, c_out: int, dtype: int,
                   d_out: int, hip_stream: int) -> None:
    _check(lib().spconv_forward(d_feats, d_weights, handle, c_in, c_out, dtype, d_out, hip_stream))


def spconv_forward_noalloc(d_feats: int, d_weights: int, handle: int, c_in: int, c_out: int, dtype: int,
                           d_out: int, hip_stream: int) -> None:
    _check(lib().spconv_forward_noalloc(d_feats, d_weights, handle, c_in, c_out, dtype, d_out, hip_stream))


def spconv_weights_prepare(d_weights: int, kernel_volume: int, c_in: int, c_out: int, dtype: int,
                           hip_stream: int) -> int:
    h = ctypes.c_void_p()
    _check(lib().spconv_weights_prepare(d_weights, kernel_volume, c_in, c_out, dtype, hip_stream, ctypes.byref(h)))
    return int(h.value)


def spconv_forward_prepared(d_feats: int, weights: int, handle: int, d_out: int, hip_stream: int) -> None:
    _check(lib().spconv_forward_prepared(d_feats, weights, handle, d_out, hip_stream))


def spconv_weights_free(weights: int) -> None:
    lib().spconv_weights_free(weights)


def spconv_backward_data(d_grad_out: int, d_weights: int, handle: int, c_in: int, c_out: int, dtype: int,
                         d_grad_in: int, hip_stream: int) -> None:
    _check(lib().spconv_backward_data(d_grad_out, d_weights, handle, c_in, c_out, dtype, d_grad_in, hip_stream))


def spconv_backward_weights(d_feats: int, d_grad_out: int, handle: int, c_in: int, c_out: int, dtype: int,
                            d_grad_w: int, hip_stream: int) -> None:
    _check(lib().spconv_backward_weights(d_feats, d_grad_out, handle, c_in, c_out, dtype, d_grad_w, hip_stream))


def spconv_build_map_strided(d_coords: int, n_in: int, kernel_size: int, stride: int, hip_stream: int) -> int:
    h = ctypes.c_void_p()
    _check(lib().spconv_build_map_strided(d_coords, n_in, kernel_size, stride, hip_stream, ctypes.byref(h)))
    return int(h.value)


def spconv_map_transpose(handle: int, hip_stream: int) -> int:
    h = ctypes.c_void_p()
    _check(lib().spconv_map_transpose(handle, hip_stream, ctypes.byref(h)))
    return int(h.value)


def spconv_map_geometry(handle: int) -> Tuple[int, int, int, int]:
    n_in, n_out = ctypes.c_int64(), ctypes.c_int64()
    stride, kind = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().spconv_map_geometry(handle, ctypes.byref(n_in), ctypes.byref(n_out), ctypes.byref(stride),
                                     ctypes.byref(kind)))
    return n_in.value, n_out.value, stride.value, kind.value


def spconv_map_out_coords(handle: int) -> int:
    p = ctypes.c_void_p()
    _check(lib().spconv_map_out_coords(handle, ctypes.byref(p)))
    return int(p.value or 0)


def spconv_group_plan(handle: int, epsilon: float, S: float, kernel_volume: int):
    """(offsets, groups, n_groups, padded_rows) of the plan: offsets and
    group indices of the entries in execution order."""
    offs = (ctypes.c_int32 * kernel_volume)()
    grp = (ctypes.c_int32 * kernel_volume)()
    n, ng, pad = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
    _check(lib().spconv_group_plan(handle, float(epsilon), float(S), kernel_volume, offs, grp, ctypes.byref(n),
                                   ctypes.byref(ng), ctypes.byref(pad)))
    return list(offs[:n.value]), list(grp[:n.value]), ng.value, pad.value


def spconv_group_plan_counts(counts, epsilon: float, S: float, centre: int = -1):
    """(offsets, groups, n_groups, padded_rows) of the plan over the given
    per-offset map sizes (no map, no device)."""
    kv = len(counts)
    arr = (ctypes.c_int64 * max(kv, 1))(*[int(c) for c in counts])
    offs = (ctypes.c_int32 * max(kv, 1))()
    grp = (ctypes.c_int32 * max(kv, 1))()
    n, ng, pad = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
    _check(lib().spconv_group_plan_counts(arr, kv, int(centre), float(epsilon), float(S), kv, offs, grp,
                                          ctypes.byref(n), ctypes.byref(ng), ctypes.byref(pad)))
    return list(offs[:n.value]), list(grp[:n.value]), ng.value, pad.value


def spconv_forward_grouped(d_feats: int, d_weights: int, handle: int, c_in: int, c_out: int, dtype: int,
                           epsilon: float, S: float, d_out: int, hip_stream: int) -> None:
    _check(lib().spconv_forward_grouped(d_feats, d_weights, handle, c_in, c_out, dtype, float(epsilon), float(S),
                                        d_out, hip_stream))


def spconv_select_dataflow(d_feats: int, d_weights: int, handle: int, c_in: int, c_out: int, dtype: int,
                           epsilons, thresholds, reps: int, d_out: int, hip_stream: int) -> spconv_dataflow:
    def grid(v):
        if v is None:
            return None, 0
        arr = (ctypes.c_double * len(v))(*[float(x) for x in v])
        return arr, len(v)
    e, ne = grid(epsilons)
    t, nt = grid(thresholds)
    best = spconv_dataflow()
    _check(lib().spconv_select_dataflow(d_feats, d_weights, handle, c_in, c_out, dtype, e, ne, t, nt, int(reps),
                                        d_out, hip_stream, ctypes.byref(best)))
    return best


def spconv_attention_forward(args: spconv_attention, d_out: int, d_lse: int, hip_stream: int) -> None:
    _check(lib().spconv_attention_forward(ctypes.byref(args), d_out, d_lse, hip_stream))


def spconv_attention_backward(args: spconv_attention, d_out: int, d_lse: int, grads: spconv_attention_gradients,
                              hip_stream: int) -> None:
    _check(lib().spconv_attention_backward(ctypes.byref(args), d_out, d_lse, ctypes.byref(grads), hip_stream))


def spconv_attention_workspace(args: spconv_attention) -> Tuple[int, int]:
    """Bytes of workspace of the forward and of the gradient."""
    return _attention_workspace(ctypes.byref(args))


def _attention_workspace(args) -> Tuple[int, int]:
    f, b = ctypes.c_uint64(), ctypes.c_uint64()
    _check(lib().spconv_attention_workspace(args, ctypes.byref(f), ctypes.byref(b)))
    return f.value, b.value


def spconv_attention_forward_noalloc(args: spconv_attention, d_out: int, d_lse: int, d_workspace: int, workspace_bytes: int,
                                     hip_stream: int) -> None:
    _check(lib().spconv_attention_forward_noalloc(ctypes.byref(args), d_out, d_lse, d_workspace, workspace_bytes, hip_stream))


def spconv_attention_backward_noalloc(args: spconv_attention, d_out: int, d_lse: int, grads: spconv_attention_gradients,
                                      d_workspace: int, workspace_bytes: int, hip_stream: int) -> None:
    _check(lib().spconv_attention_backward_noalloc(ctypes.byref(args), d_out, d_lse, ctypes.byref(grads), d_workspace,
                                                   workspace_bytes, hip_stream))


def spconv_norm_rotary_workspace(head_dim: int) -> int:
    """Bytes of workspace of the gradient."""
    b = ctypes.c_uint64()
    _check(lib().spconv_norm_rotary_workspace(head_dim, ctypes.byref(b)))
    return b.value


def spconv_norm_rotary_backward_noalloc(args: spconv_norm_rotary, grads: spconv_norm_rotary_gradients, d_workspace: int,
                                        workspace_bytes: int, hip_stream: int) -> None:
    _check(lib().spconv_norm_rotary_backward_noalloc(ctypes.byref(args), ctypes.byref(grads), d_workspace, workspace_bytes,
                                                     hip_stream))


def spconv_norm_rotary_forward(args: spconv_norm_rotary, d_q_out: int, q_out_row_stride: int, q_out_head_stride: int,
                               d_k_out: int, k_out_row_stride: int, k_out_head_stride: int, hip_stream: int) -> None:
    _check(lib().spconv_norm_rotary_forward(ctypes.byref(args), d_q_out, q_out_row_stride, q_out_head_stride,
                                            d_k_out, k_out_row_stride, k_out_head_stride, hip_stream))


def spconv_norm_rotary_backward(args: spconv_norm_rotary, grads: spconv_norm_rotary_gradients,
                                hip_stream: int) -> None:
    _check(lib().spconv_norm_rotary_backward(ctypes.byref(args), ctypes.byref(grads), hip_stream))


def spconv_rotary_table(d_table: int, extent: int, pairs: int, base: float, position_scale: float,
                        hip_stream: int) -> None:
    _check(lib().spconv_rotary_table(d_table, extent, pairs, float(base), float(position_scale), hip_stream))


def spconv_map_free(handle: int) -> None:
    lib().spconv_map_free(handle)


def spconv_status_string(status: int) -> str:
    return lib().spconv_status_string(status).decode()


def spconv_last_error() -> str:
    return lib().spconv_last_error().decode(errors="replace")


# ------------------------------------------------------------------ torch front end


def _torch():
    import torch
    return torch


def _stream() -> int:
    """Handle of torch's current stream on the current device."""
    return int(_torch().cuda.current_stream().cuda_stream)


def _run(device: int, call, *args) -> None:
    """call(*args, stream) with ``device`` current, on torch's current stream
    there, and its status checked: what :class:`_OnDevice` and :func:`_stream`
    do, at a tenth of the host time (the stream's handle without a stream
    object).

    A call that needs a workspace is refused under graph capture and runs with
    one of torch's allocator instead, which the graph keeps."""
    C = _TORCH._C
    if C._cuda_getDevice() != device:
        with _TORCH.cuda.device(device):
            return _run(device, call, *args)
    rc = call(*args, C._cuda_getCurrentRawStream(device))
    if rc and call.__name__ in _WORKSPACES and _TORCH.cuda.is_current_stream_capturing():
        workspace = _TORCH.empty(_WORKSPACES[call.__name__](args[0]), dtype=_TORCH.uint8, device=f"cuda:{device}")
        rc = getattr(_LIB, call.__name__ + "_noalloc")(*args, workspace.data_ptr(), workspace.numel(),
                                                       C._cuda_getCurrentRawStream(device))
    if rc:
        _check(rc)


# Bytes of workspace of the calls that have a _noalloc variant, from their packed arguments.
_WORKSPACES = {
    "spconv_attention_forward": lambda a: _attention_workspace(a)[0],
    "spconv_attention_backward": lambda a: _attention_workspace(a)[1],
    "spconv_norm_rotary_backward": lambda a: spconv_norm_rotary_workspace(spconv_norm_rotary.from_buffer_copy(a).head_dim),
}


_TORCH = None


def _bind():
    """torch and the library, for the calls below (loaded on the first one)."""
    global _TORCH
    if _TORCH is None or _LIB is None:
        lib()
        _TORCH = _torch()
    return _TORCH, _LIB


class _OnDevice:
    """Makes ``device`` current for the call only when it is not already."""

    __slots__ = ("idx", "prev")

    def __init__(self, device):
        self.idx = device.index if device.index is not None else 0
        self.prev = None

    def __enter__(self):
        torch = _torch()
        cur = torch.cuda.current_device()
        if cur != self.idx:
            self.prev = cur
            torch.cuda.set_device(self.idx)

    def __exit__(self, *exc):
        if self.prev is not None:
            _torch().cuda.set_device(self.prev)


class SpconvMap:
    """A kernel map on the GPU (owns the C handle).  ``n`` is its number of
    output rows and ``n_in`` of input rows (equal for a submanifold map);
    ``kind`` is "submanifold", "strided" or "transposed"."""

    def __init__(self, handle: int, device, kernel_size: int, n: int, n_in: Optional[int] = None,
                 stride: int = 1, kind: str = "submanifold"):
        self.handle = handle
        self.device = device
        self.kernel_size, self.n = kernel_size, n
        self.n_in = n if n_in is None else n_in
        self.stride, self.kind = stride, kind
        self.kernel_volume = self.kernel_size ** 3
        self._counts = None
        self._total = None

    @classmethod
    def _from_handle(cls, h: int, device, kernel_size: int) -> "SpconvMap":
        n_in, n_out, stride, kind = spconv_map_geometry(h)
        return cls(h, device, kernel_size, n_out, n_in, stride, MAP_KINDS[kind])

    def out_coords(self):
        """Output coordinates (int32 [n, 4] device tensor, a stream-ordered
        copy) of a strided or transposed map."""
        torch = _torch()
        src = spconv_map_out_coords(self.handle)
        out = torch.empty((self.n, 4), dtype=torch.int32, device=self.device)
        if self.n:
            with _OnDevice(self.device):
                rc = lib().hipMemcpyAsync(out.data_ptr(), src, 16 * self.n, 3, _stream())
                if rc != 0:
                    raise SpconvError(6, f"hipMemcpyAsync failed with {rc}")
        return out

    def transpose(self) -> "SpconvMap":
        """The transposed (upsampling) map of a strided map."""
        with _OnDevice(self.device):
            h = spconv_map_transpose(self.handle, _stream())
        return SpconvMap._from_handle(h, self.device, self.kernel_size)

    def wait(self) -> None:
        """Waits for the build (a no-op once done); raises its device error."""
        spconv_map_wait(self.handle)

    @property
    def total_entries(self) -> int:
        if self._total is None:
            self._total = spconv_map_info(self.handle)[2]
        return self._total

    def _load_counts(self):
        if self._counts is None:
            self._counts = spconv_map_counts(self.handle, self.kernel_volume)
        return self._counts

    @property
    def counts(self) -> np.ndarray:
        """Entries per offset, int64 [K^3]."""
        return self._load_counts()[0]

    @property
    def offsets(self) -> np.ndarray:
        """List offsets, int64 [K^3 + 1]."""
        return self._load_counts()[1]

    def lists(self):
        """(in_idx, out_idx) as int32 device tensors: stream-ordered copies of
        the map's lists (the map owns the originals)."""
        torch = _torch()
        a, b = spconv_map_lists(self.handle)
        e = self.total_entries
        out = torch.empty((2, e), dtype=torch.int32, device=self.device)
        if e:
            with _OnDevice(self.device):
                stream = _stream()
                for dst, src in ((out[0].data_ptr(), a), (out[1].data_ptr(), b)):
                    rc = lib().hipMemcpyAsync(dst, src, 4 * e, 3, stream)  # device to device
                    if rc != 0:
                        raise SpconvError(6, f"hipMemcpyAsync failed with {rc}")
        return out[0], out[1]

    def free(self):
        if self.handle:
            spconv_map_free(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def build_map(coords, kernel_size: int, wait: bool = True) -> SpconvMap:
    """Kernel map of a K^3 submanifold convolution over int32 [N, 4]
    (b, z, y, x) coordinates resident on a HIP device.  With wait=False the
    build is only enqueued (device errors then surface in ``SpconvMap.wait``
    or the first query of counts)."""
    torch = _torch()
    if not (isinstance(coords, torch.Tensor) and coords.is_cuda and coords.dtype == torch.int32
            and coords.dim() == 2 and coords.shape[1] == 4 and coords.is_contiguous()):
        raise SpconvError(1, "coords must be a contiguous int32 [N, 4] tensor on a HIP device")
    call = spconv_build_map if wait else spconv_build_map_async
    with _OnDevice(coords.device):
        h = call(coords.data_ptr(), coords.shape[0], int(kernel_size), _stream())
    return SpconvMap(h, coords.device, int(kernel_size), int(coords.shape[0]))


def build_map_strided(coords, kernel_size: int, stride: int) -> SpconvMap:
    """Kernel map of a strided (downsampling) convolution with a K^3 kernel
    (offset components -floor((K-1)/2) ..) over int32 [N, 4] coordinates on a
    HIP device; its outputs (``out_coords``) follow the regular output
    definition in lexicographic order."""
    torch = _torch()
    if not (isinstance(coords, torch.Tensor) and coords.is_cuda and coords.dtype == torch.int32
            and coords.dim() == 2 and coords.shape[1] == 4 and coords.is_contiguous()):
        raise SpconvError(1, "coords must be a contiguous int32 [N, 4] tensor on a HIP device")
    with _OnDevice(coords.device):
        h = spconv_build_map_strided(coords.data_ptr(), coords.shape[0], int(kernel_size), int(stride), _stream())
    return SpconvMap._from_handle(h, coords.device, int(kernel_size))


_DT = None


def forward(feats, weights, kmap: SpconvMap, out=None, noalloc=False):
    """f_out = sparse convolution of feats [n_in, C_in] with weights
    [K^3, C_in, C_out] over ``kmap``; returns out [n, C_out] (same dtype;
    n_in = n for a submanifold map).
    With ``noalloc`` the call goes to ``spconv_forward_noalloc`` (the
    library's fixed per-device scratch instead of an allocated workspace;
    ``out`` must then be given, so that nothing is allocated here either)."""
    global _DT
    torch = _torch()
    if _DT is None:
        _DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    if not (feats.is_cuda and weights.is_cuda and feats.is_contiguous() and weights.is_contiguous()):
        raise SpconvError(1, "feats and weights must be contiguous tensors on a HIP device")
    if feats.dim() != 2 or weights.dim() != 3:
        raise SpconvError(1, "feats must be [N, C_in] and weights [K^3, C_in, C_out]")
    n_in, cin = feats.shape
    n = kmap.n
    kv, wcin, cout = weights.shape
    if n_in != kmap.n_in or kv != kmap.kernel_volume or wcin != cin:
        raise SpconvError(1, f"shape mismatch: feats {tuple(feats.shape)}, weights "
                             f"{tuple(weights.shape)}, map n_in={kmap.n_in} K^3={kmap.kernel_volume}")
    dt = feats.dtype
    if weights.dtype != dt:
        raise SpconvError(1, "feats and weights must share one dtype")
    code = _DT.get(dt)
    if code is None:
        raise SpconvError(4, f"dtype {dt} not supported")
    if out is None:
        if noalloc:
            raise SpconvError(1, "noalloc needs a caller-allocated out")
        out = torch.empty((n, cout), dtype=dt, device=feats.device)
    elif not (out.is_cuda and out.is_contiguous() and out.dtype == dt and tuple(out.shape) == (n, cout)):
        raise SpconvError(1, "out must be a contiguous [N, C_out] tensor of the feature dtype")
    with _OnDevice(feats.device):
        fn = spconv_forward_noalloc if noalloc else spconv_forward
        fn(feats.data_ptr(), weights.data_ptr(), kmap.handle, cin, cout, code, out.data_ptr(), _stream())
    return out


class PreparedWeights:
    """A layer's weights copied once for repeated forwards
    (``spconv_weights_prepare``); later changes to the tensor it was made
    from do not reach it."""

    def __init__(self, weights):
        global _DT
        torch = _torch()
        if _DT is None:
            _DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
        if not (weights.is_cuda and weights.is_contiguous() and weights.dim() == 3):
            raise SpconvError(1, "weights must be a contiguous [K^3, C_in, C_out] tensor on a HIP device")
        code = _DT.get(weights.dtype)
        if code is None:
            raise SpconvError(4, f"dtype {weights.dtype} not supported")
        self.kernel_volume, self.c_in, self.c_out = (int(v) for v in weights.shape)
        self.dtype, self.device, self.handle = weights.dtype, weights.device, None
        with _OnDevice(weights.device):
            self.handle = spconv_weights_prepare(weights.data_ptr(), self.kernel_volume, self.c_in, self.c_out,
                                                 code, _stream())

    def free(self) -> None:
        if self.handle:
            spconv_weights_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def prepare_weights(weights) -> PreparedWeights:
    """Prepares [K^3, C_in, C_out] weights for ``forward_prepared``."""
    return PreparedWeights(weights)


def forward_prepared(feats, pw: PreparedWeights, kmap: SpconvMap, out=None):
    """``forward`` with prepared weights (bit-identical output)."""
    torch = _torch()
    if pw.handle is None:
        raise SpconvError(1, "the prepared weights were freed")
    if not (feats.is_cuda and feats.is_contiguous() and feats.dim() == 2 and feats.dtype == pw.dtype):
        raise SpconvError(1, "feats must be a contiguous [N, C_in] tensor on a HIP device of the weights' dtype")
    if feats.shape[0] != kmap.n_in or feats.shape[1] != pw.c_in or pw.kernel_volume != kmap.kernel_volume:
        raise SpconvError(1, f"shape mismatch: feats {tuple(feats.shape)}, weights "
                             f"[{pw.kernel_volume}, {pw.c_in}, {pw.c_out}], map n_in={kmap.n_in} "
                             f"K^3={kmap.kernel_volume}")
    if out is None:
        out = torch.empty((kmap.n, pw.c_out), dtype=pw.dtype, device=feats.device)
    elif not (out.is_cuda and out.is_contiguous() and out.dtype == pw.dtype and tuple(out.shape) == (kmap.n, pw.c_out)):
        raise SpconvError(1, "out must be a contiguous [N, C_out] tensor of the feature dtype")
    with _OnDevice(feats.device):
        spconv_forward_prepared(feats.data_ptr(), pw.handle, kmap.handle, out.data_ptr(), _stream())
    return out


def _check_pair(a, b, kmap: SpconvMap, what, rows_a=None):
    rows_a = kmap.n if rows_a is None else rows_a
    if not (a.is_cuda and b.is_cuda and a.is_contiguous() and b.is_contiguous()):
        raise SpconvError(1, f"{what} must be contiguous tensors on a HIP device")
    if a.dim() != 2 or b.dim() != 2 or a.shape[0] != rows_a or b.shape[0] != kmap.n:
        raise SpconvError(1, f"{what} must be [{rows_a}, C] and [{kmap.n}, C]")
    if a.dtype != b.dtype:
        raise SpconvError(1, f"{what} must share one dtype")


def backward_data(grad_out, weights, kmap: SpconvMap, out=None):
    """Gradient of ``forward`` with respect to its features: grad_in
    [N, C_in] from grad_out [N, C_out] and the forward's weights
    [K^3, C_in, C_out] (same dtype)."""
    global _DT
    torch = _torch()
    if _DT is None:
        _DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    if not (weights.is_cuda and weights.is_contiguous() and weights.dim() == 3):
        raise SpconvError(1, "weights must be a contiguous [K^3, C_in, C_out] tensor on a HIP device")
    kv, cin, cout = weights.shape
    _check_pair(grad_out, grad_out, kmap, "grad_out")
    if kv != kmap.kernel_volume or grad_out.shape[1] != cout or weights.dtype != grad_out.dtype:
        raise SpconvError(1, f"shape mismatch: grad_out {tuple(grad_out.shape)}, weights {tuple(weights.shape)}")
    code = _DT.get(grad_out.dtype)
    if code is None:
        raise SpconvError(4, f"dtype {grad_out.dtype} not supported")
    if out is None:
        out = torch.empty((kmap.n_in, cin), dtype=grad_out.dtype, device=grad_out.device)
    elif not (out.is_cuda and out.is_contiguous() and out.dtype == grad_out.dtype
              and tuple(out.shape) == (kmap.n_in, cin)):
        raise SpconvError(1, "out must be a contiguous [n_in, C_in] tensor of the gradient dtype")
    with _OnDevice(grad_out.device):
        spconv_backward_data(grad_out.data_ptr(), weights.data_ptr(), kmap.handle, cin, cout, code, out.data_ptr(),
                             _stream())
    return out


def backward_weights(feats, grad_out, kmap: SpconvMap, out=None):
    """Gradient of ``forward`` with respect to its weights: fp32
    [K^3, C_in, C_out] from feats [n_in, C_in] and grad_out [n, C_out]."""
    global _DT
    torch = _torch()
    if _DT is None:
        _DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    _check_pair(feats, grad_out, kmap, "feats and grad_out", rows_a=kmap.n_in)
    code = _DT.get(feats.dtype)
    if code is None:
        raise SpconvError(4, f"dtype {feats.dtype} not supported")
    cin, cout = feats.shape[1], grad_out.shape[1]
    shape = (kmap.kernel_volume, cin, cout)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=feats.device)
    elif not (out.is_cuda and out.is_contiguous() and out.dtype == torch.float32 and tuple(out.shape) == shape):
        raise SpconvError(1, "out must be a contiguous fp32 [K^3, C_in, C_out] tensor")
    with _OnDevice(feats.device):
        spconv_backward_weights(feats.data_ptr(), grad_out.data_ptr(), kmap.handle, cin, cout, code, out.data_ptr(),
                                _stream())
    return out


def _forward_operands(feats, weights, kmap: SpconvMap, out):
    """Checks the operands of a forward and returns (c_in, c_out, dtype
    code, out)."""
    global _DT
    torch = _torch()
    if _DT is None:
        _DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    if not (feats.is_cuda and weights.is_cuda and feats.is_contiguous() and weights.is_contiguous()):
        raise SpconvError(1, "feats and weights must be contiguous tensors on a HIP device")
    if feats.dim() != 2 or weights.dim() != 3:
        raise SpconvError(1, "feats must be [N, C_in] and weights [K^3, C_in, C_out]")
    n_in, cin = feats.shape
    kv, wcin, cout = weights.shape
    if n_in != kmap.n_in or kv != kmap.kernel_volume or wcin != cin:
        raise SpconvError(1, f"shape mismatch: feats {tuple(feats.shape)}, weights "
                             f"{tuple(weights.shape)}, map n_in={kmap.n_in} K^3={kmap.kernel_volume}")
    dt = feats.dtype
    if weights.dtype != dt:
        raise SpconvError(1, "feats and weights must share one dtype")
    code = _DT.get(dt)
    if code is None:
        raise SpconvError(4, f"dtype {dt} not supported")
    if out is None:
        out = torch.empty((kmap.n, cout), dtype=dt, device=feats.device)
    elif not (out.is_cuda and out.is_contiguous() and out.dtype == dt and tuple(out.shape) == (kmap.n, cout)):
        raise SpconvError(1, "out must be a contiguous [N, C_out] tensor of the feature dtype")
    return cin, cout, code, out


def group_plan(kmap: SpconvMap, epsilon: float, S: float):
    """The offset groups of the adaptive grouping with (epsilon, S) over
    ``kmap``, in execution order (a list of lists of offset indices), and the
    rows of the padded batches."""
    offs, grp, ng, pad = spconv_group_plan(kmap.handle, epsilon, S, kmap.kernel_volume)
    groups = [[] for _ in range(ng)]
    for k, g in zip(offs, grp):
        groups[g].append(k)
    return groups, pad


def group_plan_counts(counts, epsilon: float, S: float, centre: Optional[int] = None):
    """The groups (a list of lists of offset indices, in execution order) and
    padded rows of the adaptive grouping over per-offset map sizes."""
    offs, grp, ng, pad = spconv_group_plan_counts(counts, epsilon, S, -1 if centre is None else centre)
    groups = [[] for _ in range(ng)]
    for k, g in zip(offs, grp):
        groups[g].append(k)
    return groups, pad


def forward_grouped(feats, weights, kmap: SpconvMap, epsilon: float, S: float = float("inf"), out=None):
    """``forward`` in the weight-stationary dataflow with adaptive grouping
    (epsilon, S): gather, one batched MFMA product per group, reduction
    (f16 / bf16, C_in % 32 == 0, C_out % 16 == 0)."""
    cin, cout, code, out = _forward_operands(feats, weights, kmap, out)
    with _OnDevice(feats.device):
        spconv_forward_grouped(feats.data_ptr(), weights.data_ptr(), kmap.handle, cin, cout, code, epsilon, S,
                               out.data_ptr(), _stream())
    return out


def select_dataflow(feats, weights, kmap: SpconvMap, epsilons=None, thresholds=None, reps: int = 3, out=None):
    """Times the fused forward and the grouped forward over a grid of
    (epsilon, S) on these operands and returns (choice, out): choice is a
    dict (dataflow, groups, epsilon, S, ms, fused_ms, candidates) and out
    holds the chosen dataflow's result."""
    cin, cout, code, out = _forward_operands(feats, weights, kmap, out)
    with _OnDevice(feats.device):
        b = spconv_select_dataflow(feats.data_ptr(), weights.data_ptr(), kmap.handle, cin, cout, code, epsilons,
                                   thresholds, reps, out.data_ptr(), _stream())
    choice = {"dataflow": DATAFLOWS.get(b.kind, str(b.kind)), "groups": b.groups, "epsilon": b.epsilon, "S": b.S,
              "ms": b.ms, "fused_ms": b.fused_ms, "candidates": b.candidates}
    return choice, out


def forward_with(choice, feats, weights, kmap: SpconvMap, out=None):
    """The forward in the dataflow ``select_dataflow`` chose."""
    if choice["dataflow"] == "grouped":
        return forward_grouped(feats, weights, kmap, choice["epsilon"], choice["S"], out=out)
    return forward(feats, weights, kmap, out=out)


# ------------------------------------------------------------------ attention over packed rows

# The C structs as packed bytes (native sizes and alignment): one pack costs a
# fraction of setting a ctypes struct's fields one by one.
_PACK_ATTENTION = struct.Struct("@3P6q2P2q6ifi")
_PACK_ATTENTION_GRADIENTS = struct.Struct("@" + "P2q" * 4)
_PACK_NORM_ROTARY = struct.Struct("@2P4q4P2q7ifi0q")
_PACK_NORM_ROTARY_GRADIENTS = struct.Struct("@2P4q2P4q2P")


def _dtype_code(dtype):
    global _DT
    if _DT is None:
        torch = _torch()
        _DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    code = _DT.get(dtype)
    if code is None:
        raise SpconvError(4, f"dtype {dtype} not supported")
    return code


def _heads_tensor(name, t, like=None, shape=None):
    """Checks a [rows, heads, head_dim] tensor whose last dimension is
    contiguous; returns (pointer, row stride, head stride)."""
    if t.dim() != 3 or not t.is_cuda:
        raise SpconvError(1, f"{name} must be a [rows, heads, head_dim] tensor on a HIP device")
    row, head, last = t.stride()
    if last != 1 and t.shape[2] > 1:
        raise SpconvError(1, f"{name} must have a contiguous last dimension")
    if like is not None and (t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise SpconvError(1, f"{name} must have the dtype and device of the other tensors")
    if shape is not None and t.shape != shape:
        raise SpconvError(1, f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr(), row, head


def _offsets_tensor(name, cu, device: int):
    if not (cu.get_device() == device and cu.dtype is _TORCH.int32 and cu.dim() == 1 and cu.is_contiguous()
            and cu.shape[0] >= 1):
        raise SpconvError(1, f"{name} must be a contiguous int32 [batch + 1] tensor on the tensors' device")
    return cu.data_ptr()


def _attention_args(q, k, v, cu_q, cu_k, causal, window, scale):
    """The packed spconv_attention of a call."""
    qp, qr, qh = _heads_tensor("q", q)
    kp, kr, kh = _heads_tensor("k", k, q)
    vp, vr, vh = _heads_tensor("v", v, q, k.shape)
    code = _dtype_code(q.dtype)
    total_q, heads, dim = q.shape
    total_k, kv_heads, kdim = k.shape
    if kdim != dim:
        raise SpconvError(1, f"q and k must share one head_dim, not {dim} and {kdim}")
    device = q.get_device()
    cq = _offsets_tensor("cu_q", cu_q, device)
    if cu_k is None or cu_k is cu_q:
        ck = cq
    else:
        ck = _offsets_tensor("cu_k", cu_k, device)
        if cu_q.shape != cu_k.shape:
            raise SpconvError(1, "cu_q and cu_k must hold the same number of sequences")
    left, right = window
    left, right = max(-1, min(int(left), 1 << 30)), max(-1, min(int(right), 1 << 30))
    scale = float(dim) ** -0.5 if scale is None else float(scale)
    if not 0.0 < scale < 3e38:  # an fp32 number
        raise SpconvError(1, f"scale = {scale} must be positive and finite")
    return _PACK_ATTENTION.pack(qp, kp, vp, qr, qh, kr, kh, vr, vh, cq, ck, total_q, total_k, cu_q.shape[0] - 1, heads,
                                kv_heads, dim, left, 0 if causal else right, scale, code)


def attention(q, k, v, cu_q, cu_k=None, *, causal: bool = False, window=(-1, -1), scale: Optional[float] = None,
              out=None, return_lse: bool = False):
    """Softmax attention over packed sequences: q [total_q, heads, head_dim],
    k and v [total_k, kv_heads, head_dim] (f32, f16 or bf16; any row and head
    strides that are multiples of 16 bytes, so slices of one projection's
    output serve), cu_q and cu_k int32 [batch + 1] row offsets of the
    sequences on the device (cu_k None: the queries' own).

    The last query of a sequence stands at its last key.  ``causal``: no key
    after a query's place; ``window`` (left, right): only keys from place -
    left to place + right, -1 for unbounded.  ``scale`` defaults to
    head_dim ** -0.5.  A query that sees no key gets zeros.

    Returns out [total_q, heads, head_dim], or (out, lse) with
    ``return_lse``: lse fp32 [total_q, heads], what
    :func:`attention_backward` needs.  Both calls may be captured in a graph
    (their workspaces then come from torch's allocator, and stay the graph's)."""
    torch, L = _bind()
    a = _attention_args(q, k, v, cu_q, cu_k, causal, window, scale)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif not (out.get_device() == q.get_device() and out.is_contiguous() and out.dtype is q.dtype and out.shape == q.shape):
        raise SpconvError(1, "out must be a contiguous [total_q, heads, head_dim] tensor of the dtype")
    lse = q.new_empty(q.shape[:2], dtype=torch.float32)
    _run(q.get_device(), L.spconv_attention_forward, a, out.data_ptr(), lse.data_ptr())
    return (out, lse) if return_lse else out


def attention_backward(grad_out, q, k, v, out, lse, cu_q, cu_k=None, *, causal: bool = False, window=(-1, -1),
                       scale: Optional[float] = None, grads=None):
    """Gradients (grad_q, grad_k, grad_v) of :func:`attention` from the
    gradient of its output, its inputs, and its out and lse.  ``grads``: three
    tensors to write, such as the slices of one projection's gradient."""
    torch, L = _bind()
    a = _attention_args(q, k, v, cu_q, cu_k, causal, window, scale)
    if not (out.get_device() == q.get_device() and out.is_contiguous() and out.dtype is q.dtype and out.shape == q.shape):
        raise SpconvError(1, "out must be the forward's contiguous [total_q, heads, head_dim] output")
    if not (lse.get_device() == q.get_device() and lse.is_contiguous() and lse.dtype is torch.float32
            and lse.shape == q.shape[:2]):
        raise SpconvError(1, "lse must be the forward's contiguous fp32 [total_q, heads] output")
    if grads is None:
        grads = tuple(torch.empty_like(x, memory_format=torch.contiguous_format) for x in (q, k, v))
    g = _PACK_ATTENTION_GRADIENTS.pack(*_heads_tensor("grad_out", grad_out, q, q.shape),
                                       *_heads_tensor("grad_q", grads[0], q, q.shape),
                                       *_heads_tensor("grad_k", grads[1], q, k.shape),
                                       *_heads_tensor("grad_v", grads[2], q, v.shape))
    _run(q.get_device(), L.spconv_attention_backward, a, out.data_ptr(), lse.data_ptr(), g)
    return tuple(grads)


# ------------------------------------------------------------------ head norm and position rotation


def rotary_table(extent: int, pairs: int, base: float = 10000.0, position_scale: float = 1.0, device="cuda"):
    """Cosines and sines [extent, pairs, 2] (fp32) of the angles
    position * position_scale * base ** (-i / pairs), i < pairs."""
    torch, L = _bind()
    table = torch.empty((int(extent), int(pairs), 2), dtype=torch.float32, device=device)
    _run(table.get_device(), L.spconv_rotary_table, table.data_ptr(), int(extent), int(pairs), float(base), float(position_scale))
    return table


_NO_TENSOR = (0, 0, 0)


def _norm_rotary_args(q, k, q_weight, k_weight, table, positions, rotary_dim, interleaved, eps):
    """The packed spconv_norm_rotary of a call."""
    like = k if q is None else q
    if like is None:
        raise SpconvError(1, "q and k are both None")
    qp, qr, qh = _NO_TENSOR if q is None else _heads_tensor("q", q)
    kp, kr, kh = _NO_TENSOR if k is None else _heads_tensor("k", k, like)
    rows, _, dim = like.shape
    code = _dtype_code(like.dtype)
    if k is not None and (k.shape[0] != rows or k.shape[2] != dim):
        raise SpconvError(1, f"q and k must share rows and head_dim, not {tuple(like.shape)} and {tuple(k.shape)}")
    device = like.get_device()
    weights = [0, 0]
    for i, w in enumerate((q_weight, k_weight)):
        if w is None:
            continue
        if not (w.get_device() == device and w.dim() == 1 and w.shape[0] == dim and w.is_contiguous()
                and w.dtype is like.dtype):
            raise SpconvError(1, f"{'qk'[i]}_weight must be a contiguous [head_dim] tensor of the dtype on the tensors' device")
        weights[i] = w.data_ptr()
    tp = pp = pr = rotary = axes = extent = 0
    if table is None:
        if rotary_dim:
            raise SpconvError(1, "a rotation needs a table and positions")
    else:
        if not (table.get_device() == device and table.dtype is _TORCH.float32 and table.dim() == 3
                and table.shape[2] == 2 and table.is_contiguous()):
            raise SpconvError(1, "table must be a contiguous fp32 [extent, pairs, 2] tensor on the tensors' device")
        if positions is None or not (positions.get_device() == device and positions.dtype is _TORCH.int32
                                     and positions.dim() in (1, 2)):
            raise SpconvError(1, "positions must be an int32 [rows] or [rows, axes] tensor on the tensors' device")
        strides = positions.stride()
        axes = 1 if len(strides) == 1 else positions.shape[1]
        if positions.shape[0] != rows or (axes > 1 and strides[1] != 1):
            raise SpconvError(1, f"positions must hold {rows} rows of contiguous components")
        extent, pairs, _ = table.shape
        rotary = 2 * axes * pairs
        if rotary_dim is not None and rotary_dim != rotary:
            raise SpconvError(1, f"rotary_dim = {rotary_dim} must be 2 x {axes} axes x {pairs} pairs of the table")
        tp, pp, pr = table.data_ptr(), positions.data_ptr(), strides[0]
    if not 0.0 <= eps < 3e38:
        raise SpconvError(1, f"eps = {eps} must be finite and not negative")
    return _PACK_NORM_ROTARY.pack(qp, kp, qr, qh, kr, kh, weights[0], weights[1], tp, pp, pr, rows,
                                  0 if q is None else q.shape[1], 0 if k is None else k.shape[1], dim, rotary, axes,
                                  extent, 1 if interleaved else 0, eps, code)


def norm_rotary(q, k, q_weight=None, k_weight=None, table=None, positions=None, *, rotary_dim: Optional[int] = None,
                interleaved: bool = False, eps: float = 1e-6, out=None):
    """The RMS norm of every head of q [rows, heads, head_dim] and
    k [rows, kv_heads, head_dim] (weights [head_dim]; None: no norm) and the
    rotation of each head's first ``rotary_dim`` elements by the row's
    position, in one pass.

    ``table`` (:func:`rotary_table`) holds rotary_dim / (2 axes) pairs;
    ``positions`` is int32 [rows] or [rows, axes], such as ``coords[:, 1:]`` of
    voxel coordinates.  ``interleaved``: pairs (2p, 2p + 1), else
    (p, p + rotary_dim / 2).  A position outside the table gives NaN.

    Returns (q', k'); ``out``: two tensors to write, which may be q and k
    themselves.  Either of q and k may be None."""
    torch, L = _bind()
    a = _norm_rotary_args(q, k, q_weight, k_weight, table, positions, rotary_dim, interleaved, eps)
    like = k if q is None else q
    if out is None:
        out = (None if q is None else torch.empty_like(q, memory_format=torch.contiguous_format),
               None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format))
    qo = _NO_TENSOR if q is None else _heads_tensor("q_out", out[0], like, q.shape)
    ko = _NO_TENSOR if k is None else _heads_tensor("k_out", out[1], like, k.shape)
    _run(like.get_device(), L.spconv_norm_rotary_forward, a, *qo, *ko)
    return tuple(out)


def norm_rotary_backward(grad_q_out, grad_k_out, q, k, q_weight=None, k_weight=None, table=None, positions=None, *,
                         rotary_dim: Optional[int] = None, interleaved: bool = False, eps: float = 1e-6, grads=None):
    """Gradients (grad_q, grad_k, grad_q_weight, grad_k_weight) of
    :func:`norm_rotary` from the gradients of its outputs and its inputs; the
    weights' are fp32 [head_dim] (None without a weight).  ``grads``: two
    tensors for grad_q and grad_k, which may be the outputs' gradients
    themselves."""
    torch, L = _bind()
    a = _norm_rotary_args(q, k, q_weight, k_weight, table, positions, rotary_dim, interleaved, eps)
    like = k if q is None else q
    if grads is None:
        grads = tuple(None if x is None else torch.empty_like(x, memory_format=torch.contiguous_format) for x in (q, k))
    given, made, weights = [], [], [None, None]
    for i, (x, w, go) in enumerate(((q, q_weight, grad_q_out), (k, k_weight, grad_k_out))):
        if x is None:
            given.append(_NO_TENSOR)
            made.append(_NO_TENSOR)
            continue
        given.append(_heads_tensor(f"grad_{'qk'[i]}_out", go, like, x.shape))
        made.append(_heads_tensor(f"grad_{'qk'[i]}", grads[i], like, x.shape))
        if w is not None:
            weights[i] = like.new_empty(like.shape[2], dtype=torch.float32)
    (gqo, gko), (gq, gk) = given, made
    g = _PACK_NORM_ROTARY_GRADIENTS.pack(gqo[0], gko[0], *gqo[1:], *gko[1:], gq[0], gk[0], *gq[1:], *gk[1:],
                                         *(0 if w is None else w.data_ptr() for w in weights))
    _run(like.get_device(), L.spconv_norm_rotary_backward, a, g)
    return grads[0], grads[1], weights[0], weights[1]
