"""Thin ctypes binding of liblrm.so (include/lrm.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensor arguments may be torch tensors (their data_ptr() is passed)
or plain integer device addresses.  Every function raises LrmError on a
non-OK status.  There is no CPU fallback: if the library is missing or the
device is not a GB300, the calls fail loudly.
"""

from __future__ import annotations

import ctypes
import os
from fractions import Fraction

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "liblrm.so")

LRM_OK = 0
STATUS_NAMES = [
    "LRM_OK",
    "LRM_ERR_INVALID_ARG",
    "LRM_ERR_SHAPE",
    "LRM_ERR_ALIGN",
    "LRM_ERR_WORKSPACE",
    "LRM_ERR_INDEX",
    "LRM_ERR_QUOTA",
    "LRM_ERR_TIMEOUT",
    "LRM_ERR_ARCH",
    "LRM_ERR_CUDA",
]
(LRM_ERR_INVALID_ARG, LRM_ERR_SHAPE, LRM_ERR_ALIGN, LRM_ERR_WORKSPACE, LRM_ERR_INDEX, LRM_ERR_QUOTA,
 LRM_ERR_TIMEOUT, LRM_ERR_ARCH, LRM_ERR_CUDA) = range(1, 10)
LRM_OP_ROUTE_STATS = 0
LRM_OP_SELECT = 1
LRM_OP_ZERO_DROPPED = 2
LRM_OP_COMBINE = 3
LRM_OP_ROUTER = 4
DTYPE_F32, DTYPE_BF16 = 0, 1

# every entry point declared in include/lrm.h
EXPORTED = (
    "lrm_create",
    "lrm_destroy",
    "lrm_status_string",
    "lrm_abi_version",
    "lrm_sm_count",
    "lrm_workspace_size",
    "lrm_route_stats",
    "lrm_score",
    "lrm_select",
    "lrm_compact",
    "lrm_grouped_dgrad",
    "lrm_grouped_wgrad",
    "lrm_grouped_wgrad_bf16",
    "lrm_compact_padded",
    "lrm_get_device_status",
    "lrm_set_wait_budget",
    "lrm_selftest_wait_timeout",
    "lrm_route_stats_noalloc",
    "lrm_score_metric",
    "lrm_grouped_dgrad_scatter",
    "lrm_zero_dropped_rows",
    "lrm_swiglu_backward",
    "lrm_combine_rows",
    "lrm_capacity",
    "lrm_max_rows",
    "lrm_router_forward",
    "lrm_route_stats_counted",
    "lrm_counted_rows",
    "lrm_router_backward",
    "lrm_gate_grad",
    "lrm_grad_table_size",
    "lrm_grad_list_create",
    "lrm_grad_list_destroy",
    "lrm_grad_list_status",
    "lrm_grad_norm",
    "lrm_grad_clip",
    "lrm_ffn_up",
    "lrm_ffn_down",
    "lrm_ffn_combine",
    "lrm_ffn_backward_workspace",
    "lrm_ffn_backward",
    "lrm_layer_norm",
    "lrm_layer_norm_workspace",
    "lrm_layer_norm_backward",
    "lrm_dropout_add",
)

# selection metrics of lrm_score_metric (the ablation of LRMoE sec. 4.7, Table 2)
METRIC_LRM, METRIC_GRAD_L2SQ, METRIC_GRAD_L1, METRIC_RANDOM = 0, 1, 2, 3

# bytes of the library's fixed scratch array used by lrm_route_stats_noalloc
ROUTE_STATS_SCRATCH_BYTES = 4 << 20


class LrmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        name = STATUS_NAMES[code] if 0 <= code < len(STATUS_NAMES) else f"status {code}"
        super().__init__(f"{where}: {name}")


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("h", ctypes.c_int32),
                ("I", ctypes.c_int32)]


class RouteSummary(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32),
        ("C", ctypes.c_int32),
        ("slots", ctypes.c_int32),
        ("dropped", ctypes.c_int32),
        ("retained", ctypes.c_int32),
        ("max_count", ctypes.c_int32),
        ("min_count", ctypes.c_int32),
        ("nonempty", ctypes.c_int32),
        ("aux_unscaled", ctypes.c_float),
        ("drop_rate", ctypes.c_float),
        ("util", ctypes.c_float),
        ("rho_real", ctypes.c_float),
        ("max_over_mean", ctypes.c_float),
        ("sum_P", ctypes.c_float),
    ]


class RouterLosses(ctypes.Structure):
    _fields_ = [("loss", ctypes.c_float), ("aux", ctypes.c_float), ("z", ctypes.c_float), ("tokens", ctypes.c_int32)]


class Tensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class GradStats(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_float), ("coef", ctypes.c_float), ("nonfinite", ctypes.c_int32)]


SUMMARY_BYTES = ctypes.sizeof(RouteSummary)

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load liblrm.so and declare its signatures (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m backward_token_expert_gb300.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    i32 = ctypes.c_int32
    st = ctypes.c_int
    sig = {
        "lrm_create": ([ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)], st),
        "lrm_destroy": ([P], st),
        "lrm_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "lrm_abi_version": ([], i32),
        "lrm_sm_count": ([P, ctypes.POINTER(i32)], st),
        "lrm_workspace_size": ([P, ctypes.c_int, Dims, ctypes.POINTER(ctypes.c_size_t)], st),
        "lrm_route_stats": ([P, P, P, Dims, i32, i32, i32, i32, P, P, P, P, P, P, P, P, ctypes.c_size_t, P], st),
        "lrm_score": ([P, P, P, P, Dims, P, P], st),
        "lrm_select": ([P, P, P, P, P, Dims, i32, P, P, P, ctypes.c_size_t, P], st),
        "lrm_compact": ([P, P, P, P, P, P, Dims, i32, P, P, P, P], st),
        "lrm_grouped_dgrad": ([P, P, P, P, Dims, i32, P, P], st),
        "lrm_grouped_wgrad": ([P, P, P, P, Dims, i32, i32, P, P], st),
        "lrm_grouped_wgrad_bf16": ([P, P, P, P, Dims, i32, i32, P, P], st),
        "lrm_compact_padded": ([P, P, P, P, Dims, i32, P, P, P, P], st),
        "lrm_get_device_status": ([P, P, ctypes.POINTER(ctypes.c_uint32)], st),
        "lrm_set_wait_budget": ([P, ctypes.c_uint64], st),
        "lrm_selftest_wait_timeout": ([P, ctypes.c_uint64, P], st),
        "lrm_route_stats_noalloc": ([P, P, P, Dims, i32, i32, i32, i32, P, P, P, P, P, P, P, P], st),
        "lrm_score_metric": ([P, i32, P, P, P, Dims, ctypes.c_uint64, P, P], st),
        "lrm_grouped_dgrad_scatter": ([P, P, P, P, P, Dims, i32, P, P], st),
        "lrm_zero_dropped_rows": ([P, P, P, Dims, i32, P, P, ctypes.c_size_t, P], st),
        "lrm_swiglu_backward": ([P, P, P, P, Dims, i32, P, P], st),
        "lrm_combine_rows": ([P, P, P, P, Dims, i32, i32, P, P, ctypes.c_size_t, P], st),
        "lrm_capacity": ([Dims, i32, i32, ctypes.POINTER(i32)], st),
        "lrm_max_rows": ([Dims, i32, i32, i32, i32, ctypes.POINTER(i32)], st),
    }
    f32 = ctypes.c_float
    size = ctypes.c_size_t
    sig.update({
        "lrm_router_forward": ([P, P, i32, P, Dims, i32, f32, f32, P, P, P, P, P, P, P, P, size, P], st),
        "lrm_route_stats_counted": ([P, P, P, P, P, Dims] + [i32] * 4 + [P] * 8 + [size, P], st),
        "lrm_counted_rows": ([P, P, P, Dims, i32, P, P], st),
        "lrm_router_backward": ([P, P, i32, P, P, P, P, P, P, Dims, i32, f32, f32, P, i32, P], st),
        "lrm_gate_grad": ([P, P, P, P, P, Dims, i32, P, P], st),
        "lrm_grad_table_size": ([ctypes.POINTER(Tensor), i32, ctypes.POINTER(size)], st),
        "lrm_grad_list_create": ([P, ctypes.POINTER(Tensor), i32, P, size, P, ctypes.POINTER(P)], st),
        "lrm_grad_list_destroy": ([P], st),
        "lrm_grad_list_status": ([P, P, P, ctypes.POINTER(ctypes.c_uint32)], st),
        "lrm_grad_norm": ([P, P, P, P], st),
        "lrm_grad_clip": ([P, P, f32, P, P], st),
    })
    sig.update({
        "lrm_ffn_up": ([P, P, P, P, P, Dims, i32, P, P, P], st),
        "lrm_ffn_down": ([P, P, P, P, P, Dims, i32, P, P], st),
        "lrm_ffn_combine": ([P, P, P, Dims, P, P], st),
        "lrm_ffn_backward_workspace": ([P, Dims, i32, ctypes.POINTER(size)], st),
        "lrm_ffn_backward": ([P] * 6 + [Dims, i32, P, P, P, size, P], st),
        "lrm_layer_norm": ([P, P, i32, P, P, P, i32, i32, f32, P, P, P], st),
        "lrm_layer_norm_workspace": ([P, i32, i32, ctypes.POINTER(size)], st),
        "lrm_layer_norm_backward": ([P, P, i32, P, P, P, P, P, i32, i32, P, P, P, P, size, P], st),
        "lrm_dropout_add": ([P, P, P, i32, ctypes.c_int64, ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64, P, P, P],
                            st),
    })
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _ptr(x) -> int | None:
    return x if x is None or isinstance(x, int) else x.data_ptr()


_raw_stream = None  # torch's (lookup of a device's current raw stream, lookup of the current device), once CUDA is up


def _stream(stream) -> int | None:
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch

            if not torch.cuda.is_initialized():
                return torch.cuda.current_stream().cuda_stream
            _raw_stream = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        # the raw handle: making a torch stream object costs about 3 us a call, a third of a small call's host time
        return _raw_stream[0](_raw_stream[1]())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(code: int, where: str) -> None:
    if code != LRM_OK:
        raise LrmError(code, where)


def dims_of(T, E, k, h, I) -> Dims:
    return Dims(int(T), int(E), int(k), int(h), int(I))


# ---------------------------------------------------------------------------
# the C entry points, same names, argument marshalling only


def lrm_create(device: int = 0) -> int:
    lib = load_library()
    out = ctypes.c_void_p()
    _check(lib.lrm_create(int(device), ctypes.byref(out)), "lrm_create")
    return out.value


def lrm_destroy(ctx: int) -> None:
    _check(load_library().lrm_destroy(ctx), "lrm_destroy")


def lrm_status_string(code: int) -> str:
    return load_library().lrm_status_string(int(code)).decode()


def lrm_abi_version() -> int:
    return int(load_library().lrm_abi_version())


def lrm_sm_count(ctx: int) -> int:
    out = ctypes.c_int32()
    _check(load_library().lrm_sm_count(ctx, ctypes.byref(out)), "lrm_sm_count")
    return out.value


def lrm_workspace_size(ctx: int, op: int, dims: Dims) -> int:
    out = ctypes.c_size_t()
    _check(load_library().lrm_workspace_size(ctx, int(op), dims, ctypes.byref(out)), "lrm_workspace_size")
    return out.value


def lrm_capacity(dims: Dims, cf) -> int:
    """C = floor(CF * N / E), computed by the library (host only)."""
    cf = Fraction(cf)
    out = ctypes.c_int32()
    _check(load_library().lrm_capacity(dims, cf.numerator, cf.denominator, ctypes.byref(out)), "lrm_capacity")
    return out.value


def lrm_max_rows(dims: Dims, cf, rho) -> int:
    """Upper bound of the retained total over any routing, computed by the library (host only)."""
    cf = Fraction(cf)
    rho = Fraction(rho)
    out = ctypes.c_int32()
    _check(load_library().lrm_max_rows(dims, cf.numerator, cf.denominator, rho.numerator, rho.denominator,
                                       ctypes.byref(out)), "lrm_max_rows")
    return out.value


def lrm_route_stats(ctx, logits, expert_idx, dims: Dims, cf, rho, counts, offsets, bucket, P, f, quota,
                    summary, ws, ws_bytes: int, stream=None) -> None:
    cf = Fraction(cf)
    rho = Fraction(rho)
    _check(load_library().lrm_route_stats(ctx, _ptr(logits), _ptr(expert_idx), dims, cf.numerator,
                                          cf.denominator, rho.numerator, rho.denominator, _ptr(counts),
                                          _ptr(offsets), _ptr(bucket), _ptr(P), _ptr(f), _ptr(quota),
                                          _ptr(summary), _ptr(ws), int(ws_bytes), _stream(stream)),
           "lrm_route_stats")


def lrm_route_stats_noalloc(ctx, logits, expert_idx, dims: Dims, cf, rho, counts, offsets, bucket, P, f, quota,
                            summary, stream=None) -> None:
    """lrm_route_stats with the library's fixed scratch array instead of a workspace."""
    cf = Fraction(cf)
    rho = Fraction(rho)
    _check(load_library().lrm_route_stats_noalloc(ctx, _ptr(logits), _ptr(expert_idx), dims, cf.numerator,
                                                  cf.denominator, rho.numerator, rho.denominator, _ptr(counts),
                                                  _ptr(offsets), _ptr(bucket), _ptr(P), _ptr(f), _ptr(quota),
                                                  _ptr(summary), _stream(stream)),
           "lrm_route_stats_noalloc")


def lrm_score(ctx, g, phi, alpha, dims: Dims, score, stream=None) -> None:
    _check(load_library().lrm_score(ctx, _ptr(g), _ptr(phi), _ptr(alpha), dims, _ptr(score), _stream(stream)),
           "lrm_score")


def lrm_score_metric(ctx, metric: int, g, phi, alpha, dims: Dims, seed: int, score, stream=None) -> None:
    _check(load_library().lrm_score_metric(ctx, int(metric), _ptr(g), _ptr(phi), _ptr(alpha), dims,
                                           int(seed) & ((1 << 64) - 1), _ptr(score), _stream(stream)),
           "lrm_score_metric")


def lrm_grouped_dgrad_scatter(ctx, delta_c, W, sel_offsets, sel_ids, dims: Dims, max_rows: int, dphi_rows,
                              stream=None) -> None:
    _check(load_library().lrm_grouped_dgrad_scatter(ctx, _ptr(delta_c), _ptr(W), _ptr(sel_offsets), _ptr(sel_ids),
                                                    dims, int(max_rows), _ptr(dphi_rows), _stream(stream)),
           "lrm_grouped_dgrad_scatter")


def lrm_zero_dropped_rows(ctx, sel_offsets, sel_ids, dims: Dims, max_rows: int, rows, ws, ws_bytes: int,
                          stream=None) -> None:
    _check(load_library().lrm_zero_dropped_rows(ctx, _ptr(sel_offsets), _ptr(sel_ids), dims, int(max_rows),
                                                _ptr(rows), _ptr(ws), int(ws_bytes), _stream(stream)),
           "lrm_zero_dropped_rows")


def lrm_swiglu_backward(ctx, dphi_c, ab_c, sel_offsets, dims: Dims, max_rows: int, dh1, stream=None) -> None:
    _check(load_library().lrm_swiglu_backward(ctx, _ptr(dphi_c), _ptr(ab_c), _ptr(sel_offsets), dims,
                                              int(max_rows), _ptr(dh1), _stream(stream)), "lrm_swiglu_backward")


def lrm_combine_rows(ctx, rows, sel_offsets, sel_ids, dims: Dims, max_rows: int, width: int, out, ws, ws_bytes: int,
                     stream=None) -> None:
    _check(load_library().lrm_combine_rows(ctx, _ptr(rows), _ptr(sel_offsets), _ptr(sel_ids), dims, int(max_rows),
                                           int(width), _ptr(out), _ptr(ws), int(ws_bytes), _stream(stream)),
           "lrm_combine_rows")


def lrm_select(ctx, score, offsets, bucket, quota, dims: Dims, max_rows: int, sel_offsets, sel_ids, ws=None,
               ws_bytes: int = 0, stream=None) -> None:
    _check(load_library().lrm_select(ctx, _ptr(score), _ptr(offsets), _ptr(bucket), _ptr(quota), dims,
                                     int(max_rows), _ptr(sel_offsets), _ptr(sel_ids), _ptr(ws), int(ws_bytes),
                                     _stream(stream)), "lrm_select")


def lrm_compact(ctx, g, phi, alpha, sel_offsets, sel_ids, dims: Dims, max_rows: int, delta_c, phi_c,
                alpha_c=None, stream=None) -> None:
    _check(load_library().lrm_compact(ctx, _ptr(g), _ptr(phi), _ptr(alpha), _ptr(sel_offsets), _ptr(sel_ids),
                                      dims, int(max_rows), _ptr(delta_c), _ptr(phi_c), _ptr(alpha_c),
                                      _stream(stream)), "lrm_compact")


def lrm_grouped_dgrad(ctx, delta_c, W, sel_offsets, dims: Dims, max_rows: int, dphi_c, stream=None) -> None:
    _check(load_library().lrm_grouped_dgrad(ctx, _ptr(delta_c), _ptr(W), _ptr(sel_offsets), dims, int(max_rows),
                                            _ptr(dphi_c), _stream(stream)), "lrm_grouped_dgrad")


def lrm_grouped_wgrad(ctx, delta_c, phi_c, sel_offsets, dims: Dims, max_rows: int, accumulate: int, dW,
                      stream=None) -> None:
    _check(load_library().lrm_grouped_wgrad(ctx, _ptr(delta_c), _ptr(phi_c), _ptr(sel_offsets), dims,
                                            int(max_rows), int(accumulate), _ptr(dW), _stream(stream)),
           "lrm_grouped_wgrad")


def lrm_grouped_wgrad_bf16(ctx, delta_c, phi_c, sel_offsets, dims: Dims, max_rows: int, accumulate: int, dW,
                           stream=None) -> None:
    _check(load_library().lrm_grouped_wgrad_bf16(ctx, _ptr(delta_c), _ptr(phi_c), _ptr(sel_offsets), dims,
                                                 int(max_rows), int(accumulate), _ptr(dW), _stream(stream)),
           "lrm_grouped_wgrad_bf16")


def lrm_compact_padded(ctx, delta_c, phi_c, sel_offsets, dims: Dims, C: int, delta_pad, phi_pad, pad_offsets,
                       stream=None) -> None:
    _check(load_library().lrm_compact_padded(ctx, _ptr(delta_c), _ptr(phi_c), _ptr(sel_offsets), dims, int(C),
                                             _ptr(delta_pad), _ptr(phi_pad), _ptr(pad_offsets), _stream(stream)),
           "lrm_compact_padded")


def lrm_router_forward(ctx, logits, logits_dtype: int, valid, dims: Dims, renorm: bool, aux_coef: float,
                       z_coef: float, expert_idx, alpha, row_stats, counts, f, P, losses, ws, ws_bytes: int,
                       stream=None) -> None:
    _check(load_library().lrm_router_forward(ctx, _ptr(logits), logits_dtype, _ptr(valid), dims, renorm, aux_coef,
                                             z_coef, _ptr(expert_idx), _ptr(alpha), _ptr(row_stats), _ptr(counts),
                                             _ptr(f), _ptr(P), _ptr(losses), _ptr(ws), ws_bytes, _stream(stream)),
           "lrm_router_forward")


def lrm_route_stats_counted(ctx, logits, expert_idx, row_stats, losses, dims: Dims, cf: Fraction, rho: Fraction,
                            counts, offsets, bucket, P, f, quota, summary, ws, ws_bytes: int, stream=None) -> None:
    cf, rho = Fraction(cf), Fraction(rho)
    _check(load_library().lrm_route_stats_counted(ctx, _ptr(logits), _ptr(expert_idx), _ptr(row_stats), _ptr(losses),
                                                  dims, cf.numerator, cf.denominator, rho.numerator, rho.denominator,
                                                  _ptr(counts), _ptr(offsets), _ptr(bucket), _ptr(P), _ptr(f),
                                                  _ptr(quota), _ptr(summary), _ptr(ws), ws_bytes, _stream(stream)),
           "lrm_route_stats_counted")


def lrm_counted_rows(ctx, rows, row_stats, dims: Dims, width: int, out, stream=None) -> None:
    _check(load_library().lrm_counted_rows(ctx, _ptr(rows), _ptr(row_stats), dims, width, _ptr(out), _stream(stream)),
           "lrm_counted_rows")


def lrm_router_backward(ctx, logits, logits_dtype: int, expert_idx, alpha, row_stats, dgate, f, losses, dims: Dims,
                        renorm: bool, aux_coef: float, z_coef: float, dlogits, dlogits_dtype: int,
                        stream=None) -> None:
    _check(load_library().lrm_router_backward(ctx, _ptr(logits), logits_dtype, _ptr(expert_idx), _ptr(alpha),
                                              _ptr(row_stats), _ptr(dgate), _ptr(f), _ptr(losses), dims, renorm,
                                              aux_coef, z_coef, _ptr(dlogits), dlogits_dtype, _stream(stream)),
           "lrm_router_backward")


def lrm_gate_grad(ctx, dphi_c, phi_c, sel_offsets, sel_ids, dims: Dims, max_rows: int, dgate, stream=None) -> None:
    _check(load_library().lrm_gate_grad(ctx, _ptr(dphi_c), _ptr(phi_c), _ptr(sel_offsets), _ptr(sel_ids), dims,
                                        max_rows, _ptr(dgate), _stream(stream)), "lrm_gate_grad")


def tensor_array(entries):
    """A C array of lrm_tensor from (src, dst, n, dtype) entries."""
    array = (Tensor * max(1, len(entries)))()
    for t, (src, dst, n, dtype) in zip(array, entries):
        t.src, t.dst, t.n, t.dtype = _ptr(src), _ptr(dst), n, dtype
    return array


def lrm_grad_table_size(tensors, count: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().lrm_grad_table_size(tensors, int(count), ctypes.byref(out)), "lrm_grad_table_size")
    return out.value


def lrm_grad_list_create(ctx, tensors, count: int, table, table_bytes: int, stream=None) -> int:
    out = ctypes.c_void_p()
    _check(load_library().lrm_grad_list_create(ctx, tensors, int(count), _ptr(table), int(table_bytes),
                                               _stream(stream), ctypes.byref(out)), "lrm_grad_list_create")
    return out.value


def lrm_grad_list_destroy(grad_list: int) -> None:
    _check(load_library().lrm_grad_list_destroy(grad_list), "lrm_grad_list_destroy")


def lrm_grad_list_status(ctx, grad_list: int, stream=None) -> int:
    out = ctypes.c_uint32()
    _check(load_library().lrm_grad_list_status(ctx, grad_list, _stream(stream), ctypes.byref(out)),
           "lrm_grad_list_status")
    return out.value


def lrm_grad_norm(ctx, grad_list: int, stats, stream=None) -> None:
    _check(load_library().lrm_grad_norm(ctx, grad_list, _ptr(stats), _stream(stream)), "lrm_grad_norm")


def lrm_grad_clip(ctx, grad_list: int, max_norm: float, stats, stream=None) -> None:
    _check(load_library().lrm_grad_clip(ctx, grad_list, max_norm, _ptr(stats), _stream(stream)), "lrm_grad_clip")


def lrm_ffn_up(ctx, x, W1, offsets, ids, dims: Dims, max_rows: int, ab, phi, stream=None) -> None:
    _check(load_library().lrm_ffn_up(ctx, _ptr(x), _ptr(W1), _ptr(offsets), _ptr(ids), dims, max_rows, _ptr(ab),
                                     _ptr(phi), _stream(stream)), "lrm_ffn_up")


def lrm_ffn_down(ctx, phi, W, offsets, ids, dims: Dims, max_rows: int, rows, stream=None) -> None:
    _check(load_library().lrm_ffn_down(ctx, _ptr(phi), _ptr(W), _ptr(offsets), _ptr(ids), dims, max_rows, _ptr(rows),
                                       _stream(stream)), "lrm_ffn_down")


def lrm_ffn_combine(ctx, rows, alpha, dims: Dims, out, stream=None) -> None:
    _check(load_library().lrm_ffn_combine(ctx, _ptr(rows), _ptr(alpha), dims, _ptr(out), _stream(stream)),
           "lrm_ffn_combine")


def lrm_ffn_backward_workspace(ctx, dims: Dims, max_rows: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().lrm_ffn_backward_workspace(ctx, dims, max_rows, ctypes.byref(out)),
           "lrm_ffn_backward_workspace")
    return out.value


def lrm_ffn_backward(ctx, delta_c, W, ab, sel_offsets, sel_ids, dims: Dims, max_rows: int, dh1, dgate, ws,
                     ws_bytes: int, stream=None) -> None:
    _check(load_library().lrm_ffn_backward(ctx, _ptr(delta_c), _ptr(W), _ptr(ab), _ptr(sel_offsets), _ptr(sel_ids),
                                           dims, max_rows, _ptr(dh1), _ptr(dgate), _ptr(ws), ws_bytes,
                                           _stream(stream)), "lrm_ffn_backward")


def lrm_layer_norm(ctx, x, dtype: int, gamma, beta, valid, rows: int, width: int, eps: float, y, stats,
                   stream=None) -> None:
    _check(load_library().lrm_layer_norm(ctx, _ptr(x), dtype, _ptr(gamma), _ptr(beta), _ptr(valid), rows, width, eps,
                                         _ptr(y), _ptr(stats), _stream(stream)), "lrm_layer_norm")


def lrm_layer_norm_workspace(ctx, rows: int, width: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().lrm_layer_norm_workspace(ctx, rows, width, ctypes.byref(out)), "lrm_layer_norm_workspace")
    return out.value


def lrm_layer_norm_backward(ctx, x, dtype: int, dy, gamma, stats, valid, dres, rows: int, width: int, dx, dgamma,
                            dbeta, ws, ws_bytes: int, stream=None) -> None:
    _check(load_library().lrm_layer_norm_backward(ctx, _ptr(x), dtype, _ptr(dy), _ptr(gamma), _ptr(stats),
                                                  _ptr(valid), _ptr(dres), rows, width, _ptr(dx), _ptr(dgamma),
                                                  _ptr(dbeta), _ptr(ws), ws_bytes, _stream(stream)),
           "lrm_layer_norm_backward")


def lrm_dropout_add(ctx, x, residual, dtype: int, n: int, p: float, seed: int, offset: int, step, out,
                    stream=None) -> None:
    _check(load_library().lrm_dropout_add(ctx, _ptr(x), _ptr(residual), dtype, n, p, seed, offset, _ptr(step),
                                          _ptr(out), _stream(stream)), "lrm_dropout_add")


def lrm_get_device_status(ctx, stream=None) -> int:
    out = ctypes.c_uint32()
    _check(load_library().lrm_get_device_status(ctx, _stream(stream), ctypes.byref(out)),
           "lrm_get_device_status")
    return out.value


def lrm_set_wait_budget(ctx, ns: int) -> None:
    _check(load_library().lrm_set_wait_budget(ctx, int(ns)), "lrm_set_wait_budget")


def lrm_selftest_wait_timeout(ctx, budget_ns: int, stream=None) -> None:
    _check(load_library().lrm_selftest_wait_timeout(ctx, int(budget_ns), _stream(stream)),
           "lrm_selftest_wait_timeout")


def flag_names(flags: int) -> list[str]:
    return [STATUS_NAMES[c] for c in range(1, len(STATUS_NAMES)) if flags & (1 << c)]
