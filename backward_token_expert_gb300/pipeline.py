"""One backward recalibration of an MoE layer's FC2 through the C ABI.

``Recalibration`` owns the device buffers of one layer shape (allocated once
with torch, which is used here only for device memory and streams) and
enqueues the six library calls of the path on one stream, with no host
synchronisation in between:

    lrm_route_stats -> lrm_score -> lrm_select -> lrm_compact
                    -> lrm_grouped_dgrad -> lrm_grouped_wgrad

(LRMoE Alg. 1; the input-gradient product runs before the
weight-gradient product, the order TopoEP sec. 3.3 schedules them in).
"""

from __future__ import annotations

import dataclasses
from fractions import Fraction

import torch

from . import lrm as L


def capacity(T: int, E: int, k: int, cf: Fraction) -> int:
    """C = floor(CF * T k / E), as the library computes it (lrm_capacity)."""
    return L.lrm_capacity(L.dims_of(T, E, k, 8, 8), cf)


def max_retained_rows(T: int, E: int, k: int, cf: Fraction, rho: Fraction) -> int:
    """Upper bound of sum_e ceil(rho * min(n_e, C)) over any routing, as the
    library computes it (lrm_max_rows)."""
    return L.lrm_max_rows(L.dims_of(T, E, k, 8, 8), cf, rho)


@dataclasses.dataclass
class Fc1Buffers:
    """Device buffers of the FC1 side (allocated on first use)."""

    ones: torch.Tensor  # [N] fp32: unit gate weights for compacting the FC1 inputs
    xc: torch.Tensor  # [rows, h] bf16: compacted expert inputs
    abc: torch.Tensor  # [rows, 2I] bf16: compacted saved FC1 outputs
    dh1: torch.Tensor  # [rows, 2I] bf16: FC1 output gradient
    dxc: torch.Tensor  # [rows, h] bf16: FC1 input gradient per retained row
    dW1: torch.Tensor  # [E, 2I, h] fp32
    dx: torch.Tensor  # [T, h] bf16: input gradient of every token
    ws: torch.Tensor  # pair -> row map of lrm_combine_rows


@dataclasses.dataclass
class Buffers:
    counts: torch.Tensor
    offsets: torch.Tensor
    bucket: torch.Tensor
    P: torch.Tensor
    f: torch.Tensor
    quota: torch.Tensor
    summary: torch.Tensor
    ws_route: torch.Tensor
    ws_select: torch.Tensor
    score: torch.Tensor
    sel_offsets: torch.Tensor
    sel_ids: torch.Tensor
    delta_c: torch.Tensor
    phi_c: torch.Tensor
    alpha_c: torch.Tensor
    dphi_c: torch.Tensor
    dW: torch.Tensor


class Recalibration:
    """Device buffers plus the library calls of one recalibration step."""

    def __init__(self, T, E, k, h, I, cf=Fraction(5, 4), rho=Fraction(3, 4), device=0, max_rows=None):
        self.T, self.E, self.k, self.h, self.I = int(T), int(E), int(k), int(h), int(I)
        self.N = self.T * self.k
        self.cf = Fraction(cf)
        self.rho = Fraction(rho)
        self.device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        self.dims = L.dims_of(T, E, k, h, I)
        self.ctx = L.lrm_create(self.device.index or 0)
        self.C = L.lrm_capacity(self.dims, self.cf)
        self.max_rows = L.lrm_max_rows(self.dims, self.cf, self.rho) if max_rows is None else int(max_rows)
        dev = self.device
        ws_bytes = L.lrm_workspace_size(self.ctx, L.LRM_OP_ROUTE_STATS, self.dims)
        ws_sel = L.lrm_workspace_size(self.ctx, L.LRM_OP_SELECT, self.dims)
        i32 = dict(dtype=torch.int32, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        bf = dict(dtype=torch.bfloat16, device=dev)
        R = max(1, self.max_rows)
        self.buf = Buffers(
            counts=torch.empty(E, **i32),
            offsets=torch.empty(E + 1, **i32),
            bucket=torch.empty(max(1, self.N), **i32),
            P=torch.empty(E, **f32),
            f=torch.empty(E, **f32),
            quota=torch.empty(E, **i32),
            summary=torch.zeros(L.SUMMARY_BYTES, dtype=torch.uint8, device=dev),
            ws_route=torch.empty(max(256, ws_bytes), dtype=torch.uint8, device=dev),
            ws_select=torch.empty(max(256, ws_sel), dtype=torch.uint8, device=dev),
            score=torch.empty(max(1, self.N), **f32),
            sel_offsets=torch.empty(E + 1, **i32),
            sel_ids=torch.empty(R, **i32),
            delta_c=torch.empty(R, h, **bf),
            phi_c=torch.empty(R, I, **bf),
            alpha_c=torch.empty(R, **f32),
            dphi_c=torch.empty(R, I, **bf),
            dW=torch.empty(E, h, I, **f32),
        )
        self.ws_bytes = self.buf.ws_route.numel()

    def close(self):
        if getattr(self, "ctx", None):
            L.lrm_destroy(self.ctx)
            self.ctx = None

    def __del__(self):  # pragma: no cover - best effort
        try:
            self.close()
        except Exception:
            pass

    # -- the steps -----------------------------------------------------------

    def route_stats(self, logits, expert_idx, stream=None, quota_override=None, counted=None):
        """Step 1.  `counted` (``Router.counted``) leaves the tokens that the
        router did not count out of it, and so out of the whole path."""
        b = self.buf
        out = (b.counts, b.offsets, b.bucket, b.P, b.f, b.quota, b.summary, b.ws_route, self.ws_bytes, stream)
        if counted is None:
            L.lrm_route_stats(self.ctx, logits, expert_idx, self.dims, self.cf, self.rho, *out)
        else:
            L.lrm_route_stats_counted(self.ctx, logits, expert_idx, *counted, self.dims, self.cf, self.rho, *out)
        if quota_override is not None:
            b.quota.copy_(quota_override)

    def score(self, g, phi, alpha, stream=None, metric: int = L.METRIC_LRM, seed: int = 0):
        """Step 2.  `metric` selects the LRM (default) or one of the ablation's
        alternatives (gradient L2, gradient L1, seeded random)."""
        if metric == L.METRIC_LRM:
            L.lrm_score(self.ctx, g, phi, alpha, self.dims, self.buf.score, stream)
        else:
            L.lrm_score_metric(self.ctx, metric, g, phi, alpha, self.dims, seed, self.buf.score, stream)

    def select(self, stream=None, score=None):
        b = self.buf
        L.lrm_select(self.ctx, b.score if score is None else score, b.offsets, b.bucket, b.quota, self.dims,
                     self.max_rows, b.sel_offsets, b.sel_ids, b.ws_select, b.ws_select.numel(), stream)

    def compact(self, g, phi, alpha, stream=None):
        b = self.buf
        L.lrm_compact(self.ctx, g, phi, alpha, b.sel_offsets, b.sel_ids, self.dims, self.max_rows, b.delta_c,
                      b.phi_c, b.alpha_c, stream)

    def dgrad(self, W, stream=None):
        b = self.buf
        L.lrm_grouped_dgrad(self.ctx, b.delta_c, W, b.sel_offsets, self.dims, self.max_rows, b.dphi_c, stream)

    def dgrad_scatter(self, W, dphi_rows, stream=None, zero_dropped: bool = True):
        """Step 5a with the inverse mapping: the input gradient of every
        retained pair goes to its row of `dphi_rows` ([N, I] bf16, the layout
        of phi); with `zero_dropped` the rows of the other pairs become zeros."""
        b = self.buf
        L.lrm_grouped_dgrad_scatter(self.ctx, b.delta_c, W, b.sel_offsets, b.sel_ids, self.dims, self.max_rows,
                                    dphi_rows, stream)
        if zero_dropped:
            if getattr(self, "_ws_zero", None) is None:
                nbytes = L.lrm_workspace_size(self.ctx, L.LRM_OP_ZERO_DROPPED, self.dims)
                self._ws_zero = torch.empty(max(nbytes, 4), dtype=torch.uint8, device=self.buf.dW.device)
            L.lrm_zero_dropped_rows(self.ctx, b.sel_offsets, b.sel_ids, self.dims, self.max_rows, dphi_rows,
                                    self._ws_zero, self._ws_zero.numel(), stream)

    def fc1_backward(self, x, ab, W1, stream=None):
        """The FC1 side of the expert backward on the retained pairs (SwiGLU
        read), after the FC2 steps: the compacted FC1 inputs, dh1 from the FC2
        input gradient, the FC1 input gradient of every retained row, the FC1
        weight gradient and the input gradient of every token.  x [T, h] and
        ab [N, 2I] bf16 (expert inputs, saved [a | b]), W1 [E, 2I, h] bf16.
        Results: self.fc1.dW1 [E, 2I, h] fp32 and self.fc1.dx [T, h] bf16."""
        f = self._fc1_buffers()
        b = self.buf
        T, E, k, h, I = self.dims.T, self.dims.E, self.dims.k, self.dims.h, self.dims.I
        d_in = L.Dims(T, E, k, h, 2 * I)  # compact: token rows of width h, pair rows of width 2I
        d_fc1 = L.Dims(T, E, k, 2 * I, h)  # the FC2 kernels with K = 2I and output width h
        L.lrm_compact(self.ctx, x, ab, f.ones, b.sel_offsets, b.sel_ids, d_in, self.max_rows, f.xc, f.abc, None,
                      stream)
        L.lrm_swiglu_backward(self.ctx, b.dphi_c, f.abc, b.sel_offsets, self.dims, self.max_rows, f.dh1, stream)
        L.lrm_grouped_dgrad(self.ctx, f.dh1, W1, b.sel_offsets, d_fc1, self.max_rows, f.dxc, stream)
        L.lrm_grouped_wgrad(self.ctx, f.dh1, f.xc, b.sel_offsets, d_fc1, self.max_rows, 0, f.dW1, stream)
        L.lrm_combine_rows(self.ctx, f.dxc, b.sel_offsets, b.sel_ids, self.dims, self.max_rows, h, f.dx, f.ws,
                           f.ws.numel(), stream)

    def _fc1_buffers(self):
        if getattr(self, "fc1", None) is None:
            T, E, k, h, I = self.dims.T, self.dims.E, self.dims.k, self.dims.h, self.dims.I
            dev = self.buf.dW.device
            bf = dict(dtype=torch.bfloat16, device=dev)
            rows = max(self.max_rows, 1)
            ws = L.lrm_workspace_size(self.ctx, L.LRM_OP_COMBINE, self.dims)
            self.fc1 = Fc1Buffers(
                ones=torch.ones(T * k, dtype=torch.float32, device=dev),
                xc=torch.empty(rows, h, **bf), abc=torch.empty(rows, 2 * I, **bf),
                dh1=torch.empty(rows, 2 * I, **bf), dxc=torch.empty(rows, h, **bf),
                dW1=torch.empty(E, 2 * I, h, dtype=torch.float32, device=dev), dx=torch.empty(T, h, **bf),
                ws=torch.empty(max(ws, 4), dtype=torch.uint8, device=dev))
        return self.fc1

    def gate_grad(self, stream=None):
        """alpha_u dL/dalpha_u of every pair in ``self.dgate`` ([N] fp32, 0 for
        pairs that were not retained), after dgrad and compact: what
        ``Router.backward`` takes."""
        b = self.buf
        L.lrm_gate_grad(self.ctx, b.dphi_c, b.phi_c, b.sel_offsets, b.sel_ids, self.dims, self.max_rows,
                        self._dgate_buffer(), stream)
        return self.dgate

    def _dgate_buffer(self):
        if getattr(self, "dgate", None) is None:
            self.dgate = torch.empty(max(1, self.N), dtype=torch.float32, device=self.buf.dW.device)[: self.N]
        return self.dgate

    def wgrad(self, stream=None, accumulate=0):
        b = self.buf
        L.lrm_grouped_wgrad(self.ctx, b.delta_c, b.phi_c, b.sel_offsets, self.dims, self.max_rows, accumulate,
                            b.dW, stream)

    def wgrad_bf16(self, stream=None, accumulate=0):
        """Step 5b with the weight gradient stored as bf16 in ``self.dW_bf16``
        ([E, h, I], allocated on first use)."""
        b = self.buf
        if getattr(self, "dW_bf16", None) is None:
            self.dW_bf16 = torch.zeros(self.E, self.h, self.I, dtype=torch.bfloat16, device=b.dW.device)
        L.lrm_grouped_wgrad_bf16(self.ctx, b.delta_c, b.phi_c, b.sel_offsets, self.dims, self.max_rows, accumulate,
                                 self.dW_bf16, stream)

    def backward_steps(self, g, phi, alpha, W, stream=None, metric: int = L.METRIC_LRM, seed: int = 0,
                       dw_bf16: bool = False):
        """score -> select -> compact -> dgrad -> wgrad (quotas already set);
        with `dw_bf16` the weight gradient goes to ``self.dW_bf16``."""
        self.score(g, phi, alpha, stream, metric=metric, seed=seed)
        self.select(stream)
        self.compact(g, phi, alpha, stream)
        self.dgrad(W, stream)
        if dw_bf16:
            self.wgrad_bf16(stream)
        else:
            self.wgrad(stream)

    def run(self, logits, expert_idx, g, phi, alpha, W, stream=None, dw_bf16: bool = False, side_stream=None,
            counted=None):
        """The whole path, enqueued on one stream.  Route statistics and score
        read disjoint inputs, so with `side_stream` (a torch stream; `stream`
        must then be a torch stream or None) route statistics run on it beside
        score, and select waits for both.  `counted`: as in route_stats."""
        if side_stream is None:
            self.route_stats(logits, expert_idx, stream, counted=counted)
            self.backward_steps(g, phi, alpha, W, stream, dw_bf16=dw_bf16)
            return
        main = torch.cuda.current_stream(self.device) if stream is None else stream
        if not isinstance(main, torch.cuda.Stream) or not isinstance(side_stream, torch.cuda.Stream):
            raise TypeError("run(side_stream=...) needs torch streams for both branches")
        fork = torch.cuda.Event()
        fork.record(main)
        side_stream.wait_event(fork)
        self.route_stats(logits, expert_idx, side_stream, counted=counted)
        self.score(g, phi, alpha, main)
        join = torch.cuda.Event()
        join.record(side_stream)
        main.wait_event(join)
        self.select(main)
        self.compact(g, phi, alpha, main)
        self.dgrad(W, main)
        if dw_bf16:
            self.wgrad_bf16(main)
        else:
            self.wgrad(main)

    def summary(self) -> dict:
        raw = bytes(self.buf.summary.cpu().numpy().tobytes())
        s = L.RouteSummary.from_buffer_copy(raw)
        return {name: getattr(s, name) for name, _ in L.RouteSummary._fields_}

    def device_status(self, stream=None) -> int:
        return L.lrm_get_device_status(self.ctx, stream)


class StepGraph:
    """The whole step (route stats through the weight gradient) captured once
    as a CUDA graph over fixed device buffers: one launch per step instead of
    one call per kernel, so the host issues nothing per kernel.  Route
    statistics form a branch of their own beside score (they read disjoint
    inputs), joined before select.  The graph reads the tensors it was
    captured with; a caller feeds a new batch by writing into them
    (``copy_``) before ``replay``.  The first, eager run does each kernel's
    one-time set-up (function attributes, occupancy), which must not happen
    inside a capture."""

    def __init__(self, rec: "Recalibration", logits, expert_idx, g, phi, alpha, W, dw_bf16: bool = False):
        self.rec = rec
        self.inputs = dict(logits=logits, expert_idx=expert_idx, g=g, phi=phi, alpha=alpha, W=W)
        dev = rec.device
        side = torch.cuda.Stream(dev)
        branch = torch.cuda.Stream(dev)  # the route statistics branch
        side.wait_stream(torch.cuda.current_stream(dev))
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            rec.run(logits, expert_idx, g, phi, alpha, W, stream=side, dw_bf16=dw_bf16, side_stream=branch)
            side.synchronize()
            with torch.cuda.graph(self.graph, stream=side):
                rec.run(logits, expert_idx, g, phi, alpha, W, stream=side, dw_bf16=dw_bf16, side_stream=branch)
        torch.cuda.current_stream(dev).wait_stream(side)

    def replay(self) -> None:
        """Enqueue one step on the current stream."""
        self.graph.replay()


_DTYPES = {torch.float32: L.DTYPE_F32, torch.bfloat16: L.DTYPE_BF16}


def _require(t, name, dtype, shape, device):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _stream_of(owner, stream):
    """The raw handle of `stream` (None: the current one) for a call that uses
    ``owner._held()``.  The first call on a stream that is not in
    ``owner._streams`` tells the allocator, so that their memory is not given
    away while that stream still works on it.  A raw handle's owner keeps them
    alive instead: the allocator may not use it once it has been destroyed."""
    raw = L._stream(stream)
    if raw not in owner._streams:
        owner._streams.add(raw)
        if not isinstance(stream, int):
            s = torch.cuda.current_stream() if stream is None else stream
            for t in owner._held():
                t.record_stream(s)
    return raw


def _keep(buffer, t, stream):
    """A copy of `t` in `buffer`, on `stream` (a torch stream, a raw handle or None)."""
    if isinstance(stream, int):  # 0, the default stream's handle, would stand for a new stream
        dev = buffer.device
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):  # None: as it is
        buffer.copy_(t)


class Router:
    """The router of one layer shape through the C ABI: gates and balance loss
    of a batch of logits (lrm_router_forward) and the logits' gradient
    (lrm_router_backward).  The outputs of ``forward`` are the buffers
    ``expert_idx`` [T, k], ``alpha`` [T*k], ``row_stats`` [T, 2], ``counts``,
    ``f``, ``P`` [E], ``losses`` (fp32 [3]: loss, aux, z) and ``tokens`` (int32
    [1]); ``backward`` reads them and writes ``dlogits`` [T, E]."""

    def __init__(self, T, E, k, renorm: bool = True, aux_coef: float = 0.0, z_coef: float = 0.0,
                 dtype=torch.float32, dlogits_dtype=None, device=0, ctx=None):
        self.T, self.E, self.k = int(T), int(E), int(k)
        self.renorm, self.aux_coef, self.z_coef = bool(renorm), float(aux_coef), float(z_coef)
        self.dtype = dtype
        self.dlogits_dtype = dtype if dlogits_dtype is None else dlogits_dtype
        if dtype not in _DTYPES or self.dlogits_dtype not in _DTYPES:
            raise ValueError("router logits and their gradient are float32 or bfloat16")
        self.device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        if self.device.index is None:  # "cuda": tensors name the device with its index
            self.device = torch.device(self.device.type, torch.cuda.current_device())
        self.dims = L.dims_of(T, E, k, 8, 8)
        self._own_ctx = ctx is None
        self.ctx = L.lrm_create(self.device.index or 0) if ctx is None else ctx
        i32 = dict(dtype=torch.int32, device=self.device)
        f32 = dict(dtype=torch.float32, device=self.device)
        self.expert_idx = torch.empty(self.T, self.k, **i32)
        self.alpha = torch.empty(self.T * self.k, **f32)
        self.row_stats = torch.empty(self.T, 2, **f32)
        self.counts = torch.empty(self.E, **i32)
        self.f = torch.empty(self.E, **f32)
        self.P = torch.empty(self.E, **f32)
        self._losses = torch.zeros(4, **f32)  # lrm_router_losses
        self.losses = self._losses[:3]
        self.tokens = self._losses.view(torch.int32)[3:]
        self.dlogits = torch.empty(self.T, self.E, dtype=self.dlogits_dtype, device=self.device)
        need = L.lrm_workspace_size(self.ctx, L.LRM_OP_ROUTER, self.dims)
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
        # the memory is the current stream's, where the fill and work on what it held before may be pending
        home = torch.cuda.current_stream(self.device)
        self._streams = {home.cuda_stream}
        if not torch.cuda.is_current_stream_capturing():
            home.synchronize()

    def _held(self):
        return (self.expert_idx, self.alpha, self.row_stats, self.counts, self.f, self.P, self._losses, self.dlogits,
                self.ws)

    def close(self):
        if self._own_ctx and getattr(self, "ctx", None):
            L.lrm_destroy(self.ctx)
        self.ctx = None

    def __del__(self):  # pragma: no cover - best effort
        try:
            self.close()
        except Exception:
            pass

    def forward(self, logits, valid=None, stream=None):
        """Gates, counts and losses of a batch; `valid` [T] uint8 leaves the
        tokens whose entry is 0 out of the counts and losses, with gate 0."""
        _require(logits, "logits", self.dtype, (self.T, self.E), self.device)
        if valid is not None:
            _require(valid, "valid", torch.uint8, (self.T,), self.device)
        L.lrm_router_forward(self.ctx, logits, _DTYPES[self.dtype], valid, self.dims, self.renorm, self.aux_coef,
                             self.z_coef, self.expert_idx, self.alpha, self.row_stats, self.counts, self.f, self.P,
                             self._losses, self.ws, self.ws.numel(), _stream_of(self, stream))

    @property
    def counted(self):
        """What ``Recalibration.run`` takes to leave out the tokens that the last ``forward`` did not count."""
        return self.row_stats, self._losses

    def backward(self, logits, dgate=None, f=None, stream=None):
        """The gradient of the loss (with its coefficients) and, given `dgate`
        [T*k] (alpha dL/dalpha of every pair, from ``Recalibration.gate_grad``),
        of the gates, with respect to the logits of the last ``forward``.  `f`
        [E] replaces the batch's own load fractions."""
        _require(logits, "logits", self.dtype, (self.T, self.E), self.device)
        if dgate is not None and (dgate.dtype != torch.float32 or dgate.numel() != self.T * self.k
                                  or dgate.device != self.device or not dgate.is_contiguous()):
            raise ValueError(f"dgate must hold {self.T * self.k} contiguous float32 values on {self.device}")
        if f is not None:
            _require(f, "f", torch.float32, (self.E,), self.device)
        L.lrm_router_backward(self.ctx, logits, _DTYPES[self.dtype], self.expert_idx, self.alpha, self.row_stats,
                              dgate, self.f if f is None else f, self._losses, self.dims, self.renorm, self.aux_coef,
                              self.z_coef, self.dlogits, _DTYPES[self.dlogits_dtype], _stream_of(self, stream))
        return self.dlogits

    def device_status(self, stream=None) -> int:
        return L.lrm_get_device_status(self.ctx, stream)


class _Operator:
    """Device buffers of a fixed shape beside the calls that use them, for one
    device; several may share a context."""

    def _open(self, device, ctx):
        self.device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        if self.device.index is None:  # "cuda": tensors name the device with its index
            self.device = torch.device(self.device.type, torch.cuda.current_device())
        self._own_ctx = ctx is None
        self.ctx = L.lrm_create(self.device.index or 0) if ctx is None else ctx

    def _made(self, *held):
        """After the buffers: their memory is the current stream's, where fills
        and work on what it held before may be pending."""
        self._buffers = tuple(t for t in held if t is not None)
        home = torch.cuda.current_stream(self.device)
        self._streams = {home.cuda_stream}
        if not torch.cuda.is_current_stream_capturing():
            home.synchronize()

    def _held(self):
        return self._buffers

    def device_status(self, stream=None) -> int:
        return L.lrm_get_device_status(self.ctx, stream)

    def close(self):
        if getattr(self, "_own_ctx", False) and getattr(self, "ctx", None):
            L.lrm_destroy(self.ctx)
        self.ctx = None

    def __del__(self):  # pragma: no cover - best effort
        try:
            self.close()
        except Exception:
            pass


class ExpertFFN(_Operator):
    """The forward of the routed experts, the gated feed-forward block
    W (silu(Wg x) * (Wu x)), for the pairs of a routing (lrm_ffn_up,
    lrm_ffn_down, lrm_ffn_combine): ``y`` [T, h] bf16, and what the backward
    reads: ``phi`` [N, I] and, unless `save` is False, ``ab`` [N, 2I]."""

    def __init__(self, T, E, k, h, I, save: bool = True, device=0, ctx=None):
        self.T, self.E, self.k, self.h, self.I = int(T), int(E), int(k), int(h), int(I)
        self.N = self.T * self.k
        self.dims = L.dims_of(T, E, k, h, I)
        self._open(device, ctx)
        bf = dict(dtype=torch.bfloat16, device=self.device)
        self.phi = torch.zeros(self.N, self.I, **bf)
        self.ab = torch.zeros(self.N, 2 * self.I, **bf) if save else None
        self.rows = torch.empty(self.N, self.h, **bf)
        self.y = torch.empty(self.T, self.h, **bf)
        self._made(self.phi, self.ab, self.rows, self.y)

    def forward(self, x, W1, W, offsets, ids, alpha, stream=None):
        """x [T, h], W1 [E, 2I, h] (gate rows, then up rows) and W [E, h, I] bf16;
        `offsets` [E+1] and `ids` int32: the pairs of every expert (the offsets and
        the bucket of route statistics); `alpha` [N] fp32: their gates, 0 for pairs
        that are in no segment."""
        bf = torch.bfloat16
        _require(x, "x", bf, (self.T, self.h), self.device)
        _require(W1, "W1", bf, (self.E, 2 * self.I, self.h), self.device)
        _require(W, "W", bf, (self.E, self.h, self.I), self.device)
        _require(offsets, "offsets", torch.int32, (self.E + 1,), self.device)
        if alpha.numel() != self.N:
            raise ValueError(f"alpha must hold {self.N} gates")
        _require(alpha, "alpha", torch.float32, tuple(alpha.shape), self.device)
        _require(ids, "ids", torch.int32, (ids.numel(),), self.device)
        raw = _stream_of(self, stream)
        n = min(self.N, ids.numel())
        L.lrm_ffn_up(self.ctx, x, W1, offsets, ids, self.dims, n, self.ab, self.phi, raw)
        L.lrm_ffn_down(self.ctx, self.phi, W, offsets, ids, self.dims, n, self.rows, raw)
        L.lrm_ffn_combine(self.ctx, self.rows, alpha, self.dims, self.y, raw)
        return self.y


class LayerNorm(_Operator):
    """Layer norm of `rows` rows of `width` values (lrm_layer_norm,
    lrm_layer_norm_backward).  ``forward`` writes ``y`` and ``stats`` (mean and
    1 / standard deviation of every row), ``backward`` reads them and writes
    ``dx``, ``dgamma`` and ``dbeta`` (fp32)."""

    def __init__(self, rows, width, dtype=torch.bfloat16, eps: float = 1e-5, device=0, ctx=None):
        self.rows, self.width, self.dtype, self.eps = int(rows), int(width), dtype, float(eps)
        if dtype not in _DTYPES:
            raise ValueError("layer norm takes float32 or bfloat16")
        if not self.eps >= 0:
            raise ValueError("eps must be at least 0")
        self._open(device, ctx)
        need = L.lrm_layer_norm_workspace(self.ctx, self.rows, self.width)
        f32 = dict(dtype=torch.float32, device=self.device)
        self.y = torch.empty(self.rows, self.width, dtype=dtype, device=self.device)
        self.stats = torch.empty(self.rows, 2, **f32)
        self.dx = torch.empty_like(self.y)
        self.dgamma, self.dbeta = torch.zeros(self.width, **f32), torch.zeros(self.width, **f32)
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
        self._made(self.y, self.stats, self.dx, self.dgamma, self.dbeta, self.ws)

    def _check(self, valid, **tensors):
        for name, t in tensors.items():
            _require(t, name, self.dtype, (self.rows, self.width), self.device)
            if t.data_ptr() % 16 != 0:
                raise ValueError(f"{name} must be 16-byte aligned")
        if valid is not None:
            _require(valid, "valid", torch.uint8, (self.rows,), self.device)

    def forward(self, x, gamma, beta, valid=None, stream=None):
        """`gamma`, `beta` [width] fp32; rows whose entry of `valid` [rows] uint8 is
        0 become zeros and take no part in the backward."""
        self._check(valid, x=x)
        for name, t in (("gamma", gamma), ("beta", beta)):
            _require(t, name, torch.float32, (self.width,), self.device)
        L.lrm_layer_norm(self.ctx, x, _DTYPES[self.dtype], gamma, beta, valid, self.rows, self.width, self.eps, self.y,
                         self.stats, _stream_of(self, stream))
        return self.y

    def backward(self, x, dy, gamma, valid=None, dres=None, stream=None):
        """The gradients of the last ``forward`` (x, gamma and valid as there) for the
        output's gradient `dy`; `dres` is added to dx: a residual connection's share."""
        self._check(valid, x=x, dy=dy, **({} if dres is None else dict(dres=dres)))
        _require(gamma, "gamma", torch.float32, (self.width,), self.device)
        L.lrm_layer_norm_backward(self.ctx, x, _DTYPES[self.dtype], dy, gamma, self.stats, valid, dres, self.rows,
                                  self.width, self.dx, self.dgamma, self.dbeta, self.ws, self.ws.numel(),
                                  _stream_of(self, stream))
        return self.dx


class Dropout(_Operator):
    """Dropout with a residual (lrm_dropout_add): the mask is drawn from `seed`,
    `offset` and the device counter ``step`` and never stored.  ``backward`` draws
    that of the last ``forward`` again as long as ``step`` is the same;
    ``advance`` counts it up (also in a captured graph).  Every layer needs a
    `seed` of its own: `offset` and ``step`` are added up, so that offsets one apart
    under one seed draw each other's masks a step later."""

    def __init__(self, p: float, seed: int = 0, offset: int = 0, device=0, ctx=None):
        if not 0.0 <= float(p) <= 1.0:
            raise ValueError("p must be in [0, 1]")
        self.p, self.seed, self.offset = float(p), int(seed) & ((1 << 64) - 1), int(offset) & ((1 << 64) - 1)
        self._open(device, ctx)
        self.step = torch.zeros(1, dtype=torch.int64, device=self.device)
        self._made(self.step)

    def _call(self, x, residual, out, stream):
        if x.dtype not in _DTYPES:
            raise ValueError("dropout takes float32 or bfloat16")
        for name, t in (("x", x), ("out", out)) + ((("residual", residual),) if residual is not None else ()):
            _require(t, name, x.dtype, tuple(x.shape), self.device)
        L.lrm_dropout_add(self.ctx, x, residual, _DTYPES[x.dtype], x.numel(), self.p, self.seed, self.offset, self.step,
                          out, _stream_of(self, stream))
        return out

    def forward(self, x, out, residual=None, stream=None):
        """out = residual + dropout(x); out may be x or residual itself."""
        return self._call(x, residual, out, stream)

    def backward(self, dy, out, stream=None):
        """out = dy where the forward kept the element, over 1 - p, and 0 elsewhere."""
        return self._call(dy, None, out, stream)

    def advance(self, stream=None) -> None:
        """A new mask from here on.  `stream`: a torch stream or None, the current one."""
        if stream is None:
            self.step.add_(1)
        else:
            _stream_of(self, stream)
            with torch.cuda.stream(stream):
                self.step.add_(1)


def _dense(t) -> bool:
    """Whether the tensor's elements fill its memory range, in any dimension order."""
    run = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != run:
            return False
        run *= size
    return True


def _same_order(a, b) -> bool:
    """Whether two tensors of one shape hold their elements in the same order: equal strides, but in
    dimensions of one element, where a stride leads nowhere."""
    return a.stride() == b.stride() or all(x == y for x, y, n in zip(a.stride(), b.stride(), a.shape) if n != 1)


_clip_contexts: dict[int, int] = {}


def _clip_context(device: int) -> int:
    """The context of a device's clips that were given none.  They can share
    one: a list has a status word of its own."""
    if device not in _clip_contexts:
        _clip_contexts[device] = L.lrm_create(device)
    return _clip_contexts[device]


class GradClip:
    """Global gradient norm and clipping over a fixed list of tensors
    (lrm_grad_norm, lrm_grad_clip).  `outs` receive the clipped values (the
    gradients themselves where it is None).  The tensors are fp32 or bf16, of
    any shape and dimension order, but dense: their elements fill their memory
    range; an output has its gradient's type, shape and strides.  The result's
    ``norm``, ``coef`` (fp32 [1]) and ``nonfinite`` (int32 [1]) stay on the
    device; ``nonfinite`` is not 0 for a step to skip: an element was infinite
    or NaN, or a bounded wait ran out (``device_status``)."""

    def __init__(self, grads, outs=None, ctx=None, stream=None):
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if len(outs) != len(grads):
            raise ValueError("as many outputs as gradients are wanted")
        if not grads:
            raise ValueError("no gradients")
        self.device = grads[0].device
        if self.device.type != "cuda":
            raise ValueError("gradients are float32 or bfloat16 CUDA tensors")
        spans, entries = [], []
        for g, o in zip(grads, outs):
            dtype = _DTYPES.get(g.dtype)
            if dtype is None:
                raise ValueError("gradients are float32 or bfloat16 CUDA tensors")
            if g.device != self.device or (o is not g and o.device != self.device):
                raise ValueError("all tensors must be on one device")
            n, src = g.numel(), g.data_ptr()
            dst = src
            if o is not g:
                if o.dtype != g.dtype or o.shape != g.shape or (n and not _same_order(o, g)):
                    raise ValueError("an output needs its gradient's type, shape and strides")
                dst = o.data_ptr()
            if n:
                if not g.is_contiguous() and not _dense(g):
                    raise ValueError("gradients and outputs must be dense in memory")
                size = n * g.element_size()
                spans.append((src, size))
                if dst != src:
                    spans.append((dst, size))
            entries.append((src, dst, n, dtype))
        spans.sort()
        if any(a + n > b for (a, n), (b, _) in zip(spans, spans[1:])):
            raise ValueError("gradients and outputs must not overlap")
        self.grads, self.outs = grads, outs  # kept alive: the list holds their addresses
        self.ctx = _clip_context(self.device.index or 0) if ctx is None else ctx
        tensors = L.tensor_array(entries)
        need = L.lrm_grad_table_size(tensors, len(grads))
        self.table = torch.empty(need, dtype=torch.uint8, device=self.device)
        self._stats = torch.zeros(3, dtype=torch.float32, device=self.device)  # lrm_grad_stats
        self.norm, self.coef = self._stats[0:1], self._stats[1:2]
        self.nonfinite = self._stats.view(torch.int32)[2:3]
        # the memory is the current stream's, where work on what it held before may be pending, and the fill is:
        # done before the table is written, on the stream that lrm_grad_list_create waits for
        home = torch.cuda.current_stream(self.device)
        self._streams = {home.cuda_stream}
        if stream is not None and L._stream(stream) != home.cuda_stream:
            home.synchronize()
        self.list = L.lrm_grad_list_create(self.ctx, tensors, len(grads), self.table, need, stream)

    def close(self):
        if getattr(self, "list", None):
            L.lrm_grad_list_destroy(self.list)
            self.list = None
        self.ctx = None

    def __del__(self):  # pragma: no cover - best effort
        try:
            self.close()
        except Exception:
            pass

    def _held(self):
        return self.table, self._stats, *self.grads, *self.outs

    def measure(self, stream=None) -> None:
        """norm of all gradients, nothing clipped."""
        L.lrm_grad_norm(self.ctx, self.list, self._stats, _stream_of(self, stream))

    def clip(self, max_norm: float, stream=None) -> None:
        """norm, and every gradient times min(1, max_norm / norm) into its output."""
        L.lrm_grad_clip(self.ctx, self.list, max_norm, self._stats, _stream_of(self, stream))

    def device_status(self, stream=None) -> int:
        """Flags (1 << code) that calls on this list raised on the device since the last read."""
        return L.lrm_grad_list_status(self.ctx, self.list, stream)


class TrainingStep:
    """One MoE layer's share of a training step: the router's forward, the
    recalibrated backward of the experts, the router's backward and the clipping
    of the layer's weight gradients, enqueued on one stream with no host
    synchronisation in between.

        route      logits -> ids, gates, balance and z losses (``router``)
        backward   route stats .. wgrad (``rec``), gate gradients, the FC1 side,
                   dlogits, the router's weight and input gradients (one
                   "expert" of E rows through the grouped GEMMs), clipping

    Results: ``rec.buf.dW`` [E, h, I], ``rec.fc1.dW1`` [E, 2I, h] and ``dWr`` [E, h]
    fp32, clipped in place to the norm `max_norm` over all three; ``rec.fc1.dx``
    and ``dxr`` [T, h] bf16, the token gradients through the experts and through
    the router; ``clip.norm``, ``clip.coef``, ``clip.nonfinite``.  E is a multiple
    of 8 (the grouped GEMMs' row width for the router's weight [E, h])."""

    def __init__(self, T, E, k, h, I, cf=Fraction(5, 4), rho=Fraction(3, 4), aux_coef: float = 0.01,
                 z_coef: float = 0.001, max_norm: float = 1.0, device=0):
        if int(E) % 8 != 0:
            raise ValueError("the router's weight gradient needs a multiple of 8 experts")
        if not max_norm >= 0:
            raise ValueError("max_norm must be at least 0")
        self.rec = Recalibration(T, E, k, h, I, cf, rho, device=device)
        dev = self.rec.device
        self.max_norm = float(max_norm)
        self.router = Router(T, E, k, True, aux_coef, z_coef, dtype=torch.float32, dlogits_dtype=torch.bfloat16,
                             device=dev, ctx=self.rec.ctx)
        self.dWr = torch.zeros(E, h, dtype=torch.float32, device=dev)
        self.dxr = torch.zeros(T, h, dtype=torch.bfloat16, device=dev)
        self._dims_r = L.dims_of(T, 1, 1, E, h)  # the router as one expert: rows of width E, weight [E, h]
        self._segment = torch.tensor([0, T], dtype=torch.int32, device=dev)
        self._masked = False  # whether the last route had a mask
        self._x = None  # x with zeros in the rows of padding, made for the first masked batch
        # every buffer of the step is made before the clip's list, which waits for the current stream: what is pending
        # there on memory that they reuse, and their fills, do not come after another stream's step
        self.rec._dgate_buffer()
        self.clip = GradClip([self.rec.buf.dW, self.rec._fc1_buffers().dW1, self.dWr], ctx=self.rec.ctx)
        self._streams = {torch.cuda.current_stream(dev).cuda_stream}

    def _held(self):
        rec = self.rec
        held = (*vars(rec.buf).values(), *vars(rec.fc1).values(), rec.dgate, self.dWr, self.dxr, self._segment)
        return held if self._x is None else (*held, self._x)

    def route(self, logits, valid=None, stream=None):
        """Ids and gates of the batch (``router.expert_idx``, ``router.alpha``) and its losses.  The tokens
        that `valid` leaves out take no part in the backward either: capacity, quotas, selection and gradients
        are those of a batch without them, and their rows of logits, g, phi, x and ab may hold anything."""
        self._masked = valid is not None
        if self._masked and self._x is None:
            self._x = torch.empty(self.rec.T, self.rec.h, dtype=torch.bfloat16, device=self.dWr.device)
            if not torch.cuda.is_current_stream_capturing():  # work on what the memory held before may be pending
                torch.cuda.current_stream(self._x.device).synchronize()
            self._streams = {torch.cuda.current_stream(self._x.device).cuda_stream}  # the others do not know it yet
        _stream_of(self, stream)
        self.router.forward(logits, valid, stream)

    def backward(self, logits, g, phi, W, x, ab, W1, Wr, stream=None):
        """The backward of the batch that ``route`` saw last.  g [T, h] the layer
        output's gradient, phi [N, I] and ab [N, 2I] the saved FC2 input and FC1
        output of every pair, x [T, h] the layer's input (bf16); W [E, h, I],
        W1 [E, 2I, h], Wr [E, h] the weights (bf16)."""
        rec, r = self.rec, self.router
        _stream_of(self, stream)
        rec.run(logits, r.expert_idx, g, phi, r.alpha, W, stream, counted=r.counted)
        rec.gate_grad(stream)
        rec.fc1_backward(x, ab, W1, stream)
        r.backward(logits, rec.dgate, stream=stream)
        T = rec.T
        if self._masked:  # dlogits holds zeros there, whose products with NaN would not be zeros
            L.lrm_counted_rows(rec.ctx, x, r.row_stats, rec.dims, rec.h, self._x, stream)
            x = self._x
        L.lrm_grouped_wgrad(rec.ctx, r.dlogits, x, self._segment, self._dims_r, T, 0, self.dWr, stream)
        L.lrm_grouped_dgrad(rec.ctx, r.dlogits, Wr, self._segment, self._dims_r, T, self.dxr, stream)
        self.clip.clip(self.max_norm, stream)

    def device_status(self, stream=None) -> int:
        return self.rec.device_status(stream)

    def close(self):
        self.clip.close()
        self.router.close()
        self.rec.close()


class SublayerStep(TrainingStep):
    """The training step of a whole pre-norm MoE sublayer,
    out = x + dropout(experts(norm(x))), enqueued on one stream:

        normalize  x -> n, the layer norm's output (``norm``); the caller's router
                   product turns it into logits
        route      logits -> ids, gates, losses, and the pairs of every expert
        experts    n -> y (``ffn``), x + dropout(y) in ``out``; what the backward
                   needs of it is kept
        backward   the output's gradient -> the weights' gradients, clipped over
                   all of them, and ``norm.dx`` [T, h] bf16, that of x

    In the backward, lrm_ffn_backward takes the retained pairs from their output
    gradients to the first projections' and the gates' in one product.  Weight
    gradients: ``rec.buf.dW``, ``rec.fc1.dW1``, ``dWr``, ``norm.dgamma`` and
    ``norm.dbeta``.  ``drop.advance()`` draws a new mask for the next step, not
    before this one's backward; every layer needs a `seed` of its own.  The logits
    and `valid` are copied: their buffers may be another layer's by the time of
    the backward."""

    def __init__(self, T, E, k, h, I, cf=Fraction(5, 4), rho=Fraction(3, 4), aux_coef: float = 0.01,
                 z_coef: float = 0.001, max_norm: float = 1.0, p: float = 0.0, seed: int = 0, eps: float = 1e-5,
                 device=0):
        super().__init__(T, E, k, h, I, cf, rho, aux_coef, z_coef, max_norm, device)
        rec = self.rec
        dev, ctx = self.dWr.device, rec.ctx
        self.norm = LayerNorm(T, h, torch.bfloat16, eps, dev, ctx)
        self.ffn = ExpertFFN(T, E, k, h, I, device=dev, ctx=ctx)
        self.drop = Dropout(p, seed, device=dev, ctx=ctx)
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.out = torch.empty(T, h, **bf)
        self._g, self._dn = torch.empty(T, h, **bf), torch.empty(T, h, **bf)
        self._side = torch.empty(max(rec.max_rows, 1), 8, **bf)  # second operand of a compaction that has only one
        need = L.lrm_ffn_backward_workspace(ctx, rec.dims, rec.max_rows)
        self._ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        # what the backward reads of the forward's inputs: the caller's buffers may hold another layer's by then
        self._logits = torch.empty(T, E, dtype=torch.float32, device=dev)
        self._valid = torch.empty(T, dtype=torch.uint8, device=dev)
        self._padded = self._routed = False
        self.clip.close()
        self.clip = GradClip([rec.buf.dW, rec.fc1.dW1, self.dWr, self.norm.dgamma, self.norm.dbeta], ctx=ctx)

    def _held(self):
        return *super()._held(), self.out, self._g, self._dn, self._side, self._ws, self._logits, self._valid

    def normalize(self, x, gamma, beta, valid=None, stream=None):
        """The layer norm of x [T, h] bf16; rows that `valid` leaves out become zeros."""
        _stream_of(self, stream)
        self.norm.forward(x, gamma, beta, valid, stream)
        self._padded = valid is not None
        if self._padded:
            _keep(self._valid, valid, stream)
        return self.norm.y

    def route(self, logits, valid=None, stream=None):
        """As in TrainingStep (`valid` as given to ``normalize``), and the routed pairs by expert."""
        _stream_of(self, stream)
        self.router.forward(logits, valid, stream)  # padding needs no more here: its rows of n are zeros
        _keep(self._logits, logits, stream)
        self._routed = True
        self.rec.route_stats(logits, self.router.expert_idx, stream, counted=self.router.counted)

    def experts(self, x, W1, W, stream=None):
        """out = x + dropout(y), y the gated sum of the experts' outputs for the normalised rows."""
        b = self.rec.buf
        _stream_of(self, stream)
        y = self.ffn.forward(self.norm.y, W1, W, b.offsets, b.bucket[: self.rec.N], self.router.alpha, stream)
        return self.drop.forward(y, self.out, x, stream)

    def backward(self, dout, x, W, W1, Wr, gamma, stream=None):
        """For dout [T, h] bf16, the gradient of ``out``; x, W [E, h, I], W1 [E, 2I, h] and gamma as in the
        forward, Wr [E, h] bf16."""
        rec = self.rec
        T, E, k, h, I = rec.T, rec.E, rec.k, rec.h, rec.I
        if not self._routed:
            raise ValueError("the backward of a batch needs its forward")
        # all of them before the first call: the products take shapes from the layer, not from the tensors
        for name, t, shape in (("dout", dout, (T, h)), ("x", x, (T, h)), ("W", W, (E, h, I)), ("W1", W1, (E, 2 * I, h)),
                               ("Wr", Wr, (E, h))):
            _require(t, name, torch.bfloat16, shape, self.dWr.device)
        _require(gamma, "gamma", torch.float32, (h,), self.dWr.device)
        _stream_of(self, stream)
        r, f, b = self.router, rec.fc1, rec.buf
        n, R = self.norm.y, rec.max_rows
        self.drop.backward(dout, self._g, stream)
        rec.score(self._g, self.ffn.phi, r.alpha, stream)
        rec.select(stream)
        rec.compact(self._g, self.ffn.phi, r.alpha, stream)
        L.lrm_ffn_backward(rec.ctx, b.delta_c, W, self.ffn.ab, b.sel_offsets, b.sel_ids, rec.dims, R, f.dh1, rec.dgate,
                           self._ws, self._ws.numel(), stream)
        rec.wgrad(stream)
        L.lrm_compact(rec.ctx, n, self.ffn.phi, f.ones, b.sel_offsets, b.sel_ids, L.Dims(T, E, k, h, 8), R, f.xc,
                      self._side, None, stream)
        d_fc1 = L.Dims(T, E, k, 2 * I, h)
        L.lrm_grouped_dgrad(rec.ctx, f.dh1, W1, b.sel_offsets, d_fc1, R, f.dxc, stream)
        L.lrm_grouped_wgrad(rec.ctx, f.dh1, f.xc, b.sel_offsets, d_fc1, R, 0, f.dW1, stream)
        L.lrm_combine_rows(rec.ctx, f.dxc, b.sel_offsets, b.sel_ids, rec.dims, R, h, f.dx, f.ws, f.ws.numel(), stream)
        r.backward(self._logits, rec.dgate, stream=stream)
        L.lrm_grouped_wgrad(rec.ctx, r.dlogits, n, self._segment, self._dims_r, T, 0, self.dWr, stream)
        L.lrm_grouped_dgrad(rec.ctx, r.dlogits, Wr, self._segment, self._dims_r, T, self.dxr, stream)
        # the two gradients of n, through the experts and through the router
        L.lrm_dropout_add(rec.ctx, f.dx, self.dxr, L.DTYPE_BF16, T * h, 0.0, 0, 0, None, self._dn, stream)
        self.norm.backward(x, self._dn, gamma, self._valid if self._padded else None, dout, stream)
        self.clip.clip(self.max_norm, stream)
        return self.norm.dx

    def close(self):
        for part in (self.norm, self.ffn, self.drop):
            part.close()
        super().close()


def to_device_inputs(inp, device="cuda"):
    """Copy a workloads.Inputs record to device tensors (bf16 bits viewed as bf16)."""
    import numpy as np

    def bf(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).to(device)

    return dict(
        logits=torch.from_numpy(inp.logits).to(device),
        expert_idx=torch.from_numpy(inp.expert_idx).to(device),
        alpha=torch.from_numpy(inp.alpha).to(device),
        g=bf(inp.g),
        phi=bf(inp.phi),
        W=bf(inp.W),
    )


INPUT_NAMES = ("logits", "expert_idx", "g", "phi", "alpha", "W")
OUTPUT_NAMES = ("dW", "dphi_c", "sel_offsets", "sel_ids", "summary")


class HostPipeline:
    """The path over a sequence of host-resident layer batches, with the
    host->device copies of one batch and the device->host copies of the one
    before it running on their own streams while a third computes.

    Two slots (each a ``Recalibration`` with its own device inputs and
    outputs) alternate; events order every reuse: a slot's inputs are not
    overwritten before its last compute has read them, and its outputs are
    not recomputed before they were copied out.  Of the compacted input
    gradient only the retained rows go back: a batch's small outputs (the
    selection offsets first) are copied right after its compute, and its
    ``dphi_c`` rows are copied, exactly ``sel_offsets[E]`` of them, when the
    next batch is submitted (or at ``synchronize``), once that count is on
    the host.  ``submit`` otherwise only enqueues; the caller keeps each host
    buffer untouched until ``synchronize`` (or until two later submits have
    returned).  Host buffers should be pinned for the copies to run
    asynchronously.
    """

    SMALL = ("sel_offsets", "summary", "sel_ids")

    def __init__(self, T, E, k, h, I, cf=Fraction(5, 4), rho=Fraction(3, 4), device=0):
        self.recs = [Recalibration(T, E, k, h, I, cf, rho, device=device) for _ in range(2)]
        dev = self.recs[0].device
        self.device = dev
        self.E = int(E)
        N = int(T) * int(k)
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.dev_in = [dict(logits=torch.empty(T, E, dtype=torch.float32, device=dev),
                            expert_idx=torch.empty(T, k, dtype=torch.int32, device=dev),
                            g=torch.empty(T, h, **bf), phi=torch.empty(N, I, **bf),
                            alpha=torch.empty(N, dtype=torch.float32, device=dev), W=torch.empty(E, h, I, **bf))
                       for _ in range(2)]
        self.s_in, self.s_comp, self.s_out = (torch.cuda.Stream(dev) for _ in range(3))
        self.ev_in, self.ev_comp, self.ev_out, self.ev_small = (
            [torch.cuda.Event() for _ in range(2)] for _ in range(4))
        self.submitted = 0
        self.pending = None  # (slot, host_out) whose dphi_c rows are still to be copied
        self.d2h_bytes = 0  # device -> host bytes enqueued so far

    def _flush(self) -> None:
        if self.pending is None:
            return
        s, host_out = self.pending
        self.pending = None
        self.ev_small[s].synchronize()  # the batch's selection offsets are on the host
        rows = int(host_out["sel_offsets"][self.E])
        rows = max(0, min(rows, host_out["dphi_c"].shape[0]))
        with torch.cuda.stream(self.s_out):
            if rows:
                host_out["dphi_c"][:rows].copy_(self.recs[s].buf.dphi_c[:rows], non_blocking=True)
        self.d2h_bytes += rows * host_out["dphi_c"].stride(0) * host_out["dphi_c"].element_size()
        self.ev_out[s].record(self.s_out)

    def submit(self, host_in: dict, host_out: dict) -> int:
        """Enqueue one batch: copy `host_in` (the six inputs, by name) in, run
        the path, copy the results into `host_out` (dW, the retained rows of
        dphi_c, sel_offsets, sel_ids, summary).  Returns the slot used."""
        s = self.submitted % 2
        rec, din = self.recs[s], self.dev_in[s]
        reuse = self.submitted >= 2
        if reuse:
            self.s_in.wait_event(self.ev_comp[s])
        with torch.cuda.stream(self.s_in):
            for name in INPUT_NAMES:
                din[name].copy_(host_in[name], non_blocking=True)
        self.ev_in[s].record(self.s_in)
        self.s_comp.wait_event(self.ev_in[s])
        if reuse:
            self.s_comp.wait_event(self.ev_out[s])
        rec.run(din["logits"], din["expert_idx"], din["g"], din["phi"], din["alpha"], din["W"], stream=self.s_comp)
        self.ev_comp[s].record(self.s_comp)
        # the previous batch's retained rows go out first, then this batch's outputs
        self._flush()
        self.s_out.wait_event(self.ev_comp[s])
        b = rec.buf
        with torch.cuda.stream(self.s_out):
            for name in self.SMALL:
                host_out[name].copy_(getattr(b, name), non_blocking=True)
            self.ev_small[s].record(self.s_out)
            host_out["dW"].copy_(b.dW, non_blocking=True)
        self.d2h_bytes += sum(host_out[n].numel() * host_out[n].element_size() for n in self.SMALL + ("dW",))
        self.pending = (s, host_out)
        self.submitted += 1
        return s

    def host_outputs(self, pin: bool = True) -> dict:
        """A set of host buffers shaped for ``submit``'s results."""
        b = self.recs[0].buf
        out = {name: torch.empty_like(getattr(b, name), device="cpu") for name in OUTPUT_NAMES}
        return {k2: v.pin_memory() for k2, v in out.items()} if pin else out

    def synchronize(self) -> None:
        self._flush()
        for st in (self.s_in, self.s_comp, self.s_out):
            st.synchronize()

    def device_status(self) -> int:
        flags = 0
        for rec in self.recs:
            flags |= rec.device_status(self.s_comp)
        self.s_comp.synchronize()
        return flags

    def close(self) -> None:
        for rec in self.recs:
            rec.close()
