"""Layer norm's forward and backward against the fp64 oracle.

Tolerances, per value, u = 2^-24.  A row's sums: at most 72 serial additions a
thread and trees over its warps and their sums, so A = 90 u of the sum of the
magnitudes.  Stored types add their half step (2^-8 for bf16, u for fp32).  The
weights' gradients add up a thread's rows, a block's warps and the blocks:
(rows / 128 + 64) u of the magnitudes, beside xhat's own error."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import built_library, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
A = 90 * U
STORE = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    built_library()


@pytest.fixture(scope="module")
def ctx():
    from backward_token_expert_gb300 import lrm as L

    c = L.lrm_create(0)
    yield c
    L.lrm_destroy(c)


def _code(dtype):
    from backward_token_expert_gb300 import lrm as L

    return L.DTYPE_F32 if dtype == torch.float32 else L.DTYPE_BF16


def _np(t):
    return t.double().cpu().numpy()


def _placed(values, dtype, shift):
    """The values in device memory `shift` elements past a 16-byte boundary, guards around them."""
    n = values.numel()
    buf = torch.full((shift + n + 64,), 7.0, dtype=dtype, device="cuda")
    view = buf[shift:shift + n].view(values.shape)
    view.copy_(values)
    return buf, view


def _untouched(buf, shift, n):
    return bool((buf[:shift] == 7.0).all() and (buf[shift + n:] == 7.0).all())


SHAPES = [  # rows, width, shift of the tensors
    (1, 1, 0), (3, 2, 1), (5, 8, 0), (7, 16, 3), (33, 31, 0), (64, 64, 0), (129, 257, 5), (40, 256, 0), (300, 1000, 0),
    (301, 1497, 0), (500, 2048, 0), (9, 2048, 0), (150, 2050, 0), (70, 4104, 0), (60, 5120, 0), (33, 8191, 2), (20, 8192, 0),
    (17, 16384, 0), (11, 16383, 1), (5000, 24, 0), (3001, 100, 0), (1, 2048, 0), (2, 5, 0),
    # several rows of several warps a block in the backward
    (3000, 1497, 3), (2777, 704, 0), (1600, 2048, 0), (700, 6001, 1)]


def _inputs(rows, width, dtype, seed, masked):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, width)) * (0.2 + 3 * rng.random((rows, 1))) + rng.standard_normal((rows, 1))
    x[:, ::7] *= 9.0
    valid = (rng.random(rows) < 0.7).astype(np.uint8) if masked else None
    t = lambda a: torch.from_numpy(a.astype(np.float32)).to(dtype)  # noqa: E731
    x, dy, dres = t(x), t(rng.standard_normal((rows, width))), t(rng.standard_normal((rows, width)))
    if masked:
        for a in (x, dy, dres):
            a[valid == 0] = float("nan")
    gamma = rng.standard_normal(width).astype(np.float32)
    beta = rng.standard_normal(width).astype(np.float32)
    return x, dy, dres, gamma, beta, valid


@pytest.mark.parametrize("rows,width,shift", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masked", [False, True])
def test_forward_and_backward(ctx, rows, width, shift, dtype, masked):
    from backward_token_expert_gb300 import lrm as L

    x, dy, dres, gamma, beta, valid = _inputs(rows, width, dtype, rows + width, masked)
    use_res = (rows + width) % 2 == 0
    n = rows * width
    zero = torch.zeros(rows, width)
    (_, xd), (ybuf, y) = _placed(x, dtype, shift), _placed(zero, dtype, shift)
    (_, dyd), (_, dresd), (dxbuf, dx) = (_placed(dy, dtype, shift), _placed(dres, dtype, shift),
                                         _placed(zero, dtype, shift))
    g, b = torch.from_numpy(gamma).cuda(), torch.from_numpy(beta).cuda()
    v = None if valid is None else torch.from_numpy(valid).cuda()
    stats = torch.full((rows, 2), 7.0, device="cuda")
    dg, db = torch.full((width,), 7.0, device="cuda"), torch.full((width,), 7.0, device="cuda")
    need = L.lrm_layer_norm_workspace(ctx, rows, width)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    L.lrm_layer_norm(ctx, xd, _code(dtype), g, b, v, rows, width, EPS, y, stats)
    L.lrm_layer_norm_backward(ctx, xd, _code(dtype), dyd, g, stats, v, dresd if use_res else None, rows, width, dx, dg,
                              db, ws, need)
    torch.cuda.synchronize()
    assert _untouched(ybuf, shift, n) and _untouched(dxbuf, shift, n)

    xn, gn, bn = _np(torch.nan_to_num(x)), gamma.astype(np.float64), beta.astype(np.float64)
    y_ref, st_ref = O.layer_norm(xn, gn, bn, EPS, valid)
    keep = np.ones(rows, bool) if valid is None else valid != 0
    mean, rstd = st_ref[:, :1], st_ref[:, 1:]
    c = np.abs(xn - mean)
    t_mean = A * np.abs(xn).mean(1, keepdims=True) + U * np.abs(mean)
    # the centred values are off by the mean's error and a rounding; the mean's error enters the variance squared
    var = (c ** 2).mean(1, keepdims=True) + EPS
    t_rstd = (A + 4 * U + t_mean ** 2 / var + 2 * U) * np.abs(rstd)
    st = _np(stats)
    assert np.all(np.abs(st[:, :1] - mean) <= t_mean * keep[:, None])
    assert np.all(np.abs(st[:, 1:] - rstd) <= t_rstd * keep[:, None])
    t_xhat = (t_mean + 2 * U * c) * np.abs(rstd) + c * t_rstd + 2 * U * c * np.abs(rstd)
    ty = (np.abs(gn) * t_xhat + 2 * U * np.abs(y_ref)) * keep[:, None]
    assert np.all(np.abs(_np(y) - y_ref) <= ty + STORE[dtype] * (np.abs(y_ref) + ty))

    # the backward from the statistics that the forward left
    dyn, drn = _np(torch.nan_to_num(dy)), _np(torch.nan_to_num(dres))
    dx_ref, dg_ref, db_ref = O.layer_norm_backward(xn, dyn, gn, st, valid, drn if use_res else None)
    m, r = st[:, :1], st[:, 1:]
    xhat = (xn - m) * r
    t_xhat = 3 * U * np.abs(xhat)
    d = np.abs(dyn * gn)
    t0 = (A + 2 * U) * d.mean(1, keepdims=True)
    t1 = (A + 8 * U) * (d * np.abs(xhat)).mean(1, keepdims=True)
    size = d + np.abs((dyn * gn).mean(1, keepdims=True)) + np.abs(xhat) * (d * np.abs(xhat)).mean(1, keepdims=True)
    tx = r * (t0 + np.abs(xhat) * t1 + 8 * U * size) + (2 * U * np.abs(drn) if use_res else 0.0)
    tx = tx * keep[:, None]
    assert np.all(np.abs(_np(dx) - dx_ref) <= tx + STORE[dtype] * (np.abs(dx_ref) + tx))
    per = (rows / 128 + 64) * U
    kd = dyn * keep[:, None]
    assert np.all(np.abs(_np(dg) - dg_ref) <= per * np.abs(kd * xhat).sum(0) + (np.abs(kd) * t_xhat).sum(0) + 1e-300)
    assert np.all(np.abs(_np(db) - db_ref) <= per * np.abs(kd).sum(0) + 1e-300)


def test_many_rows_and_no_rows(ctx):
    from backward_token_expert_gb300 import lrm as L

    rows, width = 200000, 40
    x, dy, _, gamma, beta, _ = _inputs(rows, width, torch.bfloat16, 1, False)
    xd, dyd, g, b = x.cuda(), dy.cuda(), torch.from_numpy(gamma).cuda(), torch.from_numpy(beta).cuda()
    y, dx, stats = torch.empty_like(xd), torch.empty_like(xd), torch.empty(rows, 2, device="cuda")
    dg, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    need = L.lrm_layer_norm_workspace(ctx, rows, width)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    L.lrm_layer_norm(ctx, xd, L.DTYPE_BF16, g, b, None, rows, width, EPS, y, stats)
    L.lrm_layer_norm_backward(ctx, xd, L.DTYPE_BF16, dyd, g, stats, None, None, rows, width, dx, dg, db, ws, need)
    _, dg_ref, db_ref = O.layer_norm_backward(_np(xd), _np(dyd), _np(g), _np(stats))
    xhat = (_np(xd) - _np(stats)[:, :1]) * _np(stats)[:, 1:]
    per = (rows / 128 + 64 + 3) * U
    assert np.all(np.abs(_np(dg) - dg_ref) <= per * np.abs(_np(dyd) * xhat).sum(0))
    assert np.all(np.abs(_np(db) - db_ref) <= per * np.abs(_np(dyd)).sum(0))
    L.lrm_layer_norm(ctx, None, L.DTYPE_BF16, None, None, None, 0, width, EPS, None, None)
    L.lrm_layer_norm_backward(ctx, None, L.DTYPE_BF16, None, None, None, None, None, 0, width, None, dg, db, None, 0)
    assert (dg == 0).all() and (db == 0).all()
    valid = torch.zeros(rows, dtype=torch.uint8, device="cuda")  # nothing but padding
    dg.fill_(7.0)
    L.lrm_layer_norm_backward(ctx, xd, L.DTYPE_BF16, dyd, g, stats, valid, None, rows, width, dx, dg, db, ws, need)
    assert (dg == 0).all() and (db == 0).all() and (dx == 0).all()


def test_offsets_beyond_32_bits(ctx):
    from backward_token_expert_gb300 import lrm as L

    width = 16383
    rows = (1 << 31) // width + 5
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, width, device="cuda").to(torch.bfloat16)
    g, b = torch.ones(width, device="cuda"), torch.full((width,), 0.5, device="cuda")
    y, stats = torch.empty_like(x), torch.empty(rows, 2, device="cuda")
    L.lrm_layer_norm(ctx, x, L.DTYPE_BF16, g, b, None, rows, width, EPS, y, stats)
    ref, _ = O.layer_norm(_np(x[-3:]), np.ones(width), np.full(width, 0.5), EPS)
    assert np.all(np.abs(_np(y[-3:]) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4)
    assert (y[:-3] == 0.5).all()
    dg, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    need = L.lrm_layer_norm_workspace(ctx, rows, width)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x)
    L.lrm_layer_norm_backward(ctx, x, L.DTYPE_BF16, y, g, stats, None, None, rows, width, dx, dg, db, ws, need)
    dx_ref, _, _ = O.layer_norm_backward(_np(x[-3:]), _np(y[-3:]), np.ones(width), _np(stats[-3:]))
    assert np.all(np.abs(_np(dx[-3:]) - dx_ref) <= 2.0 ** -8 * np.abs(dx_ref) + 1e-4)


def test_constant_rows_and_non_finite_rows(ctx):
    """A row without spread gives beta (eps keeps rstd finite); NaN and infinities stay in their row."""
    from backward_token_expert_gb300 import lrm as L

    rows, width = 6, 96
    x = torch.randn(rows, width)
    x[0], x[1], x[2, 5], x[3, 7] = 3.25, 0.0, float("nan"), float("inf")
    g, b = torch.ones(width, device="cuda"), torch.arange(width, device="cuda").float()
    y, stats = torch.empty(rows, width, device="cuda"), torch.empty(rows, 2, device="cuda")
    L.lrm_layer_norm(ctx, x.cuda(), L.DTYPE_F32, g, b, None, rows, width, EPS, y, stats)
    assert torch.equal(y[0], b) and torch.equal(y[1], b)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all() and torch.isfinite(y[4:]).all()


def test_graph_and_stream_give_the_same_bits(ctx):
    from backward_token_expert_gb300 import lrm as L

    rows, width = 700, 1001
    x, dy, dres, gamma, beta, valid = _inputs(rows, width, torch.bfloat16, 4, True)
    xd, dyd, drd, v = x.cuda(), dy.cuda(), dres.cuda(), torch.from_numpy(valid).cuda()
    g, b = torch.from_numpy(gamma).cuda(), torch.from_numpy(beta).cuda()
    need = L.lrm_layer_norm_workspace(ctx, rows, width)

    def buffers():
        return [torch.zeros_like(xd), torch.zeros(rows, 2, device="cuda"), torch.zeros_like(xd),
                torch.zeros(width, device="cuda"), torch.zeros(width, device="cuda"),
                torch.zeros(need, dtype=torch.uint8, device="cuda")]

    def run(o, stream=None):
        L.lrm_layer_norm(ctx, xd, L.DTYPE_BF16, g, b, v, rows, width, EPS, o[0], o[1], stream)
        L.lrm_layer_norm_backward(ctx, xd, L.DTYPE_BF16, dyd, g, o[1], v, drd, rows, width, o[2], o[3], o[4], o[5],
                                  need, stream)

    one, two, three = buffers(), buffers(), buffers()
    run(one)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(two, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(three)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b2, c in list(zip(one, two, three))[:5]:
        assert torch.equal(a, b2) and torch.equal(a, c)


def test_refusals(ctx):
    from backward_token_expert_gb300 import lrm as L

    z = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    p = z.data_ptr()
    fwd = lambda **k: L.lrm_layer_norm(ctx, *[k.get(n, v) for n, v in  # noqa: E731
                                              dict(x=p, dt=0, g=p, b=p, valid=None, rows=4, width=16, eps=EPS, y=p,
                                                   stats=p).items()])
    bwd = lambda **k: L.lrm_layer_norm_backward(ctx, *[k.get(n, v) for n, v in  # noqa: E731
                                                       dict(x=p, dt=1, dy=p, g=p, stats=p, valid=None, dres=None,
                                                            rows=4, width=16, dx=p, dg=p, db=p, ws=p,
                                                            nb=1 << 20).items()])
    inv, al, shape, wsp = L.LRM_ERR_INVALID_ARG, L.LRM_ERR_ALIGN, L.LRM_ERR_SHAPE, L.LRM_ERR_WORKSPACE
    for call, kw, code in [
            (fwd, dict(x=None), inv), (fwd, dict(g=None), inv), (fwd, dict(b=None), inv), (fwd, dict(y=None), inv),
            (fwd, dict(stats=None), inv), (fwd, dict(dt=2), inv), (fwd, dict(rows=-1), inv), (fwd, dict(width=0), inv),
            (fwd, dict(eps=-1.0), inv), (fwd, dict(eps=float("nan")), inv), (fwd, dict(width=16385), shape),
            (fwd, dict(x=p + 2), al), (fwd, dict(y=p + 4), al), (fwd, dict(g=p + 2), al), (fwd, dict(stats=p + 4), al),
            (bwd, dict(dy=None), inv), (bwd, dict(dx=None), inv), (bwd, dict(dg=None), inv), (bwd, dict(db=None), inv),
            (bwd, dict(ws=None), wsp), (bwd, dict(nb=127), wsp), (bwd, dict(dy=p + 2), al), (bwd, dict(dres=p + 2), al),
            (bwd, dict(dx=p + 8), al), (bwd, dict(x=p + 1), al), (bwd, dict(width=16385), shape)]:
        with pytest.raises(L.LrmError) as ei:
            call(**kw)
        assert ei.value.code == code, kw
    with pytest.raises(L.LrmError):
        L.lrm_layer_norm_workspace(ctx, 4, 0)
