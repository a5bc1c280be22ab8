"""Layer norm's backward where mean times 1 / standard deviation passes fp32's range
but no value of a row does: rows that hold their mean alone.  Then xhat = 0 and
dx = rstd (d - mean(d)) + dres, dgamma = 0, dbeta = sum dy.

Tolerances as in the other tests of the norm, u = 2^-24: 90 u of the magnitudes for
a row's sum, 3 u for the product and the two differences, half a step of the stored
type; the sums of the six rows' dy 6 u of the magnitudes."""

import numpy as np
import pytest
import torch

from gpu_common import built_library, need_gpu
from test_gpu_layer_norm import A, STORE, U, _code, _np, _placed

pytestmark = pytest.mark.gpu

MEAN, RSTD = 2.0 ** 110, 2.0 ** 20


@pytest.fixture(scope="module")
def ctx():
    from backward_token_expert_gb300 import lrm as L

    need_gpu()
    built_library()
    c = L.lrm_create(0)
    yield c
    L.lrm_destroy(c)


# one lane a row up to many warps, whole vectors with lanes beyond the row, cut rows, weights in shared memory
@pytest.mark.parametrize("width,shift", [(1, 0), (4, 0), (5, 0), (8, 0), (8, 3), (24, 0), (33, 1), (136, 0), (250, 0),
                                         (1000, 0), (1497, 0), (2056, 1), (4100, 0), (4104, 0), (9001, 0), (12000, 0),
                                         (16377, 2), (16384, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_that_hold_their_mean_alone(ctx, width, shift, dtype, residual):
    from backward_token_expert_gb300 import lrm as L

    rows = 6
    g = torch.Generator().manual_seed(width)
    dy, dres = (torch.randn(rows, width, generator=g).to(dtype) for _ in range(2))
    gamma = 1 + 0.2 * torch.randn(width, generator=g)
    x = torch.full((rows, width), MEAN, dtype=dtype)
    xd, dyd, rd, dxd = (_placed(t, dtype, shift)[1] for t in (x, dy, dres, torch.zeros_like(x)))
    stats = torch.tensor([[MEAN, RSTD]] * rows, device="cuda")
    gd = gamma.cuda()
    dg, db = torch.full((width,), 7.0, device="cuda"), torch.full((width,), 7.0, device="cuda")
    need = L.lrm_layer_norm_workspace(ctx, rows, width)
    ws = torch.empty(max(need, 4), dtype=torch.uint8, device="cuda")
    L.lrm_layer_norm_backward(ctx, xd, _code(dtype), dyd, gd, stats, None, rd if residual else None, rows, width, dxd,
                              dg, db, ws, ws.numel())
    torch.cuda.synchronize()
    assert L.lrm_get_device_status(ctx) == 0
    d = _np(dy) * _np(gamma)
    mean, size = d.mean(1, keepdims=True), np.abs(d).mean(1, keepdims=True)
    r = _np(dres) if residual else np.zeros_like(d)
    want = RSTD * (d - mean) + r
    tol = RSTD * (A * size + 3 * U * (np.abs(d) + size)) + 3 * U * np.abs(r)
    assert np.all(np.abs(_np(dxd) - want) <= STORE[dtype] * (np.abs(want) + tol) + tol)
    assert np.all(_np(dg) == 0)
    sums = np.abs(_np(dy)).sum(0)
    assert np.all(np.abs(_np(db) - _np(dy).sum(0)) <= rows * U * sums)
