"""Dropout with a residual: the mask is the oracle's, element for element; the
kept values are one product with the fp32 scale 1 / (1 - p) (2^-24 off) and one
addition in one rounding: 2^-24 of the product, plus the stored type's half step."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import built_library, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STORE = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


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


def _check(out, x, res, kept, p, dtype):
    x, out = x.double().cpu().numpy(), out.double().cpu().numpy()
    res = np.zeros_like(x) if res is None else res.double().cpu().numpy()
    prod = np.where(kept, x / (1 - p) if p < 1 else 0.0, 0.0)
    ref = prod + res
    tol = 2 * U * np.abs(prod)
    assert np.all(np.abs(out - ref) <= tol + STORE[dtype] * (np.abs(ref) + tol))
    assert np.array_equal(out[~kept], res[~kept])


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 31, 255, 1024, 4099, 100003])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p,residual,shift", [(0.3, True, 0), (0.1, False, 0), (0.5, True, 1), (0.9, False, 3), (0.0, True, 0),
                                              (0.0, False, 1), (1.0, True, 0), (2.0 ** -33, False, 0)])
def test_values_and_mask(ctx, n, dtype, p, residual, shift):
    from backward_token_expert_gb300 import lrm as L

    rng = np.random.default_rng(n)
    seed, offset, step = int(rng.integers(1 << 63)) * 2 + 1, int(rng.integers(1 << 63)), int(rng.integers(1 << 40))
    mk = lambda: torch.from_numpy(rng.standard_normal(n + shift + 8).astype(np.float32)).to(dtype).cuda()  # noqa: E731
    xb, rb = mk(), mk()
    x, r = xb[shift:shift + n], rb[shift:shift + n] if residual else None
    ob = torch.full((n + shift + 8,), 7.0, dtype=dtype, device="cuda")
    counter = torch.tensor([step], dtype=torch.int64, device="cuda")
    L.lrm_dropout_add(ctx, x, r, _code(dtype), n, p, seed, offset, counter, ob[shift:])
    kept = O.dropout_kept(n, p, seed, offset + step)
    _check(ob[shift:shift + n], x, r, kept, p, dtype)
    assert (ob[:shift] == 7.0).all() and (ob[shift + n:] == 7.0).all()
    again = torch.empty(n, dtype=dtype, device="cuda")  # no step: the sum given directly
    L.lrm_dropout_add(ctx, x, r, _code(dtype), n, p, seed, offset + step, None, again)
    assert torch.equal(again, ob[shift:shift + n])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place_and_backward_share_the_mask(ctx, dtype):
    from backward_token_expert_gb300 import lrm as L

    n, p = 70001, 0.25
    x, r = torch.randn(n, device="cuda").to(dtype), torch.randn(n, device="cuda").to(dtype)
    out = torch.empty_like(x)
    L.lrm_dropout_add(ctx, x, r, _code(dtype), n, p, 5, 6, None, out)
    for target in (x.clone(), r.clone()):
        a, b = (target, r) if torch.equal(target, x) else (x, target)
        L.lrm_dropout_add(ctx, a, b, _code(dtype), n, p, 5, 6, None, target)
        assert torch.equal(target, out)
    # the gradient of <out, dy> by x: dy / (1 - p) where an element was kept
    dy, dx = torch.randn(n, device="cuda").to(dtype), torch.empty_like(x)
    L.lrm_dropout_add(ctx, dy, None, _code(dtype), n, p, 5, 6, None, dx)
    _check(dx, dy, None, O.dropout_kept(n, p, 5, 6), p, dtype)
    assert torch.equal(dx != 0, (out != r) & (dy != 0)) or dtype == torch.bfloat16


def test_dropped_elements_hide_nan_and_infinity(ctx):
    from backward_token_expert_gb300 import lrm as L

    n, p = 4096, 0.5
    kept = O.dropout_kept(n, p, 9, 0)
    x = torch.ones(n)
    x[torch.from_numpy(~kept)] = float("nan")
    out = torch.empty(n, device="cuda")
    L.lrm_dropout_add(ctx, x.cuda(), None, L.DTYPE_F32, n, p, 9, 0, None, out)
    assert np.array_equal(out.cpu().numpy(), np.where(kept, 2.0, 0.0).astype(np.float32))


def test_counters_beyond_32_bits(ctx):
    """Elements past 2^34 use the second counter word, addresses past 2^32 bytes 64-bit offsets."""
    from backward_token_expert_gb300 import lrm as L

    n = (1 << 34) + 4096
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    L.lrm_dropout_add(ctx, x, None, L.DTYPE_BF16, n, 0.5, 3, 1, None, x)
    for first in (0, (1 << 32) - 64, (1 << 34) - 64, n - 128):
        kept = O.dropout_kept(128, 0.5, 3, 1, first=first)
        assert np.array_equal(x[first:first + 128].float().cpu().numpy(), np.where(kept, 2.0, 0.0))


def test_a_replayed_graph_draws_a_new_mask(ctx):
    from backward_token_expert_gb300 import lrm as L

    n, p = 5000, 0.4
    x, out = torch.randn(n, device="cuda"), torch.empty(n, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    L.lrm_dropout_add(ctx, x, None, L.DTYPE_F32, n, p, 1, 2, step, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lrm_dropout_add(ctx, x, None, L.DTYPE_F32, n, p, 1, 2, step, out)
        step.add_(1)
    for i in range(3):
        graph.replay()
        _check(out, x, None, O.dropout_kept(n, p, 1, 2 + i), p, torch.float32)


def test_refusals(ctx):
    from backward_token_expert_gb300 import lrm as L

    z = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    q = z.data_ptr()
    call = lambda **k: L.lrm_dropout_add(ctx, *[k.get(n, v) for n, v in  # noqa: E731
                                                dict(x=q, r=None, dt=0, n=16, p=0.1, seed=1, off=1, step=None,
                                                     out=q + 1024).items()])
    inv, al = L.LRM_ERR_INVALID_ARG, L.LRM_ERR_ALIGN
    for kw, code in [(dict(x=None), inv), (dict(out=None), inv), (dict(n=-1), inv), (dict(p=-0.1), inv), (dict(p=1.01), inv),
                     (dict(p=float("nan")), inv), (dict(dt=3), inv), (dict(x=q + 2), al), (dict(out=q + 1), al),
                     (dict(r=q + 2), al), (dict(step=q + 4), al)]:
        with pytest.raises(L.LrmError) as ei:
            call(**kw)
        assert ei.value.code == code, kw
    call(n=0, x=None, out=None)
