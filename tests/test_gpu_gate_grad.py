"""Gate gradients of the retained pairs against the fp64 oracle.

A row's products of two bf16 values are exact in fp32; the sum of I of them in
at most I / 32 serial additions a lane and a tree over the warp is within
(I / 32 + 16) 2^-24 of the sum of the magnitudes."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import built_library, custom_inputs, need_gpu

pytestmark = pytest.mark.gpu


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


def _case(N, E, I, rows, spare, seed):
    rng = np.random.default_rng(seed)
    ids = rng.choice(N, rows, replace=False).astype(np.int32)
    of = np.sort(rng.integers(0, E, rows))
    off = np.searchsorted(of, np.arange(E + 1)).astype(np.int32)
    mk = lambda: torch.from_numpy(rng.standard_normal((rows + spare, I)).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    x, y = mk(), mk()
    x[rows:], y[rows:] = float("nan"), float("nan")  # beyond the total: never read into a result
    full = np.concatenate([ids, np.full(spare, 1 << 30, np.int32)])
    return x.cuda(), y.cuda(), torch.from_numpy(full).cuda(), torch.from_numpy(off).cuda(), ids


def _check(got, x, y, ids, N, I):
    rows = len(ids)
    a, b = x[:rows].double().cpu().numpy(), y[:rows].double().cpu().numpy()
    ref = O.gate_grad(a, b, ids, N)
    tol = O.gate_grad(np.abs(a), np.abs(b), ids, N) * (I / 32 + 16) * 2.0 ** -24
    got = got.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ref) <= tol)
    dropped = np.ones(N, bool)
    dropped[ids] = False
    assert np.all(got[dropped] == 0)


@pytest.mark.parametrize("N,E,I,rows,spare", [
    (1, 1, 8, 1, 0), (5, 2, 8, 0, 3), (512, 8, 32, 333, 9), (700, 4, 16, 700, 0), (901, 5, 136, 600, 1),
    (3000, 20, 248, 2999, 7), (2000, 16, 256, 1500, 0), (1000, 3, 264, 800, 0), (4001, 13, 768, 2500, 33),
    (333, 3, 1496, 200, 5), (300, 3, 1536, 211, 1), (100, 1, 65536, 40, 1), (20000, 128, 64, 15001, 100)])
def test_rows(ctx, N, E, I, rows, spare):
    from backward_token_expert_gb300 import lrm as L

    x, y, ids, off, host_ids = _case(N, E, I, rows, spare, N + I)
    out = torch.full((N,), 3.0, device="cuda")
    L.lrm_gate_grad(ctx, x, y, off, ids, L.dims_of(N, E, 1, 8, I), rows + spare, out)
    torch.cuda.synchronize()
    assert L.lrm_get_device_status(ctx) == 0
    _check(out, x, y, host_ids, N, I)


def test_offsets_beyond_32_bits(ctx):
    from backward_token_expert_gb300 import lrm as L

    I = 2048
    rows = (1 << 31) // I + 777
    x = torch.zeros(rows, I, dtype=torch.bfloat16, device="cuda")
    y = torch.ones(rows, I, dtype=torch.bfloat16, device="cuda")
    x[-3:, 5] = torch.tensor([1.0, 2.0, 3.0], dtype=torch.bfloat16, device="cuda")
    ids = torch.arange(rows, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out = torch.empty(rows, device="cuda")
    L.lrm_gate_grad(ctx, x, y, off, ids, L.dims_of(rows, 1, 1, 8, I), rows, out)
    torch.cuda.synchronize()
    assert out[-3:].tolist() == [1.0, 2.0, 3.0] and not out[:-3].any()


def test_total_beyond_max_rows_and_bad_ids(ctx):
    from backward_token_expert_gb300 import lrm as L

    N, I = 200, 64
    x, y, ids, off, host_ids = _case(N, 4, I, 100, 0, 3)
    off[-1] = 500  # clamped to max_rows
    ids[7] = -1
    ids[50] = N
    out = torch.full((N,), 3.0, device="cuda")
    L.lrm_gate_grad(ctx, x, y, off, ids, L.dims_of(N, 4, 1, 8, I), 100, out)
    assert L.lrm_get_device_status(ctx) == 1 << L.LRM_ERR_INDEX
    keep = np.array([i for i in range(100) if i not in (7, 50)])
    _check(out, x[keep], y[keep], host_ids[keep], N, I)
    off[-1] = -3
    L.lrm_gate_grad(ctx, x, y, off, ids, L.dims_of(N, 4, 1, 8, I), 100, out)
    assert L.lrm_get_device_status(ctx) == 0 and float(out.abs().sum()) == 0
    L.lrm_gate_grad(ctx, None, None, off, None, L.dims_of(N, 4, 1, 8, I), 0, out)
    assert float(out.abs().sum()) == 0


def test_refusals(ctx):
    from backward_token_expert_gb300 import lrm as L

    x, y, ids, off, _ = _case(50, 4, 32, 20, 0, 4)
    out = torch.empty(50, device="cuda")
    good = dict(x=x, y=y, off=off, ids=ids, d=L.dims_of(50, 4, 1, 8, 32), n=20, out=out)
    inv, al = L.LRM_ERR_INVALID_ARG, L.LRM_ERR_ALIGN
    for kw, code in [(dict(x=None), inv), (dict(y=None), inv), (dict(off=None), inv), (dict(ids=None), inv),
                     (dict(out=None), inv), (dict(n=-1), inv), (dict(d=L.dims_of(50, 4, 1, 8, 30)), al),
                     (dict(x=x.data_ptr() + 8), al), (dict(y=y.data_ptr() + 2), al), (dict(out=out.data_ptr() + 2), al),
                     (dict(ids=ids.data_ptr() + 1), al)]:
        a = dict(good, **kw)
        with pytest.raises(L.LrmError) as ei:
            L.lrm_gate_grad(ctx, a["x"], a["y"], a["off"], a["ids"], a["d"], a["n"], a["out"])
        assert ei.value.code == code, kw


def test_same_bits_on_another_stream(ctx):
    from backward_token_expert_gb300 import lrm as L

    x, y, ids, off, _ = _case(5000, 8, 200, 4000, 0, 5)
    d = L.dims_of(5000, 8, 1, 8, 200)
    a, b = torch.empty(5000, device="cuda"), torch.empty(5000, device="cuda")
    L.lrm_gate_grad(ctx, x, y, off, ids, d, 4000, a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    L.lrm_gate_grad(ctx, x, y, off, ids, d, 4000, b, s)
    s.synchronize()
    assert torch.equal(a, b)


def test_after_the_recalibration_step():
    # <dphi_c, phi_c> equals alpha_u g_t . (W_e phi_u) of the original inputs, to the rounding of
    # delta and dphi to bf16 (2^-9 each, in the worst direction of every product)
    from backward_token_expert_gb300.pipeline import Recalibration, to_device_inputs

    inp = custom_inputs(T=600, E=6, k=2, h=64, I=48, s=1.0, rho=Fraction(1, 2), seed=31)
    w = inp.workload
    rec = Recalibration(w.T, w.E, w.k, w.h, w.I, w.cf, w.rho)
    try:
        d = to_device_inputs(inp)
        rec.run(d["logits"], d["expert_idx"], d["g"], d["phi"], d["alpha"], d["W"])
        got = rec.gate_grad().cpu().numpy()
        assert rec.device_status() == 0
        ids = rec.buf.sel_ids[: int(rec.buf.sel_offsets[-1])].cpu().numpy()
    finally:
        rec.close()
    g, phi, W = (O.bf16_to_f64(a) for a in (inp.g, inp.phi, inp.W))
    ref, mag = np.zeros(w.N), np.zeros(w.N)
    for u in ids:
        e, t = inp.expert_idx[u // w.k, u % w.k], u // w.k
        ref[u] = inp.alpha[u] * (g[t] @ W[e] @ phi[u])
        mag[u] = inp.alpha[u] * (np.abs(g[t]) @ np.abs(W[e]) @ np.abs(phi[u]))
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * 1.1 * mag)
    assert np.all(got[np.setdiff1d(np.arange(w.N), ids)] == 0)
