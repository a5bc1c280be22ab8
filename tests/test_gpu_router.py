"""Router forward and backward against the fp64 oracle.

Tolerances, from fp32 arithmetic (unit roundoff u = 2^-24):
* l - m is rounded once: for |l - m| <= 88 (below that exp underflows) its
  error is at most 88 u, which is a relative error of exp; with expf's 2 ulp,
  the sum over E terms, and the division, a probability is within 1e-5 of its
  value, or 1e-37 where it is subnormal;
* P and the balance loss are sums of positive such terms: 1e-5 relative, with
  the rounding of at most T / 8 serial additions;
* lse is off by 1e-5 (the relative error of s) and by its own rounding;
* dlogits: 2e-5 of the sum of the magnitudes of its terms; stored as bf16,
  2^-8 of the value more.
Ids and counts are exact.
"""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import built_library, need_gpu

pytestmark = pytest.mark.gpu

REL = 1e-5
TINY = 1e-37
AUX, Z = 0.3, 0.2
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    built_library()


def _logits(T, E, dtype, seed, scale=1.5):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, E)) * scale - 0.8 * np.log(rng.permutation(E) + 1.0)
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


def _close(got, ref, tol):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bad = ~(np.abs(got - ref) <= tol + TINY)
    assert not bad.any(), (int(bad.sum()), np.abs(got - ref).max())


def check_forward(r, ref, z_scale):
    T = r.T
    assert np.array_equal(r.expert_idx.cpu().numpy(), ref["expert_idx"])
    assert np.array_equal(r.counts.cpu().numpy(), ref["counts"])
    assert int(r.tokens.item()) == ref["tokens"]
    _close(r.alpha.cpu().numpy().reshape(T, r.k), ref["alpha"], REL * np.abs(ref["alpha"]))
    stats = r.row_stats.cpu().numpy()
    assert np.array_equal(stats[:, 0], ref["row_stats"][:, 0].astype(np.float32))
    _close(stats[:, 1], ref["row_stats"][:, 1], REL * ref["row_stats"][:, 1])
    _close(r.f.cpu().numpy(), ref["f"], 2.0 ** -24 * ref["f"])
    _close(r.P.cpu().numpy(), ref["P"], REL * ref["P"])
    loss, aux, z = r.losses.cpu().numpy().astype(np.float64)
    assert abs(aux - ref["aux"]) <= REL * ref["aux"] + TINY
    z_tol = 2 * REL * (1.0 + z_scale) * (z_scale + REL)
    with np.errstate(over="ignore"):  # the oracle's values in the type they are reported in
        z_ref, loss_ref = float(np.float32(ref["z"])), float(np.float32(ref["loss"]))
    assert z == z_ref or abs(z - z_ref) <= z_tol
    assert loss == loss_ref or abs(loss - ref["loss"]) <= AUX * REL * ref["aux"] + Z * z_tol + 2.0 ** -23 * abs(ref["loss"])


def backward_tol(l, ref, f, dgate, renorm, bf16_out, want):
    E, Tc = l.shape[1], max(1, ref["tokens"])
    p = ref["p"]
    fp = (p * f).sum(1, keepdims=True)
    m, s = ref["row_stats"].T
    lse = np.abs(m + np.log(np.where(s > 0, s, 1.0)))[:, None]
    mag = p * (AUX * E / Tc * (f + fp) + 2 * Z / Tc * (lse + 1.0))
    if dgate is not None:
        S = np.abs(dgate).sum(1, keepdims=True)
        at = np.abs(dgate) + (ref["alpha"] * S if renorm else 0.0)
        for t in range(l.shape[0]):
            mag[t, ref["expert_idx"][t]] += at[t]
        if not renorm:
            mag = mag + p * S
    tol = 2e-5 * mag
    return tol + (2.0 ** -8 * np.abs(want) if bf16_out else 0.0)


def run(T, E, k, dtype="f32", renorm=True, valid=None, logits=None, out=None, with_gates=True, seed=0):
    from backward_token_expert_gb300.pipeline import Router

    r = Router(T, E, k, renorm, AUX, Z, dtype=DT[dtype], dlogits_dtype=DT[out or dtype])
    x = _logits(T, E, dtype, seed) if logits is None else logits
    d = x.cuda()
    v = None if valid is None else torch.from_numpy(valid.astype(np.uint8)).cuda()
    r.forward(d, v)
    l = x.double().numpy()
    ref = O.router_forward(l, k, renorm, AUX, Z, valid)
    m, s = ref["row_stats"][ref["counted"]].T
    z_scale = float(np.sqrt(((m + np.log(s)) ** 2).mean())) if ref["tokens"] else 0.0
    check_forward(r, ref, z_scale)
    rng = np.random.default_rng(seed + 99)
    dgate = None
    if with_gates:
        dgate = (rng.standard_normal((T, k)) * ref["alpha"]).astype(np.float32)
    r.backward(d, None if dgate is None else torch.from_numpy(dgate).cuda())
    f = r.f.cpu().numpy().astype(np.float64)
    want = O.router_backward(l, ref["expert_idx"], ref["alpha"], f, max(1, ref["tokens"]), dgate, renorm, AUX, Z,
                             ref["counted"])
    got = r.dlogits.double().cpu().numpy()
    _close(got, want, backward_tol(l, ref, f, dgate, renorm, (out or dtype) == "bf16", want))
    assert np.all(got[~ref["counted"]] == 0)
    from backward_token_expert_gb300 import lrm as L

    assert L.lrm_get_device_status(r.ctx) == 0
    return r, d, v


# every number of logits a lane can hold, odd sizes on both sides of it, k up to E and to 32
SHAPES = [(1, 1, 1), (1, 2, 2), (3, 5, 5), (256, 8, 2), (33, 16, 4), (31, 31, 7), (65, 32, 32), (70, 33, 32),
          (129, 63, 6), (500, 64, 8), (77, 96, 1), (1000, 128, 8), (64, 129, 9), (333, 160, 6), (50, 255, 32),
          (90, 256, 8), (41, 257, 10), (60, 511, 3), (40, 512, 32), (35, 1000, 12), (20, 1024, 32), (5000, 24, 3)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shapes(T, E, k, dtype):
    run(T, E, k, dtype, renorm=bool((T + E) % 2), seed=T + E)


@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("renorm", [True, False])
def test_mixed_types(dtype, out, renorm):
    run(200, 48, 4, dtype, renorm, out=out, seed=3)


@pytest.mark.parametrize("renorm", [True, False])
def test_masked_tokens(renorm):
    rng = np.random.default_rng(1)
    run(700, 40, 4, "bf16", renorm, valid=rng.random(700) < 0.6, seed=4)
    run(300, 128, 8, "f32", renorm, valid=rng.random(300) < 0.1, seed=5)


def test_no_token_counts():
    r, _, _ = run(50, 12, 3, valid=np.zeros(50), seed=6)
    assert float(r.losses.abs().sum()) == 0 and float(r.P.abs().sum()) == 0 and float(r.f.abs().sum()) == 0


def test_large_batch_uses_every_block():
    run(40000, 16, 2, seed=7)


# batches above the size from which a token is a lane's work; E off every grid of 4, 8 and 32
@pytest.mark.parametrize("T,E,k,dtype,masked", [
    (16384, 8, 2, "f32", False), (16385, 5, 5, "f32", True), (16400, 20, 8, "bf16", False), (16999, 33, 3, "f32", False),
    (20011, 160, 6, "bf16", True), (16384, 64, 8, "f32", True), (17000, 128, 8, "f32", False),
    (16390, 255, 7, "f32", False), (16384, 256, 8, "bf16", False), (16384, 256, 1, "f32", False), (16500, 1, 1, "f32", False)])
def test_large_batches(T, E, k, dtype, masked):
    valid = np.random.default_rng(T).random(T) < 0.7 if masked else None
    run(T, E, k, dtype, renorm=bool(E % 2), valid=valid, seed=T)


@pytest.mark.parametrize("E,k", [(16, 3), (100, 8), (128, 8)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_batches_with_ties_and_dead_rows(E, k, dtype):
    rng = np.random.default_rng(E)
    x = np.round(rng.standard_normal((16500, E)) * 4) / 4
    x[rng.random(x.shape) < 0.1] = -np.inf
    x[rng.random(x.shape) < 0.1] = -0.0
    x[::50] = -np.inf
    x[7::90, 1:] = float(np.finfo(np.float32).min)
    run(16500, E, k, dtype, logits=torch.from_numpy(x.astype(np.float32)).to(DT[dtype]), seed=E)


def test_logits_that_differ_below_the_keys_resolution():
    # neighbours in fp32: the last bits decide the order
    rng = np.random.default_rng(30)
    for T, E, k in [(700, 128, 8), (16400, 128, 8), (16400, 40, 5), (200, 512, 20)]:
        base = np.float32(1.5) * np.ones((T, E), np.float32)
        x = np.nextafter(base, np.float32(2), dtype=np.float32)
        step = rng.integers(0, 40, (T, E)).astype(np.int32)
        x = (base.view(np.int32) + step).view(np.float32)
        run(T, E, k, logits=torch.from_numpy(x), with_gates=False, seed=T)


@pytest.mark.parametrize("E", [20, 64, 128, 160, 256, 512, 1000])
@pytest.mark.parametrize("stride", [4, 8, 16, 32])
def test_close_logits_side_by_side(E, stride):
    # more logits than slots within a few units in the last place, in experts that lie `stride` groups of four apart
    rng = np.random.default_rng(E + stride)
    T, k = 64, 8
    near = np.flatnonzero((np.arange(E) // 4) % stride == 0)
    x = (rng.standard_normal((T, E)) - 6.0).astype(np.float32)
    close = (np.float32(1.5).view(np.int32) + rng.integers(0, 30, (T, near.size))).astype(np.int32).view(np.float32)
    x[:, near] = close
    run(T, E, k, logits=torch.from_numpy(x), seed=E)
    # a far larger logit beside them: their differences to it round together
    y = x.copy()
    y[:, near[-1]] = 40.0
    run(T, E, k, logits=torch.from_numpy(y), seed=E)
    z = x.copy()
    z[:, int(np.setdiff1d(np.arange(E), near)[0]) if near.size < E else 0] = 40.0
    run(T, E, k, logits=torch.from_numpy(z), seed=E)
    run(T, E, k + 1 if E < 300 else 9, logits=torch.from_numpy(z), seed=E)


@pytest.mark.parametrize("E,stride,k", [(160, 16, 9), (256, 16, 9), (256, 16, 12), (256, 16, 16), (128, 8, 12), (512, 32, 12),
                                        (1000, 32, 16), (1024, 32, 32)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_slots_than_a_list_from_one_lane(E, stride, k, dtype):
    # the largest logits all in experts `stride` groups of four apart
    near = np.flatnonzero((np.arange(E) // 4) % stride == 0)
    rng = np.random.default_rng(E + k)
    x = np.full((50, E), -30.0, np.float32)
    for t in range(50):
        x[t, near] = rng.permutation(near.size) * 0.25 + 1.0
    x[25:, near[: near.size // 2]] -= 40.0
    run(50, E, k, dtype, logits=torch.from_numpy(x).to(DT[dtype]), seed=k)


# rows that start on two elements' bytes, or on one's
@pytest.mark.parametrize("T,E,k", [(300, 34, 3), (301, 66, 9), (97, 210, 12), (64, 258, 8), (50, 514, 20), (111, 35, 10), (90, 213, 16)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_row_starts(T, E, k, dtype):
    run(T, E, k, dtype, renorm=bool(T % 2), out="f32" if T % 3 else "bf16", seed=T)


@pytest.mark.parametrize("E,stride", [(128, 8), (256, 16), (512, 32), (1000, 32)])
@pytest.mark.parametrize("k", [2, 4, 5, 8])
def test_last_slot_against_its_neighbour(E, stride, k):
    # k + 1 candidates `stride` groups of four apart; the largest that stays out of k and the last that
    # comes in differ by one unit in the last place, the larger one in the higher expert
    near = np.flatnonzero((np.arange(E) // 4) % stride == 0)
    assert near.size >= k + 1
    x = np.full((40, E), -90.0, np.float32)
    x[:, near[:k - 1]] = 40.0 - np.arange(k - 1, dtype=np.float32)
    x[:, near[k - 1]] = 1.5
    x[:, near[k]] = np.nextafter(np.float32(1.5), np.float32(2))
    r, _, _ = run(40, E, k, logits=torch.from_numpy(x), seed=k)
    assert int(r.expert_idx[0, -1]) == near[k]


@pytest.mark.parametrize("E,k", [(3, 2), (16, 4), (64, 8), (128, 3), (128, 8), (300, 8), (512, 20)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_both_zeros_as_the_largest_logits(E, k, dtype):
    rng = np.random.default_rng(E)
    x = rng.choice([0.0, -0.0, -1.0, -1e-30, -np.inf], size=(200, E))
    x[:, rng.integers(0, E)] = -0.0
    x[::3][x[::3] == 0] = -0.0
    run(200, E, k, dtype, logits=torch.from_numpy(x.astype(np.float32)).to(DT[dtype]), seed=E)


def test_garbage_and_nan_in_large_batches():
    from backward_token_expert_gb300.pipeline import Router

    T, E, k = 16400, 36, 4
    x = _logits(T, E, "f32", 31)
    valid = torch.ones(T, dtype=torch.uint8)
    valid[::9] = 0
    outs = []
    for fill in (0.0, float("nan"), -float("nan"), float("inf")):
        y = x.clone()
        y[valid == 0] = fill
        r = Router(T, E, k, False, AUX, Z)
        r.forward(y.cuda(), valid.cuda())
        ids = r.expert_idx.cpu()
        assert torch.all(ids.sort(1).values.diff(dim=1) > 0) and int(ids.min()) >= 0 and int(ids.max()) < E
        outs.append([t.clone() for t in (r.alpha, r.row_stats, r.counts, r.f, r.P, r._losses.view(torch.int32))])
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], o))
    y = x.clone()
    y[100, 3], y[16399, 35], y[16398] = float("nan"), float("inf"), -float("nan")
    r = Router(T, E, k, True, AUX, Z)
    r.forward(y.cuda())
    ids, alpha = r.expert_idx.cpu(), r.alpha.view(T, k).cpu()
    assert 3 not in ids[100].tolist() and ids[16399, 0] == 35 and ids[16398].tolist() == [0, 1, 2, 3]
    assert torch.isnan(r.losses[0]) and torch.isnan(alpha[16399]).any()
    good = [t for t in range(T) if t not in (100, 16398, 16399)]
    assert torch.isfinite(alpha[good]).all()


@pytest.mark.parametrize("E,k", [(8, 4), (100, 10), (128, 8)])
def test_ties_zeros_and_lowest_values(E, k):
    # few distinct values, both zeros, the type's lowest value, -inf in most places
    rng = np.random.default_rng(8)
    x = rng.choice([0.0, -0.0, 1.0, 2.0, float(np.finfo(np.float32).min), -np.inf], size=(300, E))
    x[:, 0] = 0.5  # every row counts
    run(300, E, k, logits=torch.from_numpy(x.astype(np.float32)), seed=9)


def test_rows_of_minus_infinity_are_not_counted():
    x = _logits(64, 20, "f32", 10)
    x[5] = -float("inf")
    x[63] = -float("inf")
    x[9, 1:] = -float("inf")  # one expert left
    r, _, _ = run(64, 20, 4, logits=x, seed=11)
    assert int(r.tokens.item()) == 62
    assert r.expert_idx[5].tolist() == [0, 1, 2, 3]


def test_all_rows_of_minus_infinity():
    run(10, 6, 2, logits=torch.full((10, 6), -float("inf")))


def test_wide_range_of_logits():
    x = _logits(100, 64, "f32", 12, scale=30.0)
    run(100, 64, 6, logits=x, seed=13)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_garbage_of_masked_tokens_reaches_nothing(dtype):
    from backward_token_expert_gb300.pipeline import Router

    T, E, k = 90, 32, 4
    x = _logits(T, E, dtype, 14)
    valid = torch.ones(T, dtype=torch.uint8)
    valid[::7] = 0
    outs = []
    for fill in (0.0, float("nan"), float("inf")):
        r = Router(T, E, k, True, AUX, Z, dtype=DT[dtype])
        y = x.clone()
        y[valid == 0] = fill
        r.forward(y.cuda(), valid.cuda())
        r.backward(y.cuda(), torch.full((T * k,), 0.5, device="cuda"))
        ids = r.expert_idx.cpu()
        assert torch.all(ids.sort(1).values.diff(dim=1) > 0) and int(ids.min()) >= 0 and int(ids.max()) < E
        outs.append([t.clone() for t in (r.alpha, r.row_stats, r.counts, r.f, r.P, r._losses.view(torch.int32),
                                         r.dlogits)])
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


def test_nan_and_infinity_of_counted_tokens():
    from backward_token_expert_gb300.pipeline import Router

    x = _logits(40, 10, "f32", 15)
    x[3, 4] = float("nan")
    x[8, 2] = float("inf")
    x[9] = float("nan")
    r = Router(40, 10, 3, True, AUX, Z)
    r.forward(x.cuda())
    r.backward(x.cuda())
    ids = r.expert_idx.cpu()
    assert 4 not in ids[3].tolist() and ids[8, 0] == 2 and ids[9].tolist() == [0, 1, 2]
    alpha = r.alpha.view(40, 3).cpu()
    bad = [3, 8, 9]
    assert torch.isnan(r.dlogits.cpu()[bad]).any(1).all()
    assert torch.isnan(alpha[8]).any()
    assert torch.isnan(r.losses[0]) and torch.isnan(r.P).any()
    good = [t for t in range(40) if t not in bad]
    assert torch.isfinite(alpha[good]).all()
    assert torch.equal(ids[good], torch.from_numpy(O.router_forward(x[good].double().numpy(), 3, True)["expert_idx"]).int())


def test_gradient_without_gates_and_with_own_load():
    run(120, 24, 3, with_gates=False, seed=16)
    from backward_token_expert_gb300.pipeline import Router

    r = Router(120, 24, 3, True, AUX, 0.0)
    x = _logits(120, 24, "f32", 17)
    r.forward(x.cuda())
    f = torch.rand(24, generator=torch.Generator().manual_seed(1))
    r.backward(x.cuda(), f=f.cuda())
    ref = O.router_forward(x.double().numpy(), 3, True)
    f64 = f.double().numpy()
    want = O.router_backward(x.double().numpy(), ref["expert_idx"], ref["alpha"], f64, 120, None, True, AUX, 0.0,
                             ref["counted"])
    fp = (ref["p"] * f64).sum(1, keepdims=True)
    _close(r.dlogits.cpu().numpy(), want, 2e-5 * AUX * 24 / 120 * ref["p"] * (f64 + fp))


def test_gradient_against_differences_of_the_library_losses():
    from backward_token_expert_gb300.pipeline import Router

    T, E, k = 6, 5, 2
    x = _logits(T, E, "f32", 18).cuda()
    r = Router(T, E, k, True, 0.0, 1.0)
    r.forward(x)
    g = r.backward(x).clone().cpu().numpy()
    h = 2.0 ** -6
    probe = Router(T, E, k, True, 0.0, 1.0)
    for t, e in [(0, 0), (2, 3), (5, 4)]:
        v = []
        for sign in (1.0, -1.0):
            y = x.clone()
            y[t, e] += sign * h
            probe.forward(y)
            v.append(float(probe.losses[2].item()))
        # truncation ~ h^2/6 times a third derivative of lse^2 (below 20), over T tokens; the
        # rounding of two losses of about 10 over 2h
        assert abs((v[0] - v[1]) / (2 * h) - g[t, e]) <= 20 * h * h / 6 + 4 * 2.0 ** -24 * 10 / (2 * h)


def test_same_bits_and_other_streams():
    from backward_token_expert_gb300.pipeline import Router

    T, E, k = 3000, 100, 5
    x = _logits(T, E, "f32", 19).cuda()
    dg = torch.randn(T * k, device="cuda")
    got = []
    for side in (False, True, False):
        r = Router(T, E, k, True, AUX, Z)
        torch.cuda.synchronize()
        if side:
            s = torch.cuda.Stream()
            r.forward(x, stream=s)
            r.backward(x, dg, stream=s)
            s.synchronize()
        else:
            r.forward(x)
            r.backward(x, dg)
        torch.cuda.synchronize()
        got.append([t.clone() for t in (r.expert_idx, r.alpha, r.row_stats, r.counts, r.f, r.P, r._losses, r.dlogits)])
    for o in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], o))


def test_stale_workspace_and_outputs_do_not_matter():
    from backward_token_expert_gb300.pipeline import Router

    x = _logits(900, 48, "f32", 20).cuda()
    r = Router(900, 48, 4, True, AUX, Z)
    r.forward(x)
    want = [t.clone() for t in (r.expert_idx, r.alpha, r.P, r.counts, r._losses)]
    r.ws.fill_(0xFF)
    for t in (r.expert_idx, r.alpha, r.P, r.counts, r._losses):
        t.fill_(-1)
    r.forward(x)
    assert all(torch.equal(a, b) for a, b in zip(want, (r.expert_idx, r.alpha, r.P, r.counts, r._losses)))


def test_unaligned_fp32_logits():
    # a 4-byte aligned base, and outputs at 4 bytes: contiguous tensors that start inside a buffer
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import Router

    T, E, k = 77, 64, 6
    x = _logits(T, E, "f32", 21).cuda()
    r, q = Router(T, E, k, True, AUX, Z), Router(T, E, k, True, AUX, Z)
    r.forward(x)
    dg = torch.randn(T * k, device="cuda")
    r.backward(x, dg)
    y = torch.empty(T * E + 1, device="cuda")[1:].view(T, E)
    y.copy_(x)
    out = torch.empty(T * E + 3, device="cuda")[3:].view(T, E)
    alpha = torch.empty(T * k + 1, device="cuda")[1:]
    idx = torch.empty(T * k + 1, dtype=torch.int32, device="cuda")[1:]
    L.lrm_router_forward(q.ctx, y, 0, None, q.dims, True, AUX, Z, idx, alpha, q.row_stats, q.counts, q.f, q.P,
                         q._losses, q.ws, q.ws.numel())
    L.lrm_router_backward(q.ctx, y, 0, idx, alpha, q.row_stats, dg, q.f, q._losses, q.dims, True, AUX, Z, out, 0)
    assert torch.equal(alpha, r.alpha) and torch.equal(idx, r.expert_idx.view(-1)) and torch.equal(q.P, r.P)
    assert torch.equal(out, r.dlogits)


def test_bad_ids_are_flagged_and_skipped():
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import Router

    T, E, k = 20, 8, 3
    x = _logits(T, E, "f32", 22).cuda()
    r = Router(T, E, k, False, 0.0, 0.0)
    r.forward(x)
    dg = torch.ones(T * k, device="cuda")
    r.backward(x, dg)
    want = r.dlogits.clone()
    r.expert_idx[4, 1] = 8
    r.expert_idx[7, 0] = -5
    r.expert_idx[11, 2] = r.expert_idx[11, 0]
    r.backward(x, dg)
    assert L.lrm_get_device_status(r.ctx) == 1 << L.LRM_ERR_INDEX
    same = [t for t in range(T) if t not in (4, 7, 11)]
    assert torch.equal(r.dlogits[same], want[same])
    # a skipped slot gives no gradient: the rest of the row is that of two slots, whose sum is 0 over the row
    assert torch.allclose(r.dlogits[[4, 7, 11]].sum(1), torch.zeros(3, device="cuda"), atol=1e-5)


def test_refusals():
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import Router

    T, E, k = 16, 8, 2
    r = Router(T, E, k, True, AUX, Z)
    x = torch.zeros(T, E, device="cuda")
    good = dict(logits=x, dt=0, valid=None, dims=r.dims, renorm=1, idx=r.expert_idx, alpha=r.alpha, rs=r.row_stats,
                counts=r.counts, f=r.f, P=r.P, losses=r._losses, ws=r.ws, n=r.ws.numel())

    def fwd(**kw):
        a = dict(good, **kw)
        L.lrm_router_forward(r.ctx, a["logits"], a["dt"], a["valid"], a["dims"], a["renorm"], AUX, Z, a["idx"],
                             a["alpha"], a["rs"], a["counts"], a["f"], a["P"], a["losses"], a["ws"], a["n"])

    def bwd(**kw):
        a = dict(good, out=r.dlogits, odt=0, dg=None, **kw) if "out" not in kw and "odt" not in kw and "dg" not in kw \
            else dict(dict(good, out=r.dlogits, odt=0, dg=None), **kw)
        L.lrm_router_backward(r.ctx, a["logits"], a["dt"], a["idx"], a["alpha"], a["rs"], a["dg"], a["f"],
                              a["losses"], a["dims"], a["renorm"], AUX, Z, a["out"], a["odt"])

    fwd()
    bwd()
    inv, al, shape, ws = L.LRM_ERR_INVALID_ARG, L.LRM_ERR_ALIGN, L.LRM_ERR_SHAPE, L.LRM_ERR_WORKSPACE
    big = L.dims_of(T, 1025, k, 8, 8)
    cases = [(fwd, dict(logits=None), inv), (fwd, dict(dt=2), inv), (fwd, dict(renorm=2), inv),
             (fwd, dict(idx=None), inv), (fwd, dict(losses=None), inv), (fwd, dict(counts=None), inv),
             (fwd, dict(dims=big), shape), (fwd, dict(dims=L.dims_of(T, E, E + 1, 8, 8)), shape),
             (fwd, dict(n=8), ws), (fwd, dict(ws=None), ws), (fwd, dict(logits=x.data_ptr() + 2), al),
             (fwd, dict(rs=r.row_stats.data_ptr() + 4), al), (fwd, dict(ws=r.ws.data_ptr() + 8), al),
             (fwd, dict(dt=1, logits=x.data_ptr() + 2), al),
             (bwd, dict(logits=None), inv), (bwd, dict(out=None), inv), (bwd, dict(odt=-1), inv),
             (bwd, dict(losses=None), inv), (bwd, dict(f=None), inv), (bwd, dict(renorm=-1), inv),
             (bwd, dict(dims=big), shape), (bwd, dict(out=r.dlogits.data_ptr() + 2), al),
             (bwd, dict(dg=r.alpha.data_ptr() + 1), al), (bwd, dict(odt=1, out=r.dlogits.data_ptr() + 8), al)]
    for fn, kw, code in cases:
        with pytest.raises(L.LrmError) as ei:
            fn(**kw)
        assert ei.value.code == code, (fn.__name__, kw)
    for bad in (x.double(), x[:, :4], x.t().contiguous().t(), x.cpu()):
        with pytest.raises(ValueError):
            r.forward(bad)
        with pytest.raises(ValueError):
            r.backward(bad)
    with pytest.raises(ValueError):
        r.forward(x, torch.ones(T, device="cuda"))
    with pytest.raises(ValueError):
        r.backward(x, torch.ones(T * k + 1, device="cuda"))
    with pytest.raises(ValueError):
        r.backward(x, f=torch.ones(E + 1, device="cuda"))
    with pytest.raises(ValueError):
        Router(4, 4, 2, dtype=torch.float16)


def test_offsets_beyond_32_bits():
    # 2^31 + logits: the last tokens equal those of a batch that holds nothing else
    from backward_token_expert_gb300.pipeline import Router

    E, k = 256, 4
    T = (1 << 31) // E + 20003
    x = torch.randint(0, 1 << 16, (1 << 20,), dtype=torch.int32, device="cuda").to(torch.float32).sub_(32768.0)
    x = (x / 8192.0).to(torch.bfloat16)
    big = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    big.view(-1)[: T * E // x.numel() * x.numel()].view(-1, x.numel()).copy_(x)
    big.view(-1)[T * E // x.numel() * x.numel():].copy_(x[: T * E % x.numel()])
    n = 5000
    tail = torch.randn(n, E, device="cuda").to(torch.bfloat16)
    big[-n:] = tail
    r, s = Router(T, E, k, True, 0.0, 0.0, dtype=torch.bfloat16), Router(n, E, k, True, 0.0, 0.0, dtype=torch.bfloat16)
    r.forward(big)
    s.forward(tail)
    dg = torch.zeros(T * k, device="cuda")
    dg[-n * k:] = torch.randn(n * k, device="cuda")
    r.backward(big, dg)
    s.backward(tail, dg[-n * k:].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(r.expert_idx[-n:], s.expert_idx) and torch.equal(r.alpha[-n * k:], s.alpha)
    assert torch.equal(r.row_stats[-n:], s.row_stats) and torch.equal(r.dlogits[-n:], s.dlogits)
    assert int(r.counts.sum()) == T * k and int(r.tokens) == T
    assert not r.dlogits[: T - n].any()


def test_no_tokens():
    from backward_token_expert_gb300.pipeline import Router

    r = Router(0, 8, 2, True, AUX, Z)
    r.counts.fill_(7)
    x = torch.empty(0, 8, device="cuda")
    r.forward(x)
    r.backward(x)
    assert int(r.counts.sum()) == 0 and int(r.tokens.item()) == 0 and float(r.losses.abs().sum()) == 0


def test_captured_in_a_graph():
    from backward_token_expert_gb300.pipeline import Router

    T, E, k = 400, 32, 4
    r = Router(T, E, k, True, AUX, Z)
    x = _logits(T, E, "f32", 23).cuda()
    dg = torch.randn(T * k, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r.forward(x)
        r.backward(x, dg)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            r.forward(x)
            r.backward(x, dg)
    torch.cuda.synchronize()
    x.copy_(_logits(T, E, "f32", 24))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (r.expert_idx, r.alpha, r.P, r._losses, r.dlogits)]
    r.forward(x)
    r.backward(x, dg)
    assert all(torch.equal(a, b) for a, b in zip(got, (r.expert_idx, r.alpha, r.P, r._losses, r.dlogits)))


def test_feeds_route_stats():
    # the ids, counts, P and f that the recalibration's routing statistics give for the same logits
    from fractions import Fraction

    from backward_token_expert_gb300.pipeline import Recalibration, Router

    T, E, k = 1200, 24, 3
    x = _logits(T, E, "f32", 25).cuda()
    r = Router(T, E, k, True, AUX, Z)
    r.forward(x)
    rec = Recalibration(T, E, k, 8, 8, Fraction(5, 4), Fraction(3, 4))
    try:
        rec.route_stats(x, r.expert_idx)
        torch.cuda.synchronize()
        assert rec.device_status() == 0
        assert torch.equal(rec.buf.counts, r.counts)
        assert torch.allclose(rec.buf.P, r.P, rtol=2e-5, atol=0) and torch.allclose(rec.buf.f, r.f, rtol=1e-6, atol=0)
        assert abs(rec.summary()["aux_unscaled"] - float(r.losses[1])) <= 4e-5 * float(r.losses[1])
    finally:
        rec.close()


def test_router_reports_its_device_status():
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import Router

    r = Router(4, 8, 2, True, AUX, Z)
    x = torch.zeros(4, 8, device="cuda")
    r.forward(x)
    r.expert_idx[1, 0] = 9
    r.backward(x, torch.ones(8, device="cuda"))
    assert r.device_status() == 1 << L.LRM_ERR_INDEX
    assert r.device_status() == 0


def test_router_made_while_the_current_stream_is_busy():
    # the losses' fill on the current stream does not come after another stream's forward
    from backward_token_expert_gb300.pipeline import Router

    x = _logits(50, 8, "f32", 40).cuda()
    want = Router(50, 8, 2, True, AUX, Z)
    want.forward(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ctx = want.ctx  # one that is there: making one waits for the GPU
    torch.cuda._sleep(20_000_000)
    r = Router(50, 8, 2, True, AUX, Z, ctx=ctx)
    r.forward(x, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(r._losses.view(torch.int32), want._losses.view(torch.int32)) and int(r.tokens) == 50


def test_memory_of_a_dropped_router_stays_until_its_stream_is_done():
    from backward_token_expert_gb300.pipeline import Router

    x = _logits(50, 8, "f32", 41).cuda()
    keep = Router(50, 8, 2, True, AUX, Z)
    r = Router(50, 8, 2, True, AUX, Z, ctx=keep.ctx)
    own = {t.data_ptr(): t.numel() * t.element_size() for t in (r.alpha, r.row_stats, r.expert_idx, r.dlogits, r.ws)}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    r.forward(x, stream=s)
    r.backward(x, stream=s)
    del r
    others = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in own.values() for _ in range(64)]
    assert not s.query()
    for at in own:
        assert not any(t.data_ptr() <= at < t.data_ptr() + t.numel() for t in others)
    s.synchronize()


@pytest.mark.parametrize("device", [0, "cuda", "cuda:0", torch.device("cuda"), torch.device("cuda", 0)])
def test_names_of_the_device(device):
    from backward_token_expert_gb300.pipeline import Router

    r = Router(4, 8, 2, True, AUX, Z, device=device)
    x = torch.eye(4, 8, device="cuda")
    valid = torch.ones(4, dtype=torch.uint8, device="cuda")
    r.forward(x, valid)
    r.backward(x, torch.ones(8, device="cuda"), torch.ones(8, device="cuda"))
    assert int(r.tokens) == 4 and r.expert_idx[:, 0].tolist() == [0, 1, 2, 3] and r.dlogits.device == x.device


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (700, 5, 3), (3000, 33, 4), (2500, 128, 8), (900, 500, 32), (300, 1024, 10)])
@pytest.mark.parametrize("share", [0.0, 0.4, 1.0])
def test_route_stats_of_the_counted_tokens(T, E, k, share):
    # against the statistics of a batch that holds the counted tokens alone, with garbage in the other tokens
    from fractions import Fraction

    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import Recalibration, Router

    x = _logits(T, E, "f32", T + E).cuda()
    valid = torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda") < share
    kept = valid.nonzero().flatten()
    n = kept.numel()
    r = Router(T, E, k, True, AUX, Z)
    r.forward(x, valid.to(torch.uint8))
    x[~valid] = float("nan")
    r.expert_idx[~valid] = torch.randint(-1 << 31, (1 << 31) - 1, (T - n, k), device="cuda", dtype=torch.int32)
    cf, rho = Fraction(5, 4), Fraction(2, 3)
    a, b = Recalibration(T, E, k, 8, 8, cf, rho), Recalibration(n, E, k, 8, 8, cf, rho)
    try:
        a.buf.bucket.fill_(-7)
        a.route_stats(x, r.expert_idx, counted=r.counted)
        b.route_stats(x[kept].contiguous(), r.expert_idx[kept].contiguous())
        assert a.device_status() == 0 and b.device_status() == 0
        for name in ("counts", "offsets", "quota", "f"):
            assert torch.equal(getattr(a.buf, name), getattr(b.buf, name)), name
        assert torch.allclose(a.buf.P, b.buf.P, rtol=2e-5, atol=1e-37)
        pairs = (kept[:, None] * k + torch.arange(k, device="cuda")).flatten()
        assert torch.equal(a.buf.bucket[: n * k].long(), pairs[b.buf.bucket[: n * k].long()])
        assert bool((a.buf.bucket[n * k:] == -7).all())
        sa, sb = a.summary(), b.summary()
        for name in sa:
            tol = 2e-5 * abs(sb[name]) if name in ("aux_unscaled", "sum_P") else 0
            assert abs(sa[name] - sb[name]) <= tol, name
        if n:  # a counted token's bad ids are still found
            r.expert_idx[kept[0], 0] = -(1 << 31)
            a.route_stats(x, r.expert_idx, counted=r.counted)
            assert a.device_status() == 1 << L.LRM_ERR_INDEX
            assert int(a.buf.offsets[-1]) == n * k - 1
    finally:
        a.close()
        b.close()


def test_refusals_of_the_counted_route_stats():
    from fractions import Fraction

    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import Recalibration, Router

    r, rec = Router(8, 4, 2, True, AUX, Z), Recalibration(8, 4, 2, 8, 8)
    x = torch.zeros(8, 4, device="cuda")
    r.forward(x)
    good = dict(ctx=rec.ctx, logits=x, idx=r.expert_idx, stats=r.row_stats, losses=r._losses, cf=Fraction(1), ws=rec.buf.ws_route)
    b = rec.buf

    def call(**kw):
        a = dict(good, **kw)
        L.lrm_route_stats_counted(a["ctx"], a["logits"], a["idx"], a["stats"], a["losses"], rec.dims, a["cf"],
                                  Fraction(1, 2), b.counts, b.offsets, b.bucket, b.P, b.f, b.quota, b.summary, a["ws"],
                                  rec.ws_bytes)

    call()
    inv, al = L.LRM_ERR_INVALID_ARG, L.LRM_ERR_ALIGN
    for kw, code in [(dict(ctx=None), inv), (dict(logits=None), inv), (dict(idx=None), inv), (dict(stats=None), inv),
                     (dict(losses=None), inv), (dict(cf=Fraction(0)), inv), (dict(stats=r.row_stats.data_ptr() + 4), al),
                     (dict(losses=r._losses.data_ptr() + 2), al), (dict(ws=None), L.LRM_ERR_WORKSPACE)]:
        with pytest.raises(L.LrmError) as ei:
            call(**kw)
        assert ei.value.code == code, kw
    rec.close()


@pytest.mark.parametrize("T,width", [(1, 8), (7, 264), (3000, 136), (500, 2048), (33, 65536)])
def test_counted_rows(T, width):
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import Router

    r = Router(T, 8, 2, True, AUX, Z)
    counted = torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda") < 0.5
    r.row_stats[:, 0], r.row_stats[:, 1] = 0.0, counted.float()
    rows = torch.randn(T, width, device="cuda").to(torch.bfloat16)
    rows[~counted] = float("nan")
    out = torch.full_like(rows, 5.0)
    L.lrm_counted_rows(r.ctx, rows, r.row_stats, r.dims, width, out)
    assert torch.equal(out[counted], rows[counted]) and not out[~counted].any()
    r.row_stats[0, 1] = float("nan")  # a counted token with a NaN logit
    L.lrm_counted_rows(r.ctx, rows, r.row_stats, r.dims, width, out)
    assert torch.equal(out[0].view(torch.int16), rows[0].view(torch.int16))


def test_refusals_of_counted_rows():
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import Router

    r = Router(4, 8, 2, True, AUX, Z)
    x, out = (torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    inv, al = L.LRM_ERR_INVALID_ARG, L.LRM_ERR_ALIGN
    for ctx, rows, stats, dims, width, to, code in [
            (None, x, r.row_stats, r.dims, 16, out, inv), (r.ctx, None, r.row_stats, r.dims, 16, out, inv),
            (r.ctx, x, None, r.dims, 16, out, inv), (r.ctx, x, r.row_stats, r.dims, 16, None, inv),
            (r.ctx, x, r.row_stats, r.dims, 12, out, inv), (r.ctx, x, r.row_stats, r.dims, 0, out, inv),
            (r.ctx, x, r.row_stats, r.dims, 65544, out, inv), (r.ctx, x.data_ptr() + 2, r.row_stats, r.dims, 16, out, al),
            (r.ctx, x, r.row_stats.data_ptr() + 4, r.dims, 16, out, al),
            (r.ctx, x, r.row_stats, L.dims_of(4, 8, 9, 8, 8), 16, out, L.LRM_ERR_SHAPE)]:
        with pytest.raises(L.LrmError) as ei:
            L.lrm_counted_rows(ctx, rows, stats, dims, width, to)
        assert ei.value.code == code
    L.lrm_counted_rows(r.ctx, None, None, L.dims_of(0, 8, 2, 8, 8), 16, None)


# three groups of four logits a lane, at 8, 16 and 32 lanes, and the sizes on both sides
@pytest.mark.parametrize("E,k", [(64, 6), (65, 8), (68, 1), (77, 5), (93, 8), (96, 3), (97, 8), (129, 9), (190, 16), (192, 8),
                                 (193, 10), (256, 17), (257, 8), (258, 32), (300, 20), (381, 4), (384, 8), (385, 12)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_three_groups_a_lane(E, k, dtype):
    run(700, E, k, dtype, renorm=bool(E % 2), seed=E + k)
    x = np.round(np.random.default_rng(E).standard_normal((90, E)) * 2) / 2  # ties
    run(90, E, k, dtype, logits=torch.from_numpy(x.astype(np.float32)).to(DT[dtype]), seed=E)
