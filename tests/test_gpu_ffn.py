"""The routed experts' forward and its backward against the fp64 oracle.

Tolerances, per value.  A product over K terms: products of two bf16 values are
exact in fp32 and the tensor core adds 16 of them to the accumulator at a time;
each of the K / 16 steps (one more for a remainder) loses at most 2^-22 of the
sum of the magnitudes S, so E(K) = (K / 16 + 1) 2^-22 S.  Storing bf16 adds
2^-8 of the value.  silu and silu' are evaluated in fp32 from one exponential
and one quotient: within (2 + |a|) 2^-20 of their factor."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import built_library, need_gpu

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8


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


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def _np(t):
    return t.double().cpu().numpy()


def _steps(K):
    return (K / 16 + 1) * 2.0 ** -22


def _routing(rng, T, E, k, skew, masked):
    """Pairs by expert, ascending: skewed experts, some without a pair, tokens of padding in none."""
    logits = rng.standard_normal((T, E)) - skew * np.log(rng.permutation(E) + 1.0)
    experts = np.argsort(-logits, 1)[:, :k].reshape(-1)
    kept = np.repeat(rng.random(T) < 0.8, k) if masked else np.ones(T * k, bool)
    ids = np.flatnonzero(kept)
    ids = ids[np.argsort(experts[ids], kind="stable")]
    return ids.astype(np.int64), np.searchsorted(experts[ids], np.arange(E + 1)).astype(np.int64)


def _dev(ids, offsets, spare):
    full = np.concatenate([ids, np.full(spare, 1 << 30)]).astype(np.int32)  # beyond the total: never read
    return torch.from_numpy(full).cuda(), torch.from_numpy(offsets.astype(np.int32)).cuda()


SHAPES = [  # T, E, k, h, I, skew, masked
    (1, 4, 2, 64, 32, 0.0, False), (1, 1, 1, 8, 8, 0.0, False), (3, 128, 8, 72, 40, 1.0, False),
    (256, 8, 2, 64, 32, 1.0, False), (300, 5, 3, 200, 136, 2.0, True), (520, 2, 1, 328, 64, 0.5, False),
    (900, 20, 3, 1032, 1000, 1.0, True), (700, 160, 6, 136, 264, 1.5, True), (2100, 3, 2, 64, 8, 0.3, False),
    (77, 16, 4, 8, 520, 1.0, False), (40, 1024, 32, 48, 24, 0.5, False), (513, 1, 1, 520, 776, 0.0, False),
    (64, 6, 2, 2048, 768, 0.5, False), (8, 128, 8, 264, 136, 0.5, False), (32, 2, 1, 1032, 520, 0.0, True),
    (33, 2, 1, 72, 64, 0.0, False), (13, 64, 5, 2048, 40, 3.0, True),
    # the last sizes of the kernel for few pairs and the first beyond; several tiles a cluster of one and of three stages
    (16, 2, 1, 136, 72, 0.0, False), (17, 2, 1, 136, 72, 0.0, True), (4, 32, 8, 136, 72, 1.0, False),
    (6000, 40, 2, 64, 40, 0.3, False), (6000, 40, 2, 192, 136, 0.3, True)]


@pytest.mark.parametrize("T,E,k,h,I,skew,masked", SHAPES)
@pytest.mark.parametrize("save", [True, False])
def test_forward(ctx, T, E, k, h, I, skew, masked, save):
    from backward_token_expert_gb300 import lrm as L

    rng = np.random.default_rng(T + h + I)
    ids, offsets = _routing(rng, T, E, k, skew, masked)
    N, total, spare = T * k, len(ids), 3
    x, W1 = _bf(rng, T, h), _bf(rng, E, 2 * I, h, scale=h ** -0.5)
    W, alpha = _bf(rng, E, h, I, scale=I ** -0.5), rng.random(N).astype(np.float32)
    inside = np.zeros(N, bool)
    inside[ids] = True
    x[~inside.reshape(T, k).any(1)] = float("nan")  # padding
    alpha[~inside] = 0.0
    dims = L.dims_of(T, E, k, h, I)
    dids, doff = _dev(ids, offsets, spare)
    xd, W1d, Wd, ad = x.cuda(), W1.cuda(), W.cuda(), torch.from_numpy(alpha).cuda()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    ab = torch.full((N, 2 * I), 7.0, **bf) if save else None
    phi, rows, y = torch.full((N, I), 7.0, **bf), torch.full((N, h), float("nan"), **bf), torch.empty(T, h, **bf)
    L.lrm_ffn_up(ctx, xd, W1d, doff, dids, dims, total + spare, ab, phi)
    L.lrm_ffn_down(ctx, phi, Wd, doff, dids, dims, total + spare, rows)
    L.lrm_ffn_combine(ctx, rows, ad, dims, y)
    torch.cuda.synchronize()
    assert L.lrm_get_device_status(ctx) == 0

    xn, W1n, Wn = _np(torch.nan_to_num(x)), _np(W1), _np(W)
    ab_ref, phi_ref = O.ffn_up(xn, W1n, offsets, ids, k)
    S, _ = O.ffn_up(np.abs(xn), np.abs(W1n), offsets, ids, k)
    tol = S * _steps(h)
    a, b, ta, tb = ab_ref[:, :I], ab_ref[:, I:], tol[:, :I], tol[:, I:]
    if save:
        got = _np(ab)
        assert np.all(np.abs(got[ids] - ab_ref) <= BF * (np.abs(ab_ref) + tol) + tol + 2.0 ** -133)
        assert np.all(got[~inside] == 7.0)
    # |silu'| <= 1.1
    tp = 1.1 * ta * (np.abs(b) + tb) + np.abs(a) * tb + np.abs(a * b) * (2 + np.abs(a)) * 2.0 ** -20
    got = _np(phi)
    assert np.all(np.abs(got[ids] - phi_ref) <= BF * (np.abs(phi_ref) + tp) + tp + 2.0 ** -133)
    assert np.all(got[~inside] == 7.0)
    rows_ref = O.ffn_down(got, Wn, offsets, ids)
    tr = O.ffn_down(np.abs(got), np.abs(Wn), offsets, ids) * _steps(I)
    rn = _np(rows)
    assert np.all(np.abs(rn[ids] - rows_ref) <= BF * (np.abs(rows_ref) + tr) + tr + 2.0 ** -133)
    assert np.all(np.isnan(rn[~inside]))
    al = alpha.astype(np.float64)
    y_ref = O.ffn_combine(np.nan_to_num(rn), al, k)
    ty = O.ffn_combine(np.abs(np.nan_to_num(rn)), al, k) * (k + 1) * 2.0 ** -24
    assert np.all(np.abs(_np(y) - y_ref) <= BF * (np.abs(y_ref) + ty) + ty + 2.0 ** -133)


@pytest.mark.parametrize("N,E,h,I,rows,spare", [
    (5, 2, 8, 8, 0, 3), (1, 1, 8, 8, 1, 0), (512, 8, 64, 32, 333, 40), (700, 4, 200, 16, 700, 0),
    (901, 5, 72, 136, 600, 1), (3000, 20, 264, 248, 2999, 7), (600, 3, 1032, 1496, 500, 5), (400, 160, 48, 40, 150, 2),
    (2000, 2, 128, 520, 1100, 0), (300, 1, 2048, 768, 300, 4)])
@pytest.mark.parametrize("gates", [True, False])
def test_backward(ctx, N, E, h, I, rows, spare, gates):
    from backward_token_expert_gb300 import lrm as L

    rng = np.random.default_rng(N + I)
    ids = rng.choice(N, rows, replace=False)
    of = np.sort(rng.integers(0, E, rows))
    offsets = np.searchsorted(of, np.arange(E + 1))
    room = rows + spare
    delta, W, ab = _bf(rng, room, h, scale=1e-2), _bf(rng, E, h, I, scale=h ** -0.5), _bf(rng, N, 2 * I, scale=2.0)
    delta[rows:] = float("nan")
    unused = np.ones(N, bool)
    unused[ids] = False
    ab[unused] = float("nan")  # pairs that were not retained
    dims = L.dims_of(N, E, 1, h, I)
    dids, doff = _dev(ids, offsets, spare)
    dh1 = torch.full((max(room, 1), 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    dgate = torch.full((N,), 7.0, device="cuda") if gates else None
    need = L.lrm_ffn_backward_workspace(ctx, dims, room)
    ws = torch.full((max(need, 4) // 4,), float("nan"), device="cuda")
    L.lrm_ffn_backward(ctx, delta.cuda(), W.cuda(), ab.cuda(), doff, dids, dims, room, dh1, dgate,
                       ws if gates else None, need if gates else 0)
    torch.cuda.synchronize()
    assert L.lrm_get_device_status(ctx) == 0
    got = _np(dh1)
    assert np.all(got[rows:] == 7.0)
    dn, Wn, abn = _np(delta)[:rows], _np(W), _np(torch.nan_to_num(ab))
    ref, dg_ref = O.ffn_backward(dn, Wn, abn, offsets, ids, N)
    td = np.zeros((rows, I))  # error of dphi
    dphi = np.zeros((rows, I))
    for e in range(E):
        seg = slice(offsets[e], offsets[e + 1])
        td[seg] = np.abs(dn[seg]) @ np.abs(Wn[e]) * _steps(h)
        dphi[seg] = dn[seg] @ Wn[e]
    a, b = abn[ids, :I], abn[ids, I:]
    ev = (2 + np.abs(a)) * 2.0 ** -20
    # |silu'| <= 1.1 and |silu(a)| <= |a|; the evaluation's error is relative to 1 + |a| for silu'
    ta = 1.1 * td * np.abs(b) + np.abs(dphi * b) * ev
    tb = td * np.abs(a) + np.abs(dphi * a) * ev
    t = np.concatenate([ta, tb], 1)
    assert np.all(np.abs(got[:rows] - ref) <= BF * (np.abs(ref) + t) + t + 2.0 ** -133)
    if gates:
        silu = np.abs(ref[:, I:])
        tg = np.zeros(N)
        # sums of 32 values in a lane pair, of I / 32 of those over 8 lanes
        tg[ids] = (tb * np.abs(b)).sum(1) + (silu * np.abs(b)).sum(1) * (24 + I / 256) * 2.0 ** -24
        out = _np(dgate)
        assert np.all(np.abs(out - dg_ref) <= tg)
        assert np.all(out[unused] == 0)


def test_backward_agrees_with_the_separate_steps(ctx):
    """The composed path rounds dphi to bf16 first: 2^-8 of it more, in every product it enters."""
    from backward_token_expert_gb300 import lrm as L

    rng = np.random.default_rng(3)
    N, E, h, I, rows = 1500, 7, 256, 264, 1200
    ids = rng.choice(N, rows, replace=False)
    offsets = np.searchsorted(np.sort(rng.integers(0, E, rows)), np.arange(E + 1))
    delta, W, ab = _bf(rng, rows, h).cuda(), _bf(rng, E, h, I, scale=h ** -0.5).cuda(), _bf(rng, N, 2 * I).cuda()
    dids, doff = _dev(ids, offsets, 0)
    dims = L.dims_of(N, E, 1, h, I)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    dh1, dphi, old = torch.empty(rows, 2 * I, **bf), torch.empty(rows, I, **bf), torch.empty(rows, 2 * I, **bf)
    L.lrm_ffn_backward(ctx, delta, W, ab, doff, dids, dims, rows, dh1, None, None, 0)
    L.lrm_grouped_dgrad(ctx, delta, W, doff, dims, rows, dphi)
    L.lrm_swiglu_backward(ctx, dphi, ab[dids.long()].contiguous(), doff, dims, rows, old)
    torch.cuda.synchronize()
    a, b = _np(dh1), _np(old)
    assert np.all(np.abs(a - b) <= 3 * BF * np.maximum(np.abs(a), np.abs(b)) + 2.0 ** -126)


def test_bad_ids_and_totals(ctx):
    from backward_token_expert_gb300 import lrm as L

    rng = np.random.default_rng(5)
    T, E, k, h, I = 20, 2, 2, 64, 40
    N = T * k
    ids = np.arange(N)
    offsets = np.array([0, 25, N])
    dids, doff = _dev(ids, offsets, 0)
    x, W1, W = _bf(rng, T, h).cuda(), _bf(rng, E, 2 * I, h).cuda(), _bf(rng, E, h, I).cuda()
    dims = L.dims_of(T, E, k, h, I)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    good = [torch.full((N, w), 7.0, **bf) for w in (2 * I, I, h)]

    def forward(i, o, most, out):
        L.lrm_ffn_up(ctx, x, W1, o, i, dims, most, out[0], out[1])
        L.lrm_ffn_down(ctx, out[1], W, o, i, dims, most, out[2])
        torch.cuda.synchronize()
        return L.lrm_get_device_status(ctx)

    assert forward(dids, doff, N, good) == 0
    bad_ids = dids.clone()
    bad_ids[3], bad_ids[30] = -1, N
    out = [torch.full((N, w), 7.0, **bf) for w in (2 * I, I, h)]
    assert forward(bad_ids, doff, N, out) == 1 << L.LRM_ERR_INDEX
    for g, o in zip(good, out):
        assert (o[3] == 7.0).all() and (o[30] == 7.0).all()
        keep = [u for u in range(N) if u not in (3, 30)]
        assert torch.equal(g[keep], o[keep])
    out = [torch.full((N, w), 7.0, **bf) for w in (2 * I, I, h)]
    assert forward(dids, doff, 30, out) == 1 << L.LRM_ERR_SHAPE
    for g, o in zip(good, out):
        assert torch.equal(g[:30], o[:30]) and (o[30:] == 7.0).all()
    # backward
    delta, ab = _bf(rng, N, h).cuda(), _bf(rng, N, 2 * I).cuda()
    need = L.lrm_ffn_backward_workspace(ctx, dims, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def backward(i, o, most):
        dh1, dgate = torch.full((N, 2 * I), 7.0, **bf), torch.full((N,), 7.0, device="cuda")
        L.lrm_ffn_backward(ctx, delta, W, ab, o, i, dims, most, dh1, dgate, ws, need)
        torch.cuda.synchronize()
        return dh1, dgate, L.lrm_get_device_status(ctx)

    d0, g0, flags = backward(dids, doff, N)
    assert flags == 0
    d1, g1, flags = backward(bad_ids, doff, N)
    assert flags == 1 << L.LRM_ERR_INDEX
    assert (d1[3] == 7.0).all() and (d1[30] == 7.0).all() and g1[3] == 0 and g1[30] == 0
    assert torch.equal(d0[keep], d1[keep]) and torch.equal(g0[keep], g1[keep])
    d1, g1, flags = backward(dids, doff, 30)
    assert flags == 1 << L.LRM_ERR_SHAPE
    assert torch.equal(d0[:30], d1[:30]) and (d1[30:] == 7.0).all() and (g1[30:] == 0).all()


@pytest.mark.parametrize("bad", [-1, -7, -2 ** 31])
def test_a_negative_id_is_flagged_by_every_call(ctx, bad):
    from backward_token_expert_gb300 import lrm as L

    rng = np.random.default_rng(6)
    T, E, k, h, I = 40, 2, 2, 64, 40
    N = T * k
    good, doff = _dev(np.arange(N), np.array([0, 50, N]), 0)
    ids = good.clone()
    ids[17] = bad
    x, W1, W = _bf(rng, T, h).cuda(), _bf(rng, E, 2 * I, h).cuda(), _bf(rng, E, h, I).cuda()
    delta, ab = _bf(rng, N, h).cuda(), _bf(rng, N, 2 * I).cuda()
    dims = L.dims_of(T, E, k, h, I)
    need = L.lrm_ffn_backward_workspace(ctx, dims, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    new = lambda w: torch.full((N, w), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731

    def run(i):
        phi, rows, dh1, dgate = new(I), new(h), new(2 * I), torch.full((N,), 7.0, device="cuda")
        flags = []
        for call in (lambda: L.lrm_ffn_up(ctx, x, W1, doff, i, dims, N, None, phi),
                     lambda: L.lrm_ffn_down(ctx, phi, W, doff, i, dims, N, rows),
                     lambda: L.lrm_ffn_backward(ctx, delta, W, ab, doff, i, dims, N, dh1, dgate, ws, need)):
            call()
            torch.cuda.synchronize()
            flags.append(L.lrm_get_device_status(ctx))
        return flags, (phi, rows, dh1, dgate)

    flags, want = run(good)
    assert flags == [0, 0, 0]
    flags, got = run(ids)
    assert flags == [1 << L.LRM_ERR_INDEX] * 3
    keep = [r for r in range(N) if r != 17]
    for a, b in zip(want, got):
        assert torch.equal(a[keep], b[keep])
    assert (got[0][17] == 7.0).all() and (got[1][17] == 7.0).all() and (got[2][17] == 7.0).all() and got[3][17] == 0


def test_extreme_activations(ctx):
    """Gates far below and above zero, infinities and NaN reach their own pair's outputs only."""
    from backward_token_expert_gb300 import lrm as L

    T, E, k, h, I = 6, 1, 1, 8, 8
    x = torch.zeros(T, h, dtype=torch.bfloat16)
    x[:, 0] = torch.tensor([-1000.0, 1000.0, 0.0, -80.0, float("nan"), 1.0])
    W1 = torch.zeros(E, 2 * I, h, dtype=torch.bfloat16)
    W1[0, :, 0] = 1.0
    dids, doff = _dev(np.arange(T), np.array([0, T]), 0)
    phi = torch.empty(T, I, dtype=torch.bfloat16, device="cuda")
    ab = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    dims = L.dims_of(T, E, k, h, I)
    L.lrm_ffn_up(ctx, x.cuda(), W1.cuda(), doff, dids, dims, T, ab, phi)
    torch.cuda.synchronize()
    p = _np(phi)
    a = x[:, 0].double().numpy()
    assert np.all(p[0] == 0) and np.all(p[1] == 999424.0) and np.all(p[2] == 0) and np.isnan(p[4]).all()
    ref = a[5] * a[5] / (1 + np.exp(-a[5]))
    assert np.all(np.abs(p[5] - ref) <= BF * ref)
    assert np.all(np.abs(p[3]) < 1e-30)


def test_same_bits_in_a_graph_and_on_another_stream(ctx):
    from backward_token_expert_gb300 import lrm as L

    rng = np.random.default_rng(8)
    T, E, k, h, I = 600, 6, 2, 192, 96
    ids, offsets = _routing(rng, T, E, k, 1.0, False)
    N = T * k
    dids, doff = _dev(ids, offsets, 0)
    x, W1, W = _bf(rng, T, h).cuda(), _bf(rng, E, 2 * I, h).cuda(), _bf(rng, E, h, I).cuda()
    alpha = torch.rand(N, device="cuda")
    dims = L.dims_of(T, E, k, h, I)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    need = L.lrm_ffn_backward_workspace(ctx, dims, N)
    delta = _bf(rng, N, h).cuda()

    def buffers():
        return dict(ab=torch.zeros(N, 2 * I, **bf), phi=torch.zeros(N, I, **bf), rows=torch.zeros(N, h, **bf),
                    y=torch.zeros(T, h, **bf), dh1=torch.zeros(N, 2 * I, **bf), dgate=torch.zeros(N, device="cuda"),
                    ws=torch.zeros(need, dtype=torch.uint8, device="cuda"))

    def run(b, stream=None):
        L.lrm_ffn_up(ctx, x, W1, doff, dids, dims, N, b["ab"], b["phi"], stream)
        L.lrm_ffn_down(ctx, b["phi"], W, doff, dids, dims, N, b["rows"], stream)
        L.lrm_ffn_combine(ctx, b["rows"], alpha, dims, b["y"], stream)
        L.lrm_ffn_backward(ctx, delta, W, b["ab"], doff, dids, dims, N, b["dh1"], b["dgate"], b["ws"], need, stream)

    a, b, c = buffers(), buffers(), buffers()
    run(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(b, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for name in ("ab", "phi", "rows", "y", "dh1", "dgate"):
        assert torch.equal(a[name], b[name]) and torch.equal(a[name], c[name]), name


def test_short_wait_budgets_leave_the_context_usable():
    """Waits that may run out at once: a call either gives its result or is flagged, and the next one is whole."""
    from backward_token_expert_gb300 import lrm as L

    own = L.lrm_create(0)
    try:
        rng = np.random.default_rng(17)
        T, E, k, h, I = 700, 5, 2, 520, 264
        N = T * k
        ids, offsets = _routing(rng, T, E, k, 0.5, False)
        dids, doff = _dev(ids, offsets, 0)
        x, W1, W = _bf(rng, T, h).cuda(), _bf(rng, E, 2 * I, h).cuda(), _bf(rng, E, h, I).cuda()
        delta, dims = _bf(rng, N, h).cuda(), L.dims_of(T, E, k, h, I)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        need = L.lrm_ffn_backward_workspace(own, dims, N)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        gamma = torch.ones(h, device="cuda")
        nws = torch.empty(L.lrm_layer_norm_workspace(own, T, h), dtype=torch.uint8, device="cuda")

        def run():
            o = dict(ab=torch.zeros(N, 2 * I, **bf), phi=torch.zeros(N, I, **bf), rows=torch.zeros(N, h, **bf),
                     dh1=torch.zeros(N, 2 * I, **bf), dgate=torch.zeros(N, device="cuda"),
                     dx=torch.zeros(T, h, device="cuda"), dg=torch.zeros(h, device="cuda"),
                     db=torch.zeros(h, device="cuda"))
            L.lrm_ffn_up(own, x, W1, doff, dids, dims, N, o["ab"], o["phi"])
            L.lrm_ffn_down(own, o["phi"], W, doff, dids, dims, N, o["rows"])
            L.lrm_ffn_backward(own, delta, W, o["ab"], doff, dids, dims, N, o["dh1"], o["dgate"], ws, need)
            xf, stats = x.float(), torch.ones(T, 2, device="cuda")
            L.lrm_layer_norm_backward(own, xf, L.DTYPE_F32, xf, gamma, stats, None, None, T, h, o["dx"], o["dg"],
                                      o["db"], nws, nws.numel())
            torch.cuda.synchronize()
            return o, L.lrm_get_device_status(own)

        want, flags = run()
        assert flags == 0
        for budget in (0, 1000, 100000):
            L.lrm_set_wait_budget(own, budget)
            got, flags = run()
            assert flags in (0, 1 << L.LRM_ERR_TIMEOUT)
            assert flags or all(torch.equal(a, b) for a, b in zip(want.values(), got.values()))
        L.lrm_set_wait_budget(own, 2000000000)
        got, flags = run()
        assert flags == 0 and all(torch.equal(a, b) for a, b in zip(want.values(), got.values()))
    finally:
        L.lrm_destroy(own)


def test_two_streams_and_offsets_beyond_32_bits(ctx):
    """Two calls at once on two streams, and rows of ab past 2^31 elements."""
    from backward_token_expert_gb300 import lrm as L

    rng = np.random.default_rng(23)
    I, h, E, k = 4096, 64, 2, 1
    T = (1 << 31) // (2 * I) + 300
    x, W1 = torch.zeros(T, h, dtype=torch.bfloat16, device="cuda"), _bf(rng, E, 2 * I, h, scale=h ** -0.5).cuda()
    x[-200:] = _bf(rng, 200, h).cuda()
    ids = torch.arange(T, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, T - 100, T], dtype=torch.int32, device="cuda")
    dims = L.dims_of(T, E, k, h, I)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ab, phi = torch.full((T, 2 * I), 7.0, **bf), torch.full((T, I), 7.0, **bf)
            L.lrm_ffn_up(ctx, x, W1, off, ids, dims, T, ab, phi, s)
            outs.append((ab, phi))
    torch.cuda.synchronize()
    assert L.lrm_get_device_status(ctx) == 0
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    ab, phi = outs[0]
    assert (ab[:-200] == 0).all() and (phi[:-200] == 0).all()
    got, W1n, xn = _np(ab[-200:]), _np(W1), _np(x[-200:])
    for e, rows in ((0, slice(0, 100)), (1, slice(100, 200))):
        ref, S = xn[rows] @ W1n[e].T, np.abs(xn[rows]) @ np.abs(W1n[e]).T * _steps(h)
        assert np.all(np.abs(got[rows] - ref) <= BF * (np.abs(ref) + S) + S + 2.0 ** -133)
    # the backward reads those rows
    delta, W = _bf(rng, 200, h).cuda(), _bf(rng, E, h, I, scale=h ** -0.5).cuda()
    dh1 = torch.empty(200, 2 * I, **bf)
    soff = torch.tensor([0, 100, 200], dtype=torch.int32, device="cuda")
    L.lrm_ffn_backward(ctx, delta, W, ab, soff, ids[-200:].contiguous(), dims, 200, dh1, None, None, 0)
    torch.cuda.synchronize()
    assert L.lrm_get_device_status(ctx) == 0
    ref, _ = O.ffn_backward(_np(delta), _np(W), got, np.array([0, 100, 200]), np.arange(200), 200)
    a, b = got[:, :I], got[:, I:]
    td = np.concatenate([np.abs(_np(delta)[r]) @ np.abs(_np(W)[e]) for e, r in ((0, slice(0, 100)), (1, slice(100, 200)))])
    td = td * _steps(h)
    size = np.concatenate([td * 1.1 * np.abs(b), td * np.abs(a)], 1)
    dphi = np.concatenate([_np(delta)[r] @ _np(W)[e] for e, r in ((0, slice(0, 100)), (1, slice(100, 200)))])
    ev = (2 + np.abs(a)) * 2.0 ** -20
    size += np.concatenate([np.abs(dphi * b) * ev, np.abs(dphi * a) * ev], 1)
    assert np.all(np.abs(_np(dh1) - ref) <= BF * (np.abs(ref) + size) + size + 2.0 ** -133)


def test_refusals(ctx):
    from backward_token_expert_gb300 import lrm as L

    d = L.dims_of(16, 4, 2, 64, 32)
    z = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    p = z.data_ptr()
    up = lambda **k: L.lrm_ffn_up(ctx, *[k.get(n, v) for n, v in  # noqa: E731
                                         dict(x=p, W1=p, off=p, ids=p, dims=d, most=8, ab=p, phi=p).items()])
    down = lambda **k: L.lrm_ffn_down(ctx, *[k.get(n, v) for n, v in  # noqa: E731
                                             dict(phi=p, W=p, off=p, ids=p, dims=d, most=8, rows=p).items()])
    comb = lambda **k: L.lrm_ffn_combine(ctx, *[k.get(n, v) for n, v in  # noqa: E731
                                                dict(rows=p, alpha=p, dims=d, out=p).items()])
    bwd = lambda **k: L.lrm_ffn_backward(ctx, *[k.get(n, v) for n, v in  # noqa: E731
                                                dict(delta=p, W=p, ab=p, off=p, ids=p, dims=d, most=8, dh1=p, dgate=p,
                                                     ws=p, nb=1 << 20).items()])
    inv, al, shape, wsp = L.LRM_ERR_INVALID_ARG, L.LRM_ERR_ALIGN, L.LRM_ERR_SHAPE, L.LRM_ERR_WORKSPACE
    cases = [(up, dict(x=None), inv), (up, dict(W1=None), inv), (up, dict(off=None), inv), (up, dict(ids=None), inv),
             (up, dict(phi=None), inv), (up, dict(most=-1), inv), (up, dict(x=p + 2), al), (up, dict(ab=p + 8), al),
             (up, dict(ids=p + 1), al), (up, dict(dims=L.dims_of(16, 4, 2, 60, 32)), al),
             (up, dict(dims=L.dims_of(16, 4, 2, 64, 65544)), shape), (up, dict(dims=L.dims_of(16, 4, 5, 64, 32)), shape),
             (down, dict(phi=None), inv), (down, dict(W=None), inv), (down, dict(rows=None), inv),
             (down, dict(rows=p + 4), al), (down, dict(W=p + 8), al), (comb, dict(rows=None), inv),
             (comb, dict(alpha=None), inv), (comb, dict(out=None), inv), (comb, dict(out=p + 8), al),
             (comb, dict(alpha=p + 2), al), (bwd, dict(delta=None), inv), (bwd, dict(ab=None), inv),
             (bwd, dict(dh1=None), inv), (bwd, dict(ids=None), inv), (bwd, dict(ws=None), wsp), (bwd, dict(nb=31), wsp),
             (bwd, dict(dh1=p + 8), al), (bwd, dict(dgate=p + 2), al), (bwd, dict(ws=p + 2), al)]
    for call, kw, code in cases:
        with pytest.raises(L.LrmError) as ei:
            call(**kw)
        assert ei.value.code == code, kw
    up(most=0)
    down(dims=L.dims_of(0, 4, 2, 64, 32))
    comb(dims=L.dims_of(0, 4, 2, 64, 32))
    bwd(most=0, delta=None, ws=None, nb=0)
    torch.cuda.synchronize()
    assert L.lrm_get_device_status(ctx) == 0
