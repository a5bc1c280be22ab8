"""A layer's training step (router forward, recalibrated backward, router
backward, clipping) against the fp64 oracle, run on the GPU's own selection.

Tolerances: the experts' products are held to the path's 5e-3 relative
Frobenius bound.  The gate gradients pass two roundings to bf16 (the weighted
cotangent and dphi, 2^-9 each); the logits' gradient is stored as bf16 (2^-9)
before the router's own products, whose inputs are otherwise exact: 5e-3 holds
there too, as it does for the norm of all of them."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import bf16_np, built_library, custom_inputs, need_gpu, rel_fro
from workloads import fc1_inputs
from workloads.generate import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

RTOL = 5e-3


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    built_library()


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


@pytest.mark.parametrize("T,E,k,h,I,masked,clipped", [(256, 8, 2, 64, 32, False, True), (1000, 24, 3, 136, 72, True, True),
                                                     (333, 16, 4, 64, 40, True, False)])
def test_step_against_the_oracle(T, E, k, h, I, masked, clipped):
    from backward_token_expert_gb300.pipeline import TrainingStep

    aux, zc = 0.5, 0.1
    inp = custom_inputs(T=T, E=E, k=k, h=h, I=I, s=1.0, rho=Fraction(3, 4), seed=61)
    w, f1 = inp.workload, fc1_inputs(inp.workload)
    rng = np.random.default_rng(7)
    Wr = f32_to_bf16_bits((rng.standard_normal((E, h)) * 0.05).astype(np.float32))
    valid = (rng.random(T) < 0.8) if masked else None
    step = TrainingStep(T, E, k, h, I, w.cf, w.rho, aux, zc, max_norm=1e9)
    try:
        logits = torch.from_numpy(inp.logits).cuda()
        v = None if valid is None else torch.from_numpy(valid.astype(np.uint8)).cuda()
        args = [_dev(a) for a in (inp.g, inp.phi, inp.W, f1.x, f1.ab, f1.W1, Wr)]
        step.route(logits, v)
        step.backward(logits, *args)
        torch.cuda.synchronize()
        assert step.device_status() == 0
        r, rec = step.router, step.rec
        unclipped = [t.clone() for t in step.clip.grads]
        norm = float(step.clip.norm)
        assert float(step.clip.coef) == 1.0 and int(step.clip.nonfinite) == 0
        if clipped:
            step.max_norm = 0.25 * norm
            step.route(logits, v)
            step.backward(logits, *args)
            torch.cuda.synchronize()
            assert step.device_status() == 0 and float(step.clip.norm) == norm
            for a, b in zip(unclipped, step.clip.grads):
                assert torch.equal(b, a * step.clip.coef)
        so = rec.buf.sel_offsets.cpu().numpy().astype(np.int64)
        ids = rec.buf.sel_ids[: so[-1]].cpu().numpy().astype(np.int64)
        dW, dW1, dWr = (t.cpu().numpy() for t in unclipped)
        dlogits, dxr = O.bf16_to_f64(bf16_np(r.dlogits)), O.bf16_to_f64(bf16_np(step.dxr))
        losses, alpha_gpu, idx_gpu = r.losses.cpu().numpy(), r.alpha.cpu().numpy(), r.expert_idx.cpu().numpy()
    finally:
        step.close()

    ref = O.router_forward(inp.logits, k, True, aux, zc, valid)
    assert np.array_equal(idx_gpu, ref["expert_idx"])
    assert abs(losses[0] - ref["loss"]) <= 1e-4 * ref["loss"]
    alpha = ref["alpha"].reshape(-1)
    # the pairs of tokens that are not counted have score 0 and go first
    ref_dW = O.grouped_wgrad(inp.g, inp.phi, alpha_gpu, so, ids, E, k)
    for e in range(E):
        if np.linalg.norm(ref_dW[e]) > 0:
            assert rel_fro(dW[e], ref_dW[e]) <= RTOL
    g, phi, W, x = (O.bf16_to_f64(a) for a in (inp.g, inp.phi, inp.W, f1.x))
    dgate = np.zeros(T * k)
    for u in ids:
        dgate[u] = alpha[u] * (g[u // k] @ W[ref["expert_idx"][u // k, u % k]] @ phi[u])
    ref_dl = O.router_backward(inp.logits, ref["expert_idx"], ref["alpha"], ref["f"], ref["tokens"],
                               dgate.reshape(T, k), True, aux, zc, ref["counted"])
    assert rel_fro(dlogits, ref_dl) <= RTOL
    if masked:
        assert np.all(dlogits[~ref["counted"]] == 0) and np.all(dxr[~ref["counted"]] == 0)
    assert rel_fro(dWr, ref_dl.T @ x) <= RTOL
    assert rel_fro(dxr, ref_dl @ O.bf16_to_f64(Wr)) <= RTOL
    want = np.sqrt(sum(float((a.astype(np.float64) ** 2).sum()) for a in (dW, dW1, dWr)))
    assert abs(norm - want) <= 1e-6 * want


def test_refusals():
    from backward_token_expert_gb300.pipeline import TrainingStep

    for kw in (dict(E=12), dict(max_norm=-1.0), dict(max_norm=float("nan"))):
        with pytest.raises(ValueError):
            TrainingStep(**dict(dict(T=64, E=8, k=2, h=64, I=32), **kw))


def test_a_step_on_the_device_named_without_its_index():
    from backward_token_expert_gb300.pipeline import TrainingStep

    T, E, k, h, I = 64, 8, 2, 64, 32
    bf = dict(dtype=torch.bfloat16, device="cuda")
    step = TrainingStep(T, E, k, h, I, device="cuda")
    try:
        logits = torch.randn(T, E, device="cuda")
        step.route(logits)
        step.backward(logits, torch.randn(T, h, **bf), torch.randn(T * k, I, **bf), torch.randn(E, h, I, **bf),
                      torch.randn(T, h, **bf), torch.randn(T * k, 2 * I, **bf), torch.randn(E, 2 * I, h, **bf),
                      torch.randn(E, h, **bf))
        assert step.device_status() == 0 and int(step.clip.nonfinite) == 0
        assert abs(float(torch.cat([g.double().flatten() for g in step.clip.grads]).norm()) - 1.0) <= 1e-5
    finally:
        step.close()


def _batch(T, E, k, h, I, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = lambda *n: torch.randn(*n, generator=g, device="cuda").mul_(0.3).to(torch.bfloat16)  # noqa: E731
    skew = torch.linspace(1.5, -1.5, E, device="cuda")
    return (torch.randn(T, E, generator=g, device="cuda") + skew, bf(T, h), bf(T * k, I), bf(T, h), bf(T * k, 2 * I),
            bf(E, h, I), bf(E, 2 * I, h), bf(E, h))


def _step(T, E, k, h, I, batch, valid=None):
    """Results of a step, cloned; a batch of its own shape."""
    from backward_token_expert_gb300.pipeline import TrainingStep

    logits, g, phi, x, ab, W, W1, Wr = batch
    step = TrainingStep(T, E, k, h, I, Fraction(5, 4), Fraction(3, 4), 0.5, 0.1, max_norm=1e9)
    try:
        step.route(logits, valid)
        step.backward(logits, g, phi, W, x, ab, W1, Wr)
        torch.cuda.synchronize()
        assert step.device_status() == 0
        r, b = step.router, step.rec.buf
        total = int(b.sel_offsets[-1])
        out = dict(counts=b.counts, router_counts=r.counts, quota=b.quota, offsets=b.offsets, f=b.f, P=b.P,
                   sel_offsets=b.sel_offsets, sel_ids=b.sel_ids[:total], dW=b.dW, dW1=step.rec.fc1.dW1,
                   dx=step.rec.fc1.dx, dgate=step.rec.dgate, dlogits=r.dlogits, dxr=step.dxr, dWr=step.dWr,
                   norm=step.clip.norm, P_router=r.P, f_router=r.f)
        return {n: t.clone() for n, t in out.items()}, step.rec.summary()
    finally:
        step.close()


@pytest.mark.parametrize("T,E,k,share", [(600, 8, 2, 0.5), (1500, 24, 4, 0.3), (333, 16, 4, 0.9), (2100, 40, 8, 0.05)])
def test_padding_takes_no_part(T, E, k, share):
    # the step of a padded batch against that of the batch without its padding
    h, I = 64, 40
    batch = _batch(T, E, k, h, I, T)
    valid = torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(E), device="cuda") < share
    kept = valid.nonzero().flatten()
    n = kept.numel()
    pairs = (kept[:, None] * k + torch.arange(k, device="cuda")).flatten()
    logits, g, phi, x, ab, W, W1, Wr = batch
    alone, alone_summary = _step(n, E, k, h, I, (logits[kept], g[kept], phi[pairs], x[kept], ab[pairs], W, W1, Wr))
    for t in (logits, g):
        t[~valid] = float("nan")
    pad_pairs = torch.ones(T * k, dtype=torch.bool, device="cuda")
    pad_pairs[pairs] = False
    phi[pad_pairs], ab[pad_pairs] = float("inf"), float("nan")
    got, summary = _step(T, E, k, h, I, batch, valid.to(torch.uint8))
    for name in ("counts", "router_counts", "quota", "offsets", "f", "sel_offsets", "dW", "dW1"):
        assert torch.equal(got[name], alone[name]), name
    assert torch.equal(got["counts"], got["router_counts"]) and torch.equal(got["f"], got["f_router"])
    assert torch.allclose(got["P"], got["P_router"], rtol=2e-5, atol=0)
    assert torch.equal(got["sel_ids"].long(), pairs[alone["sel_ids"].long()])
    for name in ("dx", "dlogits", "dxr"):
        assert torch.equal(got[name][kept], alone[name]) and not got[name][~valid].any(), name
    assert torch.equal(got["dgate"][pairs], alone["dgate"]) and not got["dgate"][pad_pairs].any()
    for name in ("N", "C", "slots", "dropped", "retained", "max_count", "min_count", "nonempty", "drop_rate", "rho_real"):
        assert summary[name] == alone_summary[name], name
    assert abs(summary["aux_unscaled"] - alone_summary["aux_unscaled"]) <= 2e-5 * alone_summary["aux_unscaled"]
    # fp32 sums of the same products in another order
    mag = alone["dlogits"].double().abs().t() @ x[kept].double().abs()
    assert bool(((got["dWr"] - alone["dWr"]).abs() <= 2 * T * 2.0 ** -24 * mag).all())


def test_no_token_of_a_batch_counts():
    T, E, k, h, I = 100, 8, 2, 64, 32
    batch = _batch(T, E, k, h, I, 5)
    got, summary = _step(T, E, k, h, I, batch, torch.zeros(T, dtype=torch.uint8, device="cuda"))
    assert summary["N"] == summary["C"] == summary["retained"] == 0
    for name in ("counts", "quota", "offsets", "f", "P", "dW", "dW1", "dx", "dgate", "dlogits", "dxr", "dWr", "norm"):
        assert not got[name].any(), name


def test_rows_of_minus_infinity_take_no_part():
    T, E, k, h, I = 200, 8, 2, 64, 32
    batch = _batch(T, E, k, h, I, 6)
    batch[0][::3] = -float("inf")
    got, summary = _step(T, E, k, h, I, batch)
    dead = torch.arange(T, device="cuda") % 3 == 0
    assert summary["N"] == 2 * int((~dead).sum()) and torch.isfinite(got["P"]).all()
    assert torch.equal(got["counts"], got["router_counts"]) and not got["dx"][dead].any()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
def test_garbage_in_the_paddings_inputs_reaches_no_result(fill):
    T, E, k, h, I = 500, 16, 3, 72, 40
    batch = _batch(T, E, k, h, I, 8)
    valid = torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda") < 0.6
    want, _ = _step(T, E, k, h, I, batch, valid.to(torch.uint8))
    logits, g, phi, x, ab, *_ = batch
    for t in (logits, g, x):
        t[~valid] = fill
    phi.view(T, k, I)[~valid] = fill
    ab.view(T, k, 2 * I)[~valid] = fill
    got, _ = _step(T, E, k, h, I, batch, valid.to(torch.uint8))
    for name, t in want.items():
        assert torch.isfinite(t.float()).all() and torch.equal(got[name], t), name


def test_a_step_with_and_without_a_mask_in_turn():
    from backward_token_expert_gb300.pipeline import TrainingStep

    T, E, k, h, I = 300, 8, 2, 64, 32
    logits, g, phi, x, ab, W, W1, Wr = _batch(T, E, k, h, I, 10)
    valid = torch.ones(T, dtype=torch.uint8, device="cuda")
    valid[::4] = 0
    step = TrainingStep(T, E, k, h, I, max_norm=1e9)
    try:
        got = []
        for v in (None, valid, None, valid):
            step.route(logits, v)
            step.backward(logits, g, phi, W, x, ab, W1, Wr)
            got.append([t.clone() for t in (step.dWr, step.rec.buf.dW, step.rec.fc1.dW1, step.dxr)])
        assert step.device_status() == 0
        assert all(torch.equal(a, b) for i in (0, 1) for a, b in zip(got[i], got[i + 2]))
        assert not torch.equal(got[0][0], got[1][0])
    finally:
        step.close()


@pytest.mark.parametrize("masked", [False, True])
def test_a_first_step_on_another_stream_beside_a_busy_one(masked):
    # work pending on the current stream over memory that it has given back: no buffer of the step may take it
    from backward_token_expert_gb300.pipeline import TrainingStep

    T, E, k, h, I = 300, 8, 2, 64, 32
    logits, g, phi, x, ab, W, W1, Wr = _batch(T, E, k, h, I, 11)
    valid = (torch.arange(T, device="cuda") % 4 != 0).to(torch.uint8) if masked else None
    step, want = TrainingStep(T, E, k, h, I, max_norm=1e9), TrainingStep(T, E, k, h, I, max_norm=1e9)
    try:
        s = torch.cuda.Stream()
        want.route(logits, valid)
        want.backward(logits, g, phi, W, x, ab, W1, Wr)
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        for n in (T * k, T * h):  # of the gate gradients' size, and of x's
            held = [torch.empty(n * b, dtype=torch.uint8, device="cuda") for b in (2, 4) for _ in range(20)]
            [t.fill_(255) for t in held]
            del held
        step.route(logits, valid, s)
        step.backward(logits, g, phi, W, x, ab, W1, Wr, s)
        torch.cuda.synchronize()
        assert step.device_status() == 0
        for a, b in ((step.rec.dgate, want.rec.dgate), (step.dWr, want.dWr), (step.dxr, want.dxr),
                     (step.rec.buf.dW, want.rec.buf.dW), (step.rec.fc1.dx, want.rec.fc1.dx)):
            assert torch.equal(a, b)
    finally:
        step.close()
        want.close()


@pytest.mark.parametrize("T,E,k,h,I,masked,dead", [(256, 8, 2, 64, 32, False, 0), (1000, 24, 3, 136, 72, True, 3),
                                                  (700, 16, 4, 64, 40, True, 1)])
def test_selection_and_fc1_side_against_the_oracle(T, E, k, h, I, masked, dead):
    # quotas and selection from the oracle's statistics of the counted tokens; dW1, dx and the empty experts' zeros
    # from the GPU's own input-gradient rows, whose products are held to the path's bound
    from backward_token_expert_gb300.pipeline import TrainingStep

    inp = custom_inputs(T=T, E=E, k=k, h=h, I=I, s=1.0, rho=Fraction(3, 4), seed=62, dead=dead)
    w, f1 = inp.workload, fc1_inputs(inp.workload)
    rng = np.random.default_rng(8)
    Wr = f32_to_bf16_bits((rng.standard_normal((E, h)) * 0.05).astype(np.float32))
    valid = rng.random(T) < 0.6 if masked else np.ones(T, bool)
    step = TrainingStep(T, E, k, h, I, w.cf, w.rho, 0.5, 0.1, max_norm=1e9)
    try:
        logits = torch.from_numpy(inp.logits).cuda()
        step.route(logits, torch.from_numpy(valid.astype(np.uint8)).cuda() if masked else None)
        step.backward(logits, *[_dev(a) for a in (inp.g, inp.phi, inp.W, f1.x, f1.ab, f1.W1, Wr)])
        torch.cuda.synchronize()
        assert step.device_status() == 0
        b = step.rec.buf
        so = b.sel_offsets.cpu().numpy().astype(np.int64)
        ids = b.sel_ids[: so[-1]].cpu().numpy().astype(np.int64)
        quota, score, idx = b.quota.cpu().numpy(), b.score.cpu().numpy()[: T * k], step.router.expert_idx.cpu().numpy()
        dphi_c = O.bf16_to_f64(bf16_np(b.dphi_c[: so[-1]]))
        dW, dW1 = b.dW.cpu().numpy(), step.rec.fc1.dW1.cpu().numpy()
        dx = O.bf16_to_f64(bf16_np(step.rec.fc1.dx))
    finally:
        step.close()

    kept = np.flatnonzero(valid)
    pairs = (kept[:, None] * k + np.arange(k)).reshape(-1)
    st = O.route_stats(inp.logits[kept], idx[kept], E, w.cf, w.rho)
    assert np.array_equal(quota, st["quota"])
    ref_so, ref_ids = O.select(score[pairs].astype(np.float64), idx[kept], E, st["quota"])
    assert np.array_equal(so, ref_so) and np.array_equal(ids, pairs[ref_ids])
    ref_dW1, ref_rows = O.fc1_backward(O.bf16_to_f64(f1.x[ids // k]), O.bf16_to_f64(f1.ab[ids]),
                                       {e: O.bf16_to_f64(f1.W1[e]) for e in range(E)}, dphi_c, so, np.arange(ids.size),
                                       E, 1)
    empty = 0
    for e in range(E):
        if so[e] == so[e + 1]:
            empty += 1
            assert np.all(dW[e] == 0) and np.all(dW1[e] == 0)
        else:
            assert rel_fro(dW1[e], ref_dW1[e]) <= RTOL
    assert empty >= dead
    ref_dx = O.combine_pairs(ref_rows, ids, T, k)
    assert rel_fro(dx, ref_dx) <= RTOL
    none = np.ones(T, bool)
    none[ids // k] = False
    assert np.all(dx[none] == 0) and (not masked or none[~valid].all())


def test_statistics_of_the_counted_tokens_on_a_side_stream():
    from backward_token_expert_gb300.pipeline import Recalibration, Router

    T, E, k, h, I = 900, 16, 4, 64, 40
    logits, g, phi, _, _, W, _, _ = _batch(T, E, k, h, I, 12)
    valid = (torch.arange(T, device="cuda") % 3 != 0).to(torch.uint8)
    rec = Recalibration(T, E, k, h, I)
    r = Router(T, E, k, ctx=rec.ctx)
    try:
        r.forward(logits, valid)
        got = []
        for side in (None, torch.cuda.Stream()):
            rec.run(logits, r.expert_idx, g, phi, r.alpha, W, side_stream=side, counted=r.counted)
            got.append([t.clone() for t in (rec.buf.counts, rec.buf.quota, rec.buf.sel_offsets, rec.buf.dW)])
        assert rec.device_status() == 0 and torch.equal(got[0][0], r.counts)
        assert all(torch.equal(a, b) for a, b in zip(*got))
    finally:
        r.close()
        rec.close()
