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
