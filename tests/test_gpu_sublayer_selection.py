"""The sublayer's backward where the recalibration retains a part of the pairs:
against automatic differentiation in fp64 of the same function, in which a pair
that was not retained adds to the output and passes no gradient on, neither to its
expert nor to its gate.  Tolerances as where all are retained: the same roundings."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import built_library, need_gpu, rel_fro
from test_gpu_sublayer_step import TOL, _enqueue, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    built_library()


def _reference(d, ids, retained, kept, counted, k, aux, zc, eps):
    v = {n: t.double().clone().requires_grad_(n != "dout") for n, t in d.items()}
    T, h = v["x"].shape
    E = v["W"].shape[0]
    c = torch.from_numpy(counted)
    x = v["x"]
    mean = x.mean(1, keepdim=True)
    n = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps) * v["gamma"] + v["beta"]
    n = n * c[:, None]
    logits = n @ v["Wr"].T
    p = torch.softmax(logits, 1)
    top = torch.gather(p, 1, ids)
    alpha = top / top.sum(1, keepdim=True)
    y = torch.zeros(T, h, dtype=torch.float64)
    for e in range(E):
        for passes in (True, False):
            t, j = torch.where((ids == e) & c[:, None] & (retained == passes))
            if len(t) == 0:
                continue
            ab = n[t] @ v["W1"][e].T
            I = ab.shape[1] // 2
            r = alpha[t, j][:, None] * ((ab[:, :I] * torch.sigmoid(ab[:, :I]) * ab[:, I:]) @ v["W"][e].T)
            y = y.index_add(0, t, r if passes else r.detach())
    out = x + y * torch.from_numpy(kept)
    f = torch.bincount(ids[c].reshape(-1), minlength=E).double() / (int(counted.sum()) * k)
    loss = (out * v["dout"])[c].sum() + aux * E * (f * p[c].mean(0)).sum()
    loss = loss + zc * (torch.logsumexp(logits[c], 1) ** 2).mean()
    loss.backward()
    return out.detach().numpy(), {m: v[m].grad.numpy() for m in ("x", "W", "W1", "Wr", "gamma", "beta")}


@pytest.mark.parametrize("T,E,k,h,I,cf,rho,p,masked", [
    (200, 8, 2, 64, 32, Fraction(1), Fraction(1, 2), 0.1, False),
    (333, 16, 3, 136, 72, Fraction(5, 4), Fraction(3, 4), 0.0, True),
    (300, 8, 1, 72, 40, Fraction(1, 2), Fraction(1), 0.3, False),
    (700, 24, 4, 264, 136, Fraction(1), Fraction(1, 4), 0.2, True)])
def test_gradients_of_a_part_of_the_pairs(T, E, k, h, I, cf, rho, p, masked):
    from backward_token_expert_gb300.pipeline import SublayerStep

    aux, zc, eps = 0.5, 0.1, 1e-5
    d = _inputs(T, E, h, I, T + 1)
    rng = np.random.default_rng(T)
    valid = (rng.random(T) < 0.8) if masked else np.ones(T, bool)
    if masked:
        d["x"][torch.from_numpy(~valid)] = float("nan")
        d["dout"][torch.from_numpy(~valid)] = float("nan")
    step = SublayerStep(T, E, k, h, I, cf, rho, aux, zc, max_norm=1e9, p=p, seed=3, eps=eps)
    try:
        dev = {n: t.cuda() for n, t in d.items()}
        v = torch.from_numpy(valid.astype(np.uint8)).cuda() if masked else None
        _enqueue(step, dev, torch.empty(T, E, device="cuda"), v)
        torch.cuda.synchronize()
        assert step.device_status() == 0 and int(step.clip.nonfinite) == 0 and float(step.clip.coef) == 1.0
        b = step.rec.buf
        ids = step.router.expert_idx.long().cpu()
        total = int(b.sel_offsets[-1])
        chosen = b.sel_ids[:total].long().cpu()
        dgate = step.rec.dgate.cpu().numpy()
        got = dict(dW=b.dW, dW1=step.rec.fc1.dW1, dWr=step.dWr, dgamma=step.norm.dgamma, dbeta=step.norm.dbeta,
                   dx=step.norm.dx, out=step.out)
        got = {n: t.double().cpu().numpy() for n, t in got.items()}
    finally:
        step.close()
    assert 0 < total < int(valid.sum()) * k and len(set(chosen.tolist())) == total
    retained = torch.zeros(T * k, dtype=torch.bool)
    retained[chosen] = True
    assert np.all(dgate[~retained.numpy()] == 0) and np.count_nonzero(dgate[retained.numpy()]) > 0.9 * total
    retained = retained.view(T, k)
    assert not retained[torch.from_numpy(~valid)].any()
    kept = O.dropout_kept(T * h, p, 3, 0).reshape(T, h) / (1 - p)
    clean = {n: torch.nan_to_num(t) for n, t in d.items()}
    out, ref = _reference(clean, ids, retained, kept, valid, k, aux, zc, eps)
    assert rel_fro(got["out"][valid], out[valid]) <= TOL["out"]
    for name, key in (("dW", "W"), ("dW1", "W1"), ("dWr", "Wr"), ("dgamma", "gamma"), ("dbeta", "beta"), ("dx", "x")):
        a, r = got[name], ref[key]
        if name == "dx":
            a, r = a[valid], r[valid]
        assert rel_fro(a, r) <= TOL[name], (name, rel_fro(a, r))
