"""The training step of a whole sublayer (layer norm, router, experts, dropout,
residual; backward; clipping) against automatic differentiation of the same
function in fp64 on the CPU, with the ids that the router chose.

Tolerances, relative Frobenius.  Between two fp32 computations a value is stored
as bf16: off by at most 2^-8, 2.3e-3 in the root mean square whatever the
mantissas.  m such roundings in a chain of products add up to sqrt(m) 2.3e-3:
the output passes four (n, phi, rows, y) and its own, the experts' weight
gradients five (n, ab, g, delta, dh1 or phi), the input's nine (those and dxc,
dx, dn, dx), the gates' gradient four and dlogits one, of differences whose
cancellation is given a factor of three."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import built_library, need_gpu, rel_fro

pytestmark = pytest.mark.gpu

R = 2.3e-3
TOL = dict(out=5 ** 0.5 * R, dW=5 ** 0.5 * R, dW1=5 ** 0.5 * R, dWr=3 * 6 ** 0.5 * R, dgamma=9 ** 0.5 * R, dbeta=9 ** 0.5 * R,
           dx=9 ** 0.5 * R)


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    built_library()


def _inputs(T, E, h, I, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale)  # noqa: E731
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731
    return dict(x=bf(r(T, h)), W1=bf(r(E, 2 * I, h, scale=h ** -0.5)), W=bf(r(E, h, I, scale=I ** -0.5)),
                Wr=bf(r(E, h, scale=h ** -0.5)), gamma=1 + 0.2 * r(h), beta=0.1 * r(h), dout=bf(r(T, h)))


def _enqueue(step, d, logits, valid=None, stream=None):
    """One step as a program runs it; `logits` is the router product's buffer."""
    n = step.normalize(d["x"], d["gamma"], d["beta"], valid, stream)
    torch.matmul(n.float(), d["Wr"].float().T, out=logits)
    step.route(logits, valid, stream)
    step.experts(d["x"], d["W1"], d["W"], stream)
    return step.backward(d["dout"], d["x"], d["W"], d["W1"], d["Wr"], d["gamma"], stream)


def _reference(d, ids, kept, counted, k, aux, zc, eps):
    """fp64 autograd of sum(out dout) + the losses, ids and the dropout's mask given."""
    v = {n: t.double().clone().requires_grad_(n != "dout") for n, t in d.items()}
    T, h = v["x"].shape
    E = v["W"].shape[0]
    c = torch.from_numpy(counted)
    mean = v["x"].mean(1, keepdim=True)
    var = ((v["x"] - mean) ** 2).mean(1, keepdim=True)
    n = (v["x"] - mean) / torch.sqrt(var + eps) * v["gamma"] + v["beta"]
    n = n * c[:, None]
    logits = n @ v["Wr"].T
    p = torch.softmax(logits, 1)
    top = torch.gather(p, 1, ids)
    alpha = top / top.sum(1, keepdim=True)
    y = torch.zeros(T, h, dtype=torch.float64)
    for e in range(E):
        t, j = torch.where((ids == e) & c[:, None])
        if len(t):
            ab = n[t] @ v["W1"][e].T
            I = ab.shape[1] // 2
            phi = ab[:, :I] * torch.sigmoid(ab[:, :I]) * ab[:, I:]
            y = y.index_add(0, t, alpha[t, j][:, None] * (phi @ v["W"][e].T))
    out = v["x"] + y * torch.from_numpy(kept)
    Tc = int(counted.sum())
    f = torch.bincount(ids[c].reshape(-1), minlength=E).double() / (Tc * k)
    lse = torch.logsumexp(logits[c], 1)
    loss = (out * v["dout"])[c].sum() + aux * E * (f * p[c].mean(0)).sum() + zc * (lse ** 2).mean()
    loss.backward()
    return out.detach().numpy(), {n: v[n].grad.numpy() for n in ("x", "W", "W1", "Wr", "gamma", "beta")}


@pytest.mark.parametrize("T,E,k,h,I,p,masked", [(200, 8, 2, 64, 32, 0.0, False), (333, 16, 3, 136, 72, 0.3, True),
                                                (64, 8, 1, 72, 40, 0.1, False), (7, 8, 4, 64, 24, 0.2, False)])
def test_gradients_against_autograd(T, E, k, h, I, p, masked):
    from backward_token_expert_gb300.pipeline import SublayerStep

    aux, zc, eps = 0.5, 0.1, 1e-5
    d = _inputs(T, E, h, I, T)
    rng = np.random.default_rng(T)
    valid = (rng.random(T) < 0.8) if masked else np.ones(T, bool)
    if masked:
        d["x"][torch.from_numpy(~valid)] = float("nan")
        d["dout"][torch.from_numpy(~valid)] = float("nan")
    step = SublayerStep(T, E, k, h, I, Fraction(E), Fraction(1), aux, zc, max_norm=1e9, p=p, seed=99, eps=eps)
    try:
        dev = {n: t.cuda() for n, t in d.items()}
        v = torch.from_numpy(valid.astype(np.uint8)).cuda() if masked else None
        step.drop.step.fill_(5)
        _enqueue(step, dev, torch.empty(T, E, device="cuda"), v)
        torch.cuda.synchronize()
        assert step.device_status() == 0 and int(step.clip.nonfinite) == 0 and float(step.clip.coef) == 1.0
        ids = step.router.expert_idx.long().cpu()
        got = dict(dW=step.rec.buf.dW, dW1=step.rec.fc1.dW1, dWr=step.dWr, dgamma=step.norm.dgamma,
                   dbeta=step.norm.dbeta, dx=step.norm.dx, out=step.out)
        got = {n: t.double().cpu().numpy() for n, t in got.items()}
        norm = float(step.clip.norm)
    finally:
        step.close()
    kept = O.dropout_kept(T * h, p, 99, 5).reshape(T, h) / (1 - p)
    clean = {n: torch.nan_to_num(t) for n, t in d.items()}
    out, ref = _reference(clean, ids, kept, valid, k, aux, zc, eps)
    assert rel_fro(got["out"][valid], out[valid]) <= TOL["out"]
    if masked:
        assert np.all(got["dx"][~valid] == 0)
    for name, key in (("dW", "W"), ("dW1", "W1"), ("dWr", "Wr"), ("dgamma", "gamma"), ("dbeta", "beta"), ("dx", "x")):
        a, b = got[name], ref[key]
        if name == "dx":
            a, b = a[valid], b[valid]
        assert rel_fro(a, b) <= TOL[name], (name, rel_fro(a, b))
    want = np.sqrt(sum((got[n] ** 2).sum() for n in ("dW", "dW1", "dWr", "dgamma", "dbeta")))
    assert abs(norm - want) <= 1e-5 * want


def test_a_captured_step_draws_new_masks_and_matches_eager_steps():
    from backward_token_expert_gb300.pipeline import SublayerStep

    T, E, k, h, I = 300, 8, 2, 128, 64
    d = {n: t.cuda() for n, t in _inputs(T, E, h, I, 3).items()}
    step = SublayerStep(T, E, k, h, I, p=0.25, seed=4)
    try:
        logits = torch.empty(T, E, device="cuda")
        names = ("out", "dx", "dW", "dW1", "dWr", "dgamma")

        def results():
            torch.cuda.synchronize()
            return [t.clone() for t in (step.out, step.norm.dx, step.rec.buf.dW, step.rec.fc1.dW1, step.dWr,
                                        step.norm.dgamma)]

        eager = []
        for _ in range(2):
            _enqueue(step, d, logits)
            eager.append(results())
            step.drop.advance()
        assert not torch.equal(eager[0][0], eager[1][0])
        step.drop.step.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _enqueue(step, d, logits)
            step.drop.advance()
        for want in eager:
            graph.replay()
            for name, a, b in zip(names, results(), want):
                assert torch.equal(a, b), name
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step.drop.step.zero_()
            _enqueue(step, d, logits, stream=side)
        for name, a, b in zip(names, results(), eager[0]):
            assert torch.equal(a, b), name
        assert step.device_status() == 0
    finally:
        step.close()


def test_operators_alone_and_their_refusals():
    from backward_token_expert_gb300.pipeline import Dropout, ExpertFFN, LayerNorm

    T, E, k, h, I = 40, 4, 2, 64, 32
    bf = dict(dtype=torch.bfloat16, device="cuda")
    ffn, norm, drop = ExpertFFN(T, E, k, h, I, save=False, device="cuda"), LayerNorm(T, h), Dropout(0.5)
    x = torch.randn(T, h, **bf)
    W1, W = torch.randn(E, 2 * I, h, **bf), torch.randn(E, h, I, **bf)
    ids = torch.arange(T * k, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 20, 20, 60, 80], dtype=torch.int32, device="cuda")
    alpha = torch.rand(T, k, device="cuda")
    y = ffn.forward(x, W1, W, offsets, ids, alpha)
    assert ffn.ab is None and y.shape == (T, h) and torch.isfinite(y.float()).all()
    n = norm.forward(x, torch.ones(h, device="cuda"), torch.zeros(h, device="cuda"))
    assert torch.allclose(n.float().mean(1), torch.zeros(T, device="cuda"), atol=1e-2)
    out = drop.forward(x, torch.empty_like(x), x)
    drop.advance()
    assert int(drop.step) == 1 and not torch.equal(out, drop.forward(x, torch.empty_like(x), x))
    for part in (ffn, norm, drop):
        assert part.device_status() == 0
    odd = torch.randn(T * h + 1, **bf)[1:].view(T, h)
    g = torch.ones(h, device="cuda")
    for call in (lambda: ffn.forward(x.float(), W1, W, offsets, ids, alpha),
                 lambda: ffn.forward(x, W, W1, offsets, ids, alpha),
                 lambda: ffn.forward(x, W1, W, offsets[:3], ids, alpha),
                 lambda: ffn.forward(x, W1, W, offsets, ids.long(), alpha),
                 lambda: ffn.forward(x, W1, W, offsets, ids, alpha[:3]),
                 lambda: norm.forward(x[:3], g, g), lambda: norm.forward(x, g[:3], g), lambda: norm.forward(odd, g, g),
                 lambda: norm.forward(x, g, g, valid=g), lambda: norm.backward(x, x.float(), g),
                 lambda: LayerNorm(4, 8, torch.float16), lambda: LayerNorm(4, 8, eps=-1.0),
                 lambda: Dropout(1.5), lambda: Dropout(float("nan")), lambda: drop.forward(x, out[:3]),
                 lambda: drop.forward(x.cpu(), out), lambda: drop.forward(x.int(), out),
                 lambda: drop.forward(x, out, x.float())):
        with pytest.raises(ValueError):
            call()
    for part in (ffn, norm, drop):
        part.close()
