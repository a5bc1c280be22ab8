"""How a program may call a sublayer's training step: what it refuses, and leaves
as it was."""

import pytest
import torch

from gpu_common import built_library, need_gpu
from test_gpu_sublayer_step import _enqueue, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    built_library()


def _results(step):
    torch.cuda.synchronize()
    return {n: t.clone() for n, t in dict(out=step.out, dx=step.norm.dx, dW=step.rec.buf.dW, dW1=step.rec.fc1.dW1,
                                          dWr=step.dWr, dgamma=step.norm.dgamma, dbeta=step.norm.dbeta).items()}


def _same(a, b):
    return [n for n in a if not torch.equal(a[n], b[n])] == []


def test_a_refused_backward_leaves_the_step_as_it_was():
    from backward_token_expert_gb300.pipeline import SublayerStep

    T, E, k, h, I = 40, 8, 2, 64, 32
    d = {n: t.cuda() for n, t in _inputs(T, E, h, I, 1).items()}
    step = SublayerStep(T, E, k, h, I)
    try:
        _enqueue(step, d, torch.empty(T, E, device="cuda"))
        want = _results(step)
        args = [d[n] for n in ("dout", "x", "W", "W1", "Wr", "gamma")]
        for i, bad in ((2, d["W1"]), (3, d["W"]), (4, d["Wr"].cpu()), (0, d["dout"][:-1]), (5, d["gamma"].half())):
            with pytest.raises(ValueError):
                step.backward(*args[:i], bad, *args[i + 1:])
        assert _same(_results(step), want)
        step.backward(*args)
        assert _same(_results(step), want) and step.device_status() == 0
    finally:
        step.close()


@pytest.mark.parametrize("kind", ["TrainingStep", "SublayerStep"])
def test_memory_of_a_dropped_step_stays_until_its_stream_is_done(kind):
    # the allocator learns of another stream that works on a step's buffers: none of them is given away meanwhile
    from backward_token_expert_gb300 import pipeline as P

    T, E, k, h, I = 50, 8, 2, 64, 32
    d = {n: t.cuda() for n, t in _inputs(T, E, h, I, 5).items()}
    logits = torch.randn(T, E, device="cuda")
    phi, ab = torch.randn(T * k, I, device="cuda").bfloat16(), torch.randn(T * k, 2 * I, device="cuda").bfloat16()
    step = getattr(P, kind)(T, E, k, h, I)
    rec = step.rec  # kept: its context goes with it, which waits for the GPU
    held = [*vars(rec.buf).values(), *vars(rec.fc1).values(), rec.dgate, step.dWr, step.dxr, step._segment]
    if kind == "SublayerStep":
        held += [step.out, step._g, step._dn, step._side, step._ws]
    own = {t.data_ptr(): t.numel() * t.element_size() for t in held}
    assert len(own) == len(held)

    def run(stream):
        if kind == "SublayerStep":
            step.normalize(d["x"], d["gamma"], d["beta"], stream=stream)
            step.route(logits, stream=stream)
            step.experts(d["x"], d["W1"], d["W"], stream)
            step.backward(d["dout"], d["x"], d["W"], d["W1"], d["Wr"], d["gamma"], stream)
        else:
            step.route(logits, stream=stream)
            step.backward(logits, d["dout"], phi, d["W"], d["x"], ab, d["W1"], d["Wr"], stream)

    run(None)  # the kernels' first launches, which wait for the GPU
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(1_000_000_000)
    run(s)
    rec.buf = rec.fc1 = rec.dgate = held = None
    del step, run
    others = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in own.values() for _ in range(24)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in others]
    assert not s.query()  # still asleep, the step behind it
    assert not [at for at in own if any(a <= at < b for a, b in spans)]
    s.synchronize()
    assert rec.device_status() == 0


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("how", ["current", "stream", "raw", "default"])
def test_two_layers_forward_then_backward_with_buffers_in_common(masked, how):
    # a model's layers run forward one after the other through one buffer of logits and one mask, which hold the next
    # layer's, or the next batch's, by the time of the backward
    from backward_token_expert_gb300.pipeline import SublayerStep

    T, E, k, h, I = 120, 8, 2, 64, 32
    d = [{n: t.cuda() for n, t in _inputs(T, E, h, I, seed).items()} for seed in (6, 7)]
    masks = [(torch.arange(T, device="cuda") % m != 0).to(torch.uint8) for m in (3, 5)] if masked else [None, None]
    steps = [SublayerStep(T, E, k, h, I, p=0.2, seed=seed) for seed in (1, 2)]
    try:
        want = []
        for step, v, m in zip(steps, d, masks):
            _enqueue(step, v, torch.empty(T, E, device="cuda"), m)
            want.append(_results(step))
        side = torch.cuda.Stream()
        stream = dict(current=None, stream=side, raw=side.cuda_stream, default=0)[how]
        logits, mask = torch.empty(T, E, device="cuda"), torch.empty(T, dtype=torch.uint8, device="cuda")
        mask = mask if masked else None
        torch.cuda.synchronize()
        with torch.cuda.stream(side if how in ("stream", "raw") else torch.cuda.default_stream()):
            for step, v, m in zip(steps, d, masks):
                if masked:
                    mask.copy_(m)
                n = step.normalize(v["x"], v["gamma"], v["beta"], mask, stream)
                torch.matmul(n.float(), v["Wr"].float().T, out=logits)
                step.route(logits, mask, stream)
                step.experts(v["x"], v["W1"], v["W"], stream)
            logits.fill_(float("nan"))
            if masked:
                mask.fill_(0)
            for step, v in zip(steps[::-1], d[::-1]):
                step.backward(v["dout"], v["x"], v["W"], v["W1"], v["Wr"], v["gamma"], stream)
        for step, w in zip(steps, want):
            assert _same(_results(step), w) and step.device_status() == 0
    finally:
        for step in steps:
            step.close()


def test_a_backward_of_nothing_is_refused():
    from backward_token_expert_gb300.pipeline import SublayerStep

    T, E, k, h, I = 16, 8, 2, 64, 32
    d = {n: t.cuda() for n, t in _inputs(T, E, h, I, 8).items()}
    step = SublayerStep(T, E, k, h, I)
    try:
        with pytest.raises(ValueError):
            step.backward(d["dout"], d["x"], d["W"], d["W1"], d["Wr"], d["gamma"])
    finally:
        step.close()


def test_a_masked_batch_makes_no_buffer_and_waits_for_nothing():
    # every buffer is there from the start: a masked route in the middle of a step's launches does not stop the host
    from backward_token_expert_gb300.pipeline import SublayerStep

    T, E, k, h, I = 64, 8, 2, 64, 32
    d = {n: t.cuda() for n, t in _inputs(T, E, h, I, 9).items()}
    valid = (torch.arange(T, device="cuda") % 4 != 0).to(torch.uint8)
    step, other, logits = SublayerStep(T, E, k, h, I), SublayerStep(T, E, k, h, I), torch.randn(T, E, device="cuda")
    try:
        for s, v in ((other, valid), (step, None)):  # the kernels' first launches wait for the GPU
            s.normalize(d["x"], d["gamma"], d["beta"], v)
            s.route(logits, v)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda._sleep(500_000_000)
        step.normalize(d["x"], d["gamma"], d["beta"], valid)
        step.route(logits, valid)
        assert not torch.cuda.current_stream().query()  # still asleep
        assert torch.cuda.memory_allocated() == before
        torch.cuda.synchronize()
        assert step.device_status() == 0 and int(step.router.tokens) == int(valid.sum())
    finally:
        step.close()
        other.close()
