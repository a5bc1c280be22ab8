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
