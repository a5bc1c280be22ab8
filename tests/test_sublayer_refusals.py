"""What a sublayer's training step refuses, before it calls the library: checked
with host tensors and a library that must not be reached."""

from types import SimpleNamespace

import pytest
import torch

T, E, k, h, I = 12, 8, 2, 64, 32


@pytest.fixture
def step(monkeypatch):
    from backward_token_expert_gb300 import lrm as L
    from backward_token_expert_gb300.pipeline import SublayerStep

    def reached():
        raise AssertionError("the library was called")

    monkeypatch.setattr(L, "load_library", reached)
    s = SublayerStep.__new__(SublayerStep)
    s.rec = SimpleNamespace(T=T, E=E, k=k, h=h, I=I, N=T * k, buf=None, fc1=None, max_rows=T * k, ctx=None)
    s.dWr = torch.zeros(E, h)
    s._routed = True
    return s


def _arguments():
    bf = dict(dtype=torch.bfloat16)
    return dict(dout=torch.zeros(T, h, **bf), x=torch.zeros(T, h, **bf), W=torch.zeros(E, h, I, **bf),
                W1=torch.zeros(E, 2 * I, h, **bf), Wr=torch.zeros(E, h, **bf), gamma=torch.ones(h))


def _swapped(a):
    a["W"], a["W1"] = a["W1"], a["W"]


@pytest.mark.parametrize("change", [
    _swapped,
    lambda a: a.update(W=a["W"][:, :, : I // 2].contiguous()),
    lambda a: a.update(W=a["W"][: E - 1]),
    lambda a: a.update(W=a["W"].float()),
    lambda a: a.update(W=a["W"].transpose(1, 2)),
    lambda a: a.update(W1=a["W1"][:, :I].contiguous()),
    lambda a: a.update(W1=a["W1"].transpose(1, 2).contiguous().transpose(1, 2)),
    lambda a: a.update(Wr=a["Wr"][: E - 1]),
    lambda a: a.update(Wr=a["Wr"].T),
    lambda a: a.update(Wr=a["Wr"].float()),
    lambda a: a.update(dout=a["dout"][1:]),
    lambda a: a.update(dout=a["dout"].float()),
    lambda a: a.update(x=a["x"][:, : h // 2]),
    lambda a: a.update(gamma=a["gamma"][1:]),
    lambda a: a.update(gamma=a["gamma"].bfloat16()),
    lambda a: a.update(W=a["W"].to("meta"))])
def test_the_backward_refuses_what_does_not_fit_its_layer(step, change):
    a = _arguments()
    change(a)
    with pytest.raises(ValueError):
        step.backward(**a)
