"""The examples' autograd functions have first derivatives only: asked for a second one, they say so
instead of giving one that leaves their own part out.  Runs without a GPU, on stand-ins of the calls."""
import importlib.util
import os

import pytest
import torch

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(EXAMPLES, name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def distill(monkeypatch):
    m = load("distill_step")
    monkeypatch.setattr(m, "distill_loss", lambda x, ids, q, **k: dict(
        loss=(x * x).sum(1), logprobs=x.sum(1), slot_logprobs=q, slot_grads=q, stats=q[:, :1]))
    monkeypatch.setattr(m, "distill_loss_grad", lambda x, *a, **k: 2 * x * a[4][:, None] + k["grad_logprobs"][:, None])
    ids, q, t = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), torch.zeros(2, dtype=torch.int32)
    return lambda x: m.DistillLoss.apply(x, ids, q, t, torch.ones(2), "forward")


def policy(monkeypatch):
    m = load("policy_step")
    monkeypatch.setattr(m, "token_logprobs", lambda x, t, **k: dict(logprobs=x.sum(1), entropy=(x * x).sum(1), stats=x[:, :2]))
    monkeypatch.setattr(m, "token_logprobs_grad", lambda x, t, stats, g, **k: g[:, None] + 2 * x * k["grad_entropy"][:, None])
    return lambda x: m.TokenLogprobs.apply(x, torch.zeros(2, dtype=torch.int32), torch.ones(2))


@pytest.mark.parametrize("make", [distill, policy])
def test_second_derivatives_are_refused(make, monkeypatch):
    call = make(monkeypatch)
    x = torch.arange(6.0).reshape(2, 3).requires_grad_()
    a, b = call(x)
    (a.sum() + b.sum()).backward()  # the first one is there
    assert torch.equal(x.grad, 2 * x.detach() + 1)
    a, b = call(x)
    d, = torch.autograd.grad((a * a).sum() + b.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        d.sum().backward()
