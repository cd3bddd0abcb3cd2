"""Processing, sampling, the teacher's alternatives, the divergence and its gradient as they are
used together: the example runs, and its autograd function has the gradients that
torch.autograd finds in float64."""
import importlib.util
import os

import pytest
import torch

import top_selection_stats_gb300 as lib

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_step.py")


def example():
    spec = importlib.util.spec_from_file_location("distill_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kind", ["forward", "reverse"])
def test_example_runs(kind):
    lines = []
    results = example().run(steps=2, kind=kind, log=lines.append)
    assert len(lines) == len(results) == 2
    for loss, logprob in results:
        assert 0 < loss < 100 and logprob < 0


def divergence(x, ids, q, T, kind):
    """The definition in float64 torch operations."""
    logp = torch.log_softmax(x / T, 1)
    outside = torch.ones_like(x, dtype=torch.bool).scatter_(1, ids, False)
    log_s = torch.logsumexp(logp.masked_fill(~outside, -torch.inf), 1)
    a, r = logp.gather(1, ids), 1 - q.exp().sum(1)
    if kind == "reverse":
        return (a.exp() * (a - q)).sum(1) + log_s.exp() * (log_s - r.log()), logp
    return (q.exp() * (q - a)).sum(1) + r * (r.log() - log_s), logp


@pytest.mark.parametrize("kind", ["forward", "reverse"])
def test_teacher_to_student_with_autograd(kind):
    """A teacher's token_logprobs feeds the student's loss; the gradient is autograd's, to
    binary32's rounding: its terms, weighted by at most 2, to 1e-5."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, V = 9, 5000
    x = (torch.randn(B, V, generator=g, device="cuda") * 2).requires_grad_()
    y = x.detach() + torch.randn(B, V, generator=g, device="cuda")
    T = 0.7 + 0.6 * torch.rand(B, generator=g, device="cuda")
    best = lib.token_logprobs(y, torch.full((B,), -1, dtype=torch.int32, device="cuda"), temperature=T, n_top=20)
    labels = best["top_ids"][:, 3].contiguous()
    loss, lp = example().DistillLoss.apply(x, best["top_ids"], best["top_logprobs"], labels, T, kind)
    a, b = torch.rand(B, generator=g, device="cuda"), -torch.rand(B, generator=g, device="cuda")
    (a * loss + b * lp).sum().backward()
    z = x.detach().double().requires_grad_()
    want, logp = divergence(z, best["top_ids"].long(), best["top_logprobs"].double(), T.double()[:, None], kind)
    wlp = logp.gather(1, labels.long()[:, None])[:, 0]
    (a.double() * want + b.double() * wlp).sum().backward()
    assert torch.allclose(loss.double(), want, atol=1e-5) and torch.allclose(lp.double(), wlp, atol=1e-5)
    assert (x.grad.double() - z.grad).abs().max() < 2e-5


def test_processed_logits_are_what_is_sampled():
    """A banned or masked token is never drawn, greedy draws are the processed argmax, and the raw
    logits stay for scoring."""
    g = torch.Generator(device="cuda").manual_seed(4)
    B, V = 64, 32000
    x = torch.randn(B, V, generator=g, device="cuda").bfloat16()
    raw = x.clone()
    h = torch.randint(0, V, (B, 200), generator=g, device="cuda").int()
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, V // 32), generator=g, device="cuda").int()
    ban = raw.float().topk(3, 1).indices.int()
    y = lib.process_logits(x, h, repetition=torch.full((B,), 1.5, device="cuda"), bias_ids=ban,
                           bias=torch.full((B, 3), -float("inf"), device="cuda"), bitmask=bits, dtype=torch.float32)["logits"]
    s = lib.Sampler(0, max_batch=B, max_vocab=V)
    zero = torch.zeros(B, device="cuda")
    k, p = torch.full((B,), V, dtype=torch.int32, device="cuda"), torch.ones(B, device="cuda")
    i = torch.arange(B, device="cuda")
    out = s.sample(y, zero, k, p, i, i)
    assert torch.equal(out["tokens"].long(), y.argmax(1)) and torch.equal(x, raw)
    out = s.sample(y, p, k, p, i, i)
    t = out["tokens"].long()
    assert not (out["status"] != 0).any() and not (t[:, None] == ban).any()
    assert ((bits[i, t // 32] >> (t % 32)) & 1).all()
    s.close()
