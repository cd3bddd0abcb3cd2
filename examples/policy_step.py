"""A few policy-gradient steps on an output head: sample, score, update, score again.

    python examples/policy_step.py

Hidden states stand in for a model's last layer.  Each step draws one token per state
with the sampler, scores the drawn tokens under the raw distribution (log
probability, entropy, rank and the best alternatives), pushes the head towards
tokens that were rewarded, with an entropy bonus, and scores the same tokens
again straight from the hidden states, without their logits.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from top_selection_stats_gb300 import (Sampler, head_logprobs, token_logprobs,  # noqa: E402
                                       token_logprobs_grad)


class TokenLogprobs(torch.autograd.Function):
    """Log probabilities and entropies of `targets` as differentiable outputs."""

    @staticmethod
    def forward(ctx, logits, targets, temperature):
        out = token_logprobs(logits, targets, temperature=temperature)
        ctx.save_for_backward(logits, targets, temperature, out["stats"], out["entropy"])
        return out["logprobs"], out["entropy"]

    @staticmethod
    def backward(ctx, grad_logprobs, grad_entropy):
        logits, targets, temperature, stats, entropy = ctx.saved_tensors
        grad = token_logprobs_grad(logits, targets, stats, grad_logprobs.contiguous(), entropy=entropy,
                                   grad_entropy=grad_entropy.contiguous(), temperature=temperature)
        return grad, None, None


def run(states=512, vocab=32000, width=256, steps=4, seed=0, log=print):
    """Returns per step (mean reward, mean log probability of the rewarded tokens before and after)."""
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev).manual_seed(seed)
    hidden = torch.randn(states, width, generator=g, device=dev).bfloat16()
    master = torch.randn(vocab, width, generator=g, device=dev) * (1.5 / width ** 0.5)
    rewarded = torch.rand(vocab, generator=g, device=dev) < 0.1
    temperature = torch.full((states,), 0.9, device=dev)
    top_k = torch.full((states,), vocab, dtype=torch.int32, device=dev)
    top_p = torch.ones(states, device=dev)
    key = torch.full((states,), seed, dtype=torch.int64, device=dev)
    offset = torch.arange(states, dtype=torch.int64, device=dev)
    sampler = Sampler(0, max_batch=states, max_vocab=vocab)
    history = []
    for step in range(steps):
        weight = master.bfloat16().requires_grad_()
        logits = hidden @ weight.t()
        drawn = sampler.sample(logits.detach(), temperature, top_k, top_p, key, offset)
        offset += states
        tokens = drawn["tokens"]  # -1 where a row failed: it has no gradient
        gain = rewarded[tokens.clamp(min=0).long()].float() - 0.1

        report = token_logprobs(logits.detach(), tokens, temperature=temperature, n_top=5)
        logprobs, entropy = TokenLogprobs.apply(logits, tokens, temperature)
        loss = -(gain * logprobs).mean() - 1e-3 * entropy.mean()
        loss.backward()
        master -= 2.0 * weight.grad.float()

        after = head_logprobs(hidden, master.bfloat16(), tokens, temperature=temperature)
        hit = gain > 0
        history.append((gain.mean().item() + 0.1, logprobs[hit].mean().item(), after["logprobs"][hit].mean().item()))
        log(f"step {step}: reward {history[-1][0]:.3f}, entropy {entropy.mean().item():.2f}, median rank "
            f"{report['rank'].median().item()}, rewarded tokens' log probability {history[-1][1]:.3f} -> "
            f"{history[-1][2]:.3f}")
    sampler.close()
    return history


if __name__ == "__main__":
    run()
