"""A few on-policy distillation steps on an output head: process, sample, ask the teacher, update.

    python examples/distill_step.py

Hidden states stand in for a model's last layer.  Each step penalises tokens that a
sequence has already, adds biases and a grammar mask, draws one token per sequence from what
is left, takes the teacher's best tokens at the same place, and moves the student's head
towards them: the divergence from the teacher's top tokens, with the log probability of the
token that the teacher finds best beside it.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from top_selection_stats_gb300 import (Sampler, distill_loss, distill_loss_grad, process_logits,  # noqa: E402
                                       token_logprobs)


class DistillLoss(torch.autograd.Function):
    """Divergence from a teacher's top tokens and log probabilities of `targets` as
    differentiable outputs."""

    @staticmethod
    def forward(ctx, logits, teacher_ids, teacher, targets, temperature, kind):
        out = distill_loss(logits, teacher_ids, teacher, kind=kind, targets=targets, temperature=temperature)
        ctx.save_for_backward(logits, teacher_ids, targets, temperature, out["slot_logprobs"], out["slot_grads"],
                              out["stats"], out["logprobs"])
        return out["loss"], out["logprobs"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, grad_logprobs):
        logits, ids, targets, temperature, slot_logprobs, slot_grads, stats, logprobs = ctx.saved_tensors
        grad = distill_loss_grad(logits, ids, slot_logprobs, slot_grads, stats, grad_loss.contiguous(), targets=targets,
                                 logprobs=logprobs, grad_logprobs=grad_logprobs.contiguous(), temperature=temperature)
        return grad, None, None, None, None, None


def run(sequences=256, vocab=32000, width=256, steps=3, n_top=20, kind="forward", seed=0, log=print):
    """Returns per step (mean divergence, mean log probability of the teacher's best token)."""
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev).manual_seed(seed)
    master = torch.randn(vocab, width, generator=g, device=dev) * (1.5 / width ** 0.5)
    taught = (master + torch.randn(vocab, width, generator=g, device=dev) * (1.0 / width ** 0.5)).bfloat16()
    temperature = torch.full((sequences,), 0.9, device=dev)
    top_k = torch.full((sequences,), 200, dtype=torch.int32, device=dev)
    top_p = torch.full((sequences,), 0.95, device=dev)
    key = torch.full((sequences,), seed, dtype=torch.int64, device=dev)
    offset = torch.arange(sequences, dtype=torch.int64, device=dev)
    # a prompt of 16 tokens, then what is drawn; half of the vocabulary is allowed
    history = torch.full((sequences, 16 + steps), -1, dtype=torch.int32, device=dev)
    history[:, :16] = torch.randint(0, vocab, (sequences, 16), generator=g, device=dev).int()
    prompts = torch.full((sequences,), 16, dtype=torch.int32, device=dev)
    full = lambda v: torch.full((sequences,), v, device=dev)  # noqa: E731
    bitmask = torch.full((sequences, (vocab + 31) // 32), 0x55555555, dtype=torch.int32, device=dev)
    bias_ids = torch.randint(0, vocab, (sequences, 4), generator=g, device=dev).int()
    bias = torch.tensor([2.0, -2.0, -100.0, -float("inf")], device=dev).expand(sequences, 4).contiguous()
    sampler = Sampler(0, max_batch=sequences, max_vocab=vocab)
    results = []
    for step in range(steps):
        hidden = torch.randn(sequences, width, generator=g, device=dev).bfloat16()
        weight = master.bfloat16().requires_grad_()
        logits = hidden @ weight.t()
        ready = process_logits(logits.detach(), history, lengths=prompts + step, prompt_lengths=prompts,
                               repetition=full(1.2), presence=full(0.3), frequency=full(0.2), bias_ids=bias_ids,
                               bias=bias, bitmask=bitmask, dtype=torch.float32)
        drawn = sampler.sample(ready["logits"], temperature, top_k, top_p, key, offset)
        offset += sequences
        history[:, 16 + step] = drawn["tokens"]

        best = token_logprobs(hidden @ taught.t(), drawn["tokens"], temperature=temperature, n_top=n_top)
        labels = best["top_ids"][:, 0].contiguous()
        loss, logprobs = DistillLoss.apply(logits, best["top_ids"], best["top_logprobs"], labels, temperature, kind)
        (loss.mean() - 0.1 * logprobs.mean()).backward()
        master -= 2.0 * weight.grad.float()
        results.append((loss.mean().item(), logprobs.mean().item()))
        log(f"step {step}: divergence {results[-1][0]:.4f}, the teacher's best token {results[-1][1]:.3f}, drawn tokens "
            f"under the teacher {best['logprobs'].mean().item():.3f}")
    sampler.close()
    return results


if __name__ == "__main__":
    run()
