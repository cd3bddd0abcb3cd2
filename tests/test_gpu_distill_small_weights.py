"""Probabilities below binary32's least normal number in a reverse loss, where a teacher's lowest
finite log probabilities weigh them up.

A weight p below 2^-126 is a multiple of 2^-149; an exponential of two units, a quotient and a
product leave it within 4 of them, so that a term p u is off by 4 2^-149 |u| beside the bounds
of test_gpu_distill.  Those count |u| only where q is above 0 in binary64; a reverse loss has the
teacher's logarithm, not q, so the same terms are added for slots whose q is 0 there."""
import numpy as np
import pytest
import torch

import test_gpu_distill as G

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -149


@pytest.mark.parametrize("K", [5, 40, 100])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lowest_teacher_values(dtype, K):
    """Student probabilities of 1e-37 to 1e-42 on a token that the teacher's mask has at the type's
    lowest value: up to tens of units of loss."""
    depths = [85.0, 87.0, 87.5, 88.0, 89.0, 91.0, 93.0, 96.0]
    c = G.make(len(depths), 3000, K, dtype, K, "reverse", temps=[1.0], unused=0.0)
    low = float(np.finfo(np.float32).min)
    for r, depth in enumerate(depths):
        c["x"][r, c["ids"][r, K // 2].long()] = 30.0
        c["x"][r, c["ids"][r, 0].long()] = 30.0 - depth
        c["teacher"][r, 0] = low
    for shift in (0, 1, K // 2, K - 1):
        d = dict(c, ids=c["ids"].roll(shift, 1).contiguous(), teacher=c["teacher"].roll(shift, 1).contiguous())
        got = {k: v.double().cpu().numpy() for k, v in G.run(d).items()}
        for r, o in enumerate(G.reference(d)):
            e = G.errors(o, 3000, 1.0, "reverse")
            assert got["status"][r] == 0
            none = (o["q"] == 0) & (o["lq"] > -np.inf)
            u = np.abs(np.where(none, o["u"], 0.0))
            terms = o["p"] * u * (e["slot_logprobs"] + 40 * G.U)  # errors of p u
            loss = e["loss"] + terms.sum() + 4 * UNIT * abs(low)
            G.close(got["loss"][r], o["loss"], loss, (r, "loss"))
            G.close(got["slot_grads"][r], o["slot_grads"], e["slot_grads"] + terms + 4 * UNIT * u + o["p"] * loss, (r, "grads"))
            G.close(got["stats"][r, 2], o["stats"][2], e["A"] + o["stats"][3] * loss, (r, "A"))
