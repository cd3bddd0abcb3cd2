"""Incoming gradients at binary32's largest values, each finite but not their sum: results are the
formula's, infinite only where they are past the type."""
import numpy as np
import pytest
import torch

import test_gpu_distill as G
import top_selection_stats_gb300 as lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", G.KINDS)
def test_sum_past_binary32(kind):
    """From the forward call's outputs in float64: products and a sum of two terms, 200 units of the
    larger one (they cancel where the two gradients are the same)."""
    B, V, K = 6, 900, 9
    c = G.make(B, V, K, "f32", 4, kind, temps=[1.0, 4.0])
    c["targets"] = c["ids"].amax(1)
    f = G.run(c)
    pairs = [(3e38, 3e38), (3e38, -3e38), (-2e38, 2.5e38), (1e38, 3.4e38), (-3e38, -3e38), (3.4e38, 1.0)]
    g, gl = (torch.tensor([p[i] for p in pairs], device="cuda") for i in (0, 1))
    d = lib.distill_loss_grad(c["x"], c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"], g, targets=c["targets"],
                              logprobs=f["logprobs"], grad_logprobs=gl, temperature=c["temperature"], V=V)
    d = d[:, :V].double().cpu().numpy()
    x, _, ids, _, t, T = G.host(c)
    h = {k: f[k].double().cpu().numpy() for k in ("slot_logprobs", "slot_grads", "stats")}
    g, gl = g.double().cpu().numpy(), gl.double().cpu().numpy()
    assert not np.isnan(d).any()
    for r in range(B):
        m, L, A, s = h["stats"][r]
        rho = np.exp((x[r] - m) / T[r] - L)
        want, size = rho * (g[r] * A - gl[r] * s) / T[r], rho * (abs(g[r] * A) + abs(gl[r] * s)) / T[r]
        used = ids[r] >= 0
        at, p = ids[r][used], np.exp(h["slot_logprobs"][r][used])
        hit = (at == t[r]).astype(float)
        want[at] = (g[r] * h["slot_grads"][r][used] + gl[r] * (hit - p)) / T[r]
        size[at] = (np.abs(g[r] * h["slot_grads"][r][used]) + np.abs(gl[r]) * (hit + p)) / T[r]
        with np.errstate(over="ignore"):
            past = np.abs(want) + 200 * G.U * size > np.finfo(np.float32).max
        assert np.all(np.abs(d[r] - want)[~past] <= 200 * G.U * size[~past] + 2.0 ** -126), r
        assert np.all(np.abs(d[r][past]) > 3e38)
