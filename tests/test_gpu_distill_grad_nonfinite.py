"""Incoming gradients that are infinite or NaN (an overflowed loss scale): tokens that are not legal
have gradient 0 all the same, and no other row is touched."""
import numpy as np
import pytest
import torch

import test_gpu_distill as G
import top_selection_stats_gb300 as lib

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
PAIRS = [(INF, 0.0), (-INF, 0.0), (NAN, 0.0), (0.0, INF), (1.0, -INF), (1.0, NAN), (INF, INF), (NAN, 1.0), (INF, 1.0), (0.5, 0.25)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", G.KINDS)
@pytest.mark.parametrize("V,K,shift", [(50, 50, 0), (300, 9, 1), (20003, 40, 3)])
def test_no_gradient_where_nothing_is_legal(V, K, shift, kind, dtype):
    B = len(PAIRS)
    c = G.make(B, V, K, dtype, V, kind, masked=True, neg_inf=0.2, shift=shift, pad=1)
    c["ids"][:, 0] = -1
    t = c["ids"][:, 1:].amax(1)
    legal = torch.from_numpy(G.host(c)[1]).cuda() & (c["x"][:, :V] > -INF)
    t = torch.where(t >= 0, t, 0)  # a token of the teacher's, or one that may not be legal
    c["targets"] = t.int()
    f = G.run(c)
    g, gl = (torch.tensor([p[i] for p in PAIRS], device="cuda") for i in (0, 1))
    a = (c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"])
    more = dict(targets=c["targets"], logprobs=f["logprobs"], temperature=c["temperature"], bitmask=c["bitmask"], V=V)
    d = lib.distill_loss_grad(c["x"], *a, grad_loss=g, grad_logprobs=gl, **more)
    assert not d[:, :V][~legal].any()
    counts = ~torch.isfinite(g) | (~torch.isfinite(gl) & (f["logprobs"] > -INF))
    # where the incoming gradient is not finite, nothing of a row that has one looks finite
    live = counts & (f["status"] == 0) & torch.isfinite(f["loss"])
    outside = legal.clone()
    rows = torch.arange(B, device="cuda")[:, None].expand_as(c["ids"])
    outside[rows[c["ids"] >= 0], c["ids"][c["ids"] >= 0].long()] = False
    assert not torch.isfinite(d[:, :V][outside & live[:, None]]).any()
    # other rows are what they are without these
    g0, gl0 = torch.where(counts, 0.0, g), torch.where(counts, 0.0, gl)
    gl0 = torch.where(torch.isfinite(gl0), gl0, 0.0)
    want = lib.distill_loss_grad(c["x"], *a, grad_loss=g0, grad_logprobs=gl0, **more)
    assert torch.equal(d[~counts], want[~counts])
    # in place, where a row's logits are read before they are written
    x = c["x"].clone()
    at = lib.distill_loss_grad(x, *a, grad_loss=g, grad_logprobs=gl, out=x, **more)
    assert np.array_equal(at[:, :V].double().cpu().numpy(), d[:, :V].double().cpu().numpy(), equal_nan=True)
