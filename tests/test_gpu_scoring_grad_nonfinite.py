"""Incoming gradients of smp_token_logprobs_grad that are infinite or NaN (an overflowed loss scale):
tokens that are not legal have gradient 0 all the same, and no other row is touched."""
import numpy as np
import pytest
import torch

import top_selection_stats_gb300 as lib
from oracle import scoring as S
from top_selection_stats_gb300 import workloads

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
PAIRS = [(INF, 0.0), (-INF, 0.0), (NAN, 0.0), (0.0, INF), (1.0, -INF), (1.0, NAN), (INF, INF), (NAN, 1.0), (INF, 1.0), (0.5, 0.25)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("V,shift", [(50, 0), (300, 1), (20003, 3)])
def test_no_gradient_where_nothing_is_legal(V, shift, entropy, dtype):
    B = len(PAIRS)
    case = workloads.random_case(V, B, V, dtype=dtype, mask_frac=0.6, neg_inf_frac=0.2)
    buf = torch.zeros(shift + B * V, dtype=workloads.TORCH_DTYPE[dtype], device="cuda")
    x = buf[shift:].view(B, V)
    x.copy_(case["logits"])
    legal = torch.from_numpy(S.unpack(case["bitmask"].numpy().view(np.uint32), V)).cuda() & (x > -INF)
    t = torch.arange(B, device="cuda").int() * (V // B)
    more = dict(bitmask=case["bitmask"].cuda())
    f = lib.token_logprobs(x, t, **more)
    g, ge = (torch.tensor([p[i] for p in PAIRS], device="cuda") for i in (0, 1))
    if entropy:
        more.update(entropy=f["entropy"])
    else:
        ge = torch.zeros_like(ge)

    def grad(a, b, y=x, **kw):
        return lib.token_logprobs_grad(y, t, f["stats"], a, grad_entropy=b if entropy else None, **more, **kw)

    d = grad(g, ge)
    assert not d[~legal].any()
    counts = ~torch.isfinite(ge) | (~torch.isfinite(g) & (f["logprobs"] > -INF))
    want = grad(torch.where(counts | ~torch.isfinite(g), 0.0, g), torch.where(counts, 0.0, ge))
    assert torch.equal(d[~counts], want[~counts])
    # nothing that counts is lost: NaN, infinities or the type's largest values where the row is not finite
    live = counts & (f["status"] == 0)
    got = d[live].float()
    assert (torch.isnan(got) | (got.abs() > 6e4))[legal[live]].any()
    y = x.clone()
    at = grad(g, ge, y=y, out=y)
    assert np.array_equal(at.double().cpu().numpy(), d.double().cpu().numpy(), equal_nan=True)
