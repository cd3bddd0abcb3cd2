"""smp_token_logprobs_grad at every temperature that the forward call accepts, and for
gradients of any size: what passes the type's range is an infinity at legal tokens only,
and a token that is not legal, or has no probability, gets exactly 0.

The gradient before its last rounding lies within `err` of the formula's (the bound of
test_gpu_scoring.check_grad: the weight's relative error and L's absolute one), plus what
flushing 2^d below 2^-150 leaves out.  Rounding is monotone, so the result lies between the
roundings of both ends, infinities included."""
import numpy as np
import pytest
import torch

import test_gpu_scoring as T
import top_selection_stats_gb300 as lib
from oracle import scoring as S

pytestmark = pytest.mark.gpu

U = T.U
TEMPS = [1e-30, 1e-3, 0.05, 1.0, 20.0, 1e4, 1e30, 1e-42, 1e-38, 3e38]


def check(c, dtype, entropy, size, in_place):
    B, V = c["x"].shape[0], c["V"]
    f = T.run(c)
    rng = np.random.Generator(np.random.PCG64(B * 7 + V))
    g = torch.from_numpy((size * rng.standard_normal(B)).astype(np.float32)).cuda()
    gh = torch.from_numpy((size * rng.standard_normal(B)).astype(np.float32)).cuda() if entropy else None
    ref = T.reference(c)
    d = lib.token_logprobs_grad(c["x"], c["targets"], f["stats"], grad_logprobs=g,
                                entropy=f["entropy"] if entropy else None, grad_entropy=gh,
                                temperature=c["temperature"], bitmask=c["bitmask"], V=V,
                                out=c["x"] if in_place else None)
    torch.cuda.synchronize()
    d = d[:, :V].float().cpu()
    t = c["targets"].cpu().numpy()
    temps = c["temperature"].double().cpu().numpy()
    g = g.double().cpu().numpy()
    gh = np.zeros(B) if gh is None else gh.double().cpu().numpy()
    for r, o in enumerate(ref):
        want = S.grad_row(o, int(t[r]), temps[r], g[r], gh[r])
        if want is None:
            assert not d[r].any(), r
            continue
        lp = o["log_p"]
        legal = lp != -np.inf
        assert not d[r][torch.from_numpy(~legal)].any(), (r, temps[r])
        p, al = np.exp(lp), np.where(legal, np.abs(lp), 0.0)
        base = T.forward_tolerance(o, V, 0.0)
        zbar = max(o["entropy"] - o["stats"][1], 0.0)
        weight = np.where(p > 0, p * (abs(g[r]) + abs(gh[r]) * (al + o["entropy"] + 1)), 0.0) / temps[r]
        err = weight * (base * (2 + zbar) + 8 * U * (1 + np.where(p > 0, al, 0.0) + zbar))
        err += 4 * U * np.abs(want)
        err += 2.0 ** -150 * (abs(g[r]) + abs(gh[r]) * (200 + o["entropy"])) / temps[r]
        if t[r] >= 0 and legal[t[r]]:
            err[t[r]] += 4 * U * abs(g[r]) / temps[r]
        low, high = (torch.from_numpy(want + s * err).to(T.DT[dtype]).float() for s in (-1, 1))
        ok = (d[r] >= low) & (d[r] <= high)
        j = int((~ok).nonzero()[0]) if not ok.all() else -1
        assert ok.all(), (r, temps[r], j, float(d[r][j]), want[j], err[j])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("grid", [None, 2])
def test_all_valid_temperatures(grid, entropy, dtype):
    """grid: few distinct logits, so that several tokens share the top at any temperature."""
    for in_place in (False, True):
        c = T.make(20, 3001, dtype, 3, pad=7, masked=True, temps=TEMPS, grid=grid, neg_inf=0.05)
        check(c, dtype, entropy, 1.0, in_place)


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("size", [1e-42, 1e-36, 1e-30, 1e30, 1e37])
def test_sizes_of_the_incoming_gradient(size, entropy):
    check(T.make(20, 1003, "f32", 4, masked=True, temps=[1.0, 0.01, 0.7, 100.0, 1.5], neg_inf=0.05), "f32",
          entropy, size, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_results_aligned_unlike_their_logits(dtype):
    check(T.make(20, 3001, dtype, 6, shift=1, masked=True, temps=TEMPS, grid=2, neg_inf=0.05), dtype, True, 1.0, False)


def test_far_rows_beside_others():
    """A row out of range leaves its neighbours' bits alone."""
    c = T.make(6, 5003, "bf16", 5, temps=[1.0])
    g = torch.randn(6, device="cuda")
    f = T.run(c)
    a = lib.token_logprobs_grad(c["x"], c["targets"], f["stats"], g, temperature=c["temperature"])
    c["temperature"][::2] = 1e-41
    f = T.run(c)
    b = lib.token_logprobs_grad(c["x"], c["targets"], f["stats"], g, temperature=c["temperature"])
    torch.cuda.synchronize()
    assert torch.equal(a[1::2], b[1::2]) and not b.isnan().any()
