"""The gradient at every valid temperature and any finite incoming gradients: no NaN, no bits lost,
infinities only where the result is past the type.

The reference is the formula in float64 on the forward call's own outputs.  Beside the output's
rounding, a token outside the slots has the error of 2^x: u times a few units, twice the
exponent's rounding (|z| and |L|, each rounded up to four times, and the factor's power, up to 250,
in two sums) and the factor's (4), and where its share of the mass times 2^24 is below the least
normal number, it is 0; a slot and a
target that of p, an exponential of a binary32 logarithm which counts as given, good to two units
of a binary32 number, 2^-149 each where p is below the normal ones; as the parts of the two incoming
gradients are added at the scale of the larger one, each of them and their products are multiples
of 2^-149 of it.  Where a result is within its error of the type's end, either side is right."""
import numpy as np
import pytest
import torch

import test_gpu_distill as G
import top_selection_stats_gb300 as lib

pytestmark = pytest.mark.gpu

U = G.U


def check(c, dtype, g, gl, in_place=False):
    B, V = c["x"].shape[0], c["V"]
    f = G.run(c)
    x, legal, ids, _, t, T = G.host(c)
    gt, glt = (torch.from_numpy(v.astype(np.float32)).cuda() for v in (g, gl))
    d = lib.distill_loss_grad(c["x"], c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"], gt, targets=c["targets"],
                              logprobs=f["logprobs"], grad_logprobs=glt, temperature=c["temperature"], bitmask=c["bitmask"], V=V,
                              out=c["x"] if in_place else None)
    d = d[:, :V].double().cpu().numpy()
    assert not np.isnan(d).any()
    h = {k: f[k].double().cpu().numpy() for k in ("slot_logprobs", "slot_grads", "stats", "logprobs", "status")}
    g, gl = gt.double().cpu().numpy(), glt.double().cpu().numpy()
    most = float(torch.finfo(G.DT[dtype]).max)
    for r in range(B):
        if h["status"][r]:
            assert not d[r].any(), r
            continue
        m, L, A, s = h["stats"][r]
        ok = legal[r] & (x[r] > -np.inf)
        assert not d[r][~ok].any(), r
        hard = gl[r] if t[r] >= 0 and h["logprobs"][r] > -np.inf else 0.0
        out, used = ok.copy(), ids[r] >= 0
        at = ids[r][used]
        out[at] = False
        want, tol = np.zeros(V), np.zeros(V)
        if out.any():
            z = (x[r][out] - m) / T[r]
            with np.errstate(under="ignore"):
                rho = np.exp(z - L)
            factor = abs(g[r] * A - hard * s) / T[r]
            power = min(250.0, abs(np.log2(factor))) if factor > 0 else 0.0
            rel = U * (64 + 8 * np.where(rho > 0, np.abs(z), 0) + 8 * abs(L) + 2 * power)
            want[out] = rho * ((g[r] * A - hard * s) / T[r])
            tol[out] = (rho * rel + 2.0 ** -149) * ((abs(g[r] * A) + abs(hard * s)) / T[r])
            if hard and out[t[r]]:
                k = t[r]
                share, p = rho[np.cumsum(out)[k] - 1], np.exp(h["logprobs"][r])
                want[k] = (g[r] * A * share - hard * np.expm1(h["logprobs"][r])) / T[r]
                tol[k] = (abs(g[r] * A) * share * rel.max() + abs(hard) * (p * rel[np.cumsum(out)[k] - 1] + 8 * U)) / T[r]
        hit = at == t[r]
        lp = h["slot_logprobs"][r][used]
        want[at] = (g[r] * h["slot_grads"][r][used] + hard * np.where(hit, -np.expm1(lp), -np.exp(lp))) / T[r]
        tol[at] = 16 * U * (np.abs(g[r] * h["slot_grads"][r][used]) + abs(hard) * (hit + np.exp(lp))) / T[r]
        least = 8 * 2.0 ** -149 * max(abs(g[r]), abs(hard)) / T[r]
        tol[at] += least
        if hard and out[t[r]]:
            tol[t[r]] += least
        tol = tol + np.abs(want) * (G.OUT_EPS[dtype] + 4 * U) + 2 * G.OUT_TINY[dtype]
        past = np.abs(want) - tol > most
        inside = np.abs(want) + tol < most
        assert np.array_equal(d[r][past], np.sign(want[past]) * np.inf), r
        off = np.abs(d[r][inside] - want[inside])
        bad = off > tol[inside]
        assert not bad.any(), (r, T[r], g[r], gl[r], d[r][inside][bad][:3], want[inside][bad][:3], tol[inside][bad][:3])


def sizes(rng, B, decades):
    v = np.sign(rng.standard_normal(B)) * 10.0 ** rng.uniform(-decades, min(decades, 38), B)
    v[rng.random(B) < 0.15] = 0.0
    return v


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", G.KINDS)
@pytest.mark.parametrize("V,K,shift,masked", [(1, 2, 0, False), (4, 2, 1, False), (60, 5, 0, True), (900, 40, 3, False), (7941, 11, 0, True)])
def test_any_temperature_and_gradients(V, K, shift, masked, kind, dtype):
    for seed, (cold, size) in enumerate(((1, 1), (6, 10), (30, 10), (30, 38), (6, 38), (44, 38))):
        rng = np.random.default_rng(seed + V)
        temps = 10.0 ** rng.uniform(-cold, min(cold, 38), 24)
        c = G.make(24, V, K, dtype, seed + V, kind, temps=temps, shift=shift, pad=1, masked=masked)
        check(c, dtype, sizes(rng, 24, size), sizes(rng, 24, size), in_place=seed % 2 == 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_targets_outside_the_slots(dtype):
    """The one token outside that has any mass, with a probability next to 1 and next to 0: its two
    parts cancel, at any size."""
    B, V = 24, 300
    rng = np.random.default_rng(5)
    for kind in G.KINDS:
        c = G.make(B, V, 4, dtype, 6, kind, temps=10.0 ** rng.uniform(-30, 1, B), unused=0.0)
        taken = c["ids"].cpu().numpy()
        t = np.array([min(set(range(V)) - set(taken[r])) for r in range(B)], np.int32)
        t[::3] = [max(set(range(V)) - set(taken[r])) for r in range(0, B, 3)]
        c["targets"] = torch.from_numpy(t).cuda()
        c["x"][torch.arange(B, device="cuda"), c["targets"].long()] = 40.0
        c["x"][1::2][torch.arange(B // 2, device="cuda"), c["ids"][1::2, 0].long()] = 41.0
        check(c, dtype, sizes(rng, B, 3), sizes(rng, B, 38))
