"""smp_distill_loss and its gradient where logits over the temperature are large: products x / T
of 1e3 to 1e31 that binary32 does not hold exactly, in every launch shape, and references of
running sums on both sides of the border between the two ways they are kept.

Cases are test_gpu_distill's, and its bounds, with one term that they leave out: a forward loss has
r (log r - log s) also where s is 0 in binary64 (log s = -1e3 to -1e31).  Its error is that of
the term where s is above 0: r times (40u |log r - log s|, that of log s, 8u (1 + |log r| + |log s|))."""
import numpy as np
import pytest
import torch

import test_gpu_distill as G
from test_gpu_distill_launches import repeated

pytestmark = pytest.mark.gpu

U = G.U
BOUNDS = G.errors


def errors(o, V, T, kind):
    e = BOUNDS(o, V, T, kind)
    if kind == "forward" and o["outside"].any() and o["stats"][3] == 0:
        log_s, L, Lr = abs(o["log_s"]), o["L"], abs(o["stats"][1])
        es = U * (4 * o["zbar"] + 4 * L + 4 * o["zbar_r"] + 4 * Lr + V / 128 + 168) + 4 * U * (log_s + L + Lr)
        e["loss"] += o["r"] * (40 * U * abs(o["ur"]) + es + 8 * U * (1 + abs(o["log_r"]) + log_s))
    return e


@pytest.fixture(autouse=True)
def bounds(monkeypatch):
    monkeypatch.setattr(G, "errors", errors)


TEMPS = [10.0 ** -e for e in (4, 5, 6, 6.5, 7, 7.5, 8, 8.5, 9, 10, 12, 15, 20, 25, 30)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", G.KINDS)
@pytest.mark.parametrize("V,K", [(77, 6), (3001, 12), (6000, 40), (20000, 20), (66001, 64)])
def test_small_temperatures(V, K, kind, dtype):
    c = G.make(len(TEMPS), V, K, dtype, V, kind, temps=TEMPS, pad=1)
    got, _ = G.check_forward(c)
    assert not np.isnan(got["loss"]).any() and not got["status"].any()
    if dtype != "f16":  # whose gradients would be past its range
        G.check_grad(c, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", G.KINDS)
@pytest.mark.parametrize("V", [900, 40000])
def test_large_logits(V, kind, dtype):
    powers = [3, 6, 7, 8, 9, 10, 11, 12, 15, 20, 25, 28, 30]
    c = G.make(len(powers), V, 20, dtype, V, kind, temps=[1.0], masked=True)
    c["x"] *= torch.tensor([10.0 ** e for e in powers], device="cuda").to(c["x"].dtype)[:, None]
    got, _ = G.check_forward(c)
    assert not np.isnan(got["loss"]).any()
    G.check_grad(c, dtype)


@pytest.mark.parametrize("K", [20, 100])
def test_in_rows_that_fill_the_sms(K):
    """With the slots in a warp of their own (K = 20) and without."""
    temps = [1e-7, 1e-8, 1e-9, 1e-12, 1e-20, 1e-30]
    small = G.make(6, 20000, K, "bf16", K, "forward", temps=temps)
    ref = G.reference(small)
    c, order = repeated(small, 460)
    got = {k: v.cpu().numpy() for k, v in G.run(c).items()}
    for r, i in enumerate(order.tolist()):
        e = G.errors(ref[i], 20000, small["temperature"][i].item(), "forward")
        G.close(got["loss"][r], ref[i]["loss"], e["loss"], r)
        G.close(got["stats"][r, 1], ref[i]["stats"][1], e["Lr"], r)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_sums_across_the_border(order, sign):
    """Logits a few apart around 2^24 ln 2, where x / T in units of ln 2 passes 2^24: rising rows
    carry their sums from one kind of reference to the other, and all of them have weight."""
    for V in (3000, 40000, 70000):
        c = G.make(6, V, 20, "f32", V, "reverse", temps=[1.0])
        centre = np.round(sign * 2.0 ** 24 * np.log(2.0))
        for r in range(6):
            # spans that cross it, in steps so small that neighbouring chunks share their weight
            x = centre + np.linspace(-8.0 - 12 * r, 9.0 + 2 * r, V).round()
            x = x if order == "up" else x[::-1] if order == "down" else np.random.default_rng(r).permutation(x)
            c["x"][r] = torch.from_numpy(x.astype(np.float32).copy())
        G.check_forward(c)
        G.check_grad(c, "f32")
