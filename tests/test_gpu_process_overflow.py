"""Penalties that are finite, as the call asks, but whose product with a count is past binary32: no
NaN and no infinity comes of it unless the result itself is past the range.  Bounds and cases are
test_gpu_process's."""
import numpy as np
import pytest
import torch

import test_gpu_process as G

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("H", [40, 3000])
def test_products_past_binary32(H, in_place):
    V = 500
    rows = [(3e38, 0.0), (-3e38, 0.0), (3e38, -3e38), (-3e38, 3e38), (2e38, 2e38), (-2e38, -3e38), (1e37, 3e38), (0.25, 0.5)]
    c = G.make(len(rows), V, H, 0, "f32", 7)
    c["repetition"][:] = 1.0
    for r, (f, p) in enumerate(rows):
        c["frequency"][r], c["presence"][r] = f, p
        c["x"][r, :V:5] = torch.tensor([3e38, -3e38, INF, -INF, 1.0], device="cuda").repeat(20)
        c["history"][r, :10] = torch.arange(0, 50, 5).int()
        c["history"][r, 10:20] = torch.arange(0, 50, 5).int()  # twice, then some more at random
        c["history"][r, 20:] = c["history"][r, 20:] % 7 * 5
        c["lengths"][r] = 40
        c["prompt_lengths"][r] = 0
    raw = c["x"].clone()
    G.check(c, "f32", in_place=in_place)
    if not in_place:
        got = G.call(c)["logits"]
        assert not torch.isnan(got).any()
        assert (got[raw == INF] == INF).all() and (got[raw == -INF] == -INF).all()
        assert np.isfinite(got[0, 0].item()) or got[0, 0] == -INF
