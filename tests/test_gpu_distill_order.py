"""Whether a row's loss is infinite follows from its probabilities alone, whatever the order of its
slots and however they fall into groups: a slot counts if its weight is not 0 in binary64.  Its
gradient is then 0, and finite otherwise.  Bounds and cases are test_gpu_distill's."""
import numpy as np
import pytest
import torch

import test_gpu_distill as G

pytestmark = pytest.mark.gpu

DEPTHS = [3, 50, 86, 89, 95, 101, 110, 200, 400, 700, 800, 5000]  # e^-745.1 is binary64's least number


def row_case(kind, K, dtype, seed):
    """Row r: one slot whose weight lies DEPTHS[r] below the largest, on a token that the other side
    does not have."""
    B, V = len(DEPTHS), 4000
    c = G.make(B, V, K, dtype, seed, kind, temps=[1.0], unused=0.0)
    x, ids = c["x"], c["ids"].long()
    for r, depth in enumerate(DEPTHS):
        j = int(ids[r, 0])
        top = int(ids[r, K // 2])
        x[r, top] = 30.0
        if kind == "reverse":
            x[r, j] = 30.0 - depth
            c["teacher"][r, 0] = -np.inf
        else:
            x[r, j] = -np.inf
            c["teacher"][r, 0] = (c["teacher"][r].max().item() if kind == "truncated" else 0.0) - depth
            if kind == "forward":
                c["teacher"][r, 1:] -= 3.0  # their sum stays below 1
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 32, 33, 64, 256])
@pytest.mark.parametrize("kind", G.KINDS)
def test_infinite_losses_in_any_order(kind, K, dtype):
    c = row_case(kind, K, dtype, K)
    rng = np.random.default_rng(K)
    rows = None
    for n in range(5):
        got, ref = G.check_forward(c)
        G.check_grad(c, dtype)
        infinite = np.isinf(got["loss"])
        assert np.array_equal(infinite, np.array(DEPTHS) < 745), infinite
        assert np.isfinite(got["slot_grads"]).all() and not got["slot_grads"][infinite].any()
        rows = infinite if rows is None else rows
        assert np.array_equal(rows, infinite)
        order = torch.from_numpy(rng.permutation(K) if n else np.roll(np.arange(K), K // 2)).cuda()
        c["ids"], c["teacher"] = c["ids"][:, order].contiguous(), c["teacher"][:, order].contiguous()
