"""head_logprobs calls whose device waits run out, in each of its launch shapes: the whole call
returns SMP_ERR_TIMEOUT with NaN, or has the bits of a call with the default bound (no wait
of it took longer), and the next call with the default bound is whole again: no copy, no
product and no tensor memory of the failed one is left."""
import numpy as np
import pytest
import torch

import top_selection_stats_gb300 as lib
import test_gpu_scoring as T

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def default_bound_again():
    yield
    lib.set_scoring_wait_limit(0)


@pytest.mark.parametrize("N,V,D", [
    (1, 33000, 4096), (20, 700, 72), (20, 50000, 1000),      # 128 tokens a tile, few states staged
    (100, 33000, 1000), (128, 300, 64),                      # all 128
    (300, 33000, 2048), (130, 700, 72), (513, 20000, 520)])  # pairs
def test_expired_waits(N, V, D):
    c = T.head_case(N, V, D, "bf16", N, temps=False)

    def run():
        out = lib.head_logprobs(c["h"], c["w"], c["targets"])
        torch.cuda.synchronize()
        return {k: v.cpu().numpy() for k, v in out.items()}

    want = run()
    assert not want["status"].any()
    late = {}
    for limit in (1, 200, 1000, 2000, 4000, 8000, 16000):
        for _ in range(3):
            lib.set_scoring_wait_limit(limit)
            got = run()
            status = set(got["status"].tolist())
            assert status in ({lib.SMP_OK}, {lib.SMP_ERR_TIMEOUT}), status
            if status == {lib.SMP_OK}:
                assert all(np.array_equal(got[k].view(np.int32), want[k].view(np.int32)) for k in got)
            else:
                assert all(np.all(np.isnan(got[k])) for k in ("logprobs", "entropy", "stats"))
                late[limit] = late.get(limit, 0) + 1
            lib.set_scoring_wait_limit(0)
            got = run()
            assert all(np.array_equal(got[k].view(np.int32), want[k].view(np.int32)) for k in got)
    print(f"{N} x {V} x {D}: calls of 3 that timed out, by bound: {late}")
    if N * V * D > 10 ** 8:  # a call of 10 us or more: its first products take longer than two looks, 2 us
        assert late[1] == 3
