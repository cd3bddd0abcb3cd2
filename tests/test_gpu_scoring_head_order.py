"""head_logprobs sees the temperatures and targets that the work right before it on the stream
wrote, in both of its launches."""
import pytest
import torch

import top_selection_stats_gb300 as lib
import test_gpu_scoring as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [20, 120, 400])
def test_row_parameters_written_right_before_the_call(N):
    c = T.head_case(N, 5000, 256, "bf16", N)
    rows = torch.arange(N, device="cuda")
    sets = [(c["temperature"] * (1 + k), (c["targets"] + 7 * k) % 5000) for k in range(4)]
    sets[3][0][::2] = 0.0  # invalid in every other row
    want = []
    for temps, targets in sets:
        out = lib.head_logprobs(c["h"], c["w"], targets, temperature=temps)
        torch.cuda.synchronize()
        want.append(out)
    assert want[3]["status"][::2].eq(lib.SMP_ERR_INVALID_PARAM).all()
    temps, targets = sets[0][0].clone(), sets[0][1].clone()
    got = []
    for turn in range(40):
        temps.copy_(sets[turn % 4][0])
        targets[rows] = sets[turn % 4][1]
        got.append(lib.head_logprobs(c["h"], c["w"], targets, temperature=temps))
        temps.mul_(0.0)
        targets.fill_(-1)
    torch.cuda.synchronize()
    for turn, r in enumerate(got):
        for k in r:
            assert torch.equal(r[k].view(torch.int32), want[turn % 4][k].view(torch.int32)), (turn, k)
