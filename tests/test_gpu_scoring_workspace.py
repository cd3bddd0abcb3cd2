"""head_logprobs' workspace lives no longer than its call unless the caller owns it."""
import gc

import pytest
import torch

import top_selection_stats_gb300 as lib
import test_gpu_scoring as T

pytestmark = pytest.mark.gpu


def test_kept_results_do_not_keep_workspaces():
    c = T.head_case(300, 5000, 64, "bf16", 1)
    need = lib.head_workspace(300, 5000)
    T.check_head(c)
    torch.cuda.synchronize()
    gc.collect()  # what other tests left is not freed in between
    before = torch.cuda.memory_allocated()
    kept = [lib.head_logprobs(c["h"], c["w"], c["targets"], temperature=c["temperature"]) for _ in range(6)]
    kept += [lib.head_logprobs(c["h"], c["w"], c["targets"], temperature=c["temperature"], out=kept[0])]
    torch.cuda.synchronize()
    results = sum(512 * -(-v.numel() * v.element_size() // 512) for r in kept[:6] for v in r.values())
    assert torch.cuda.memory_allocated() - before == results < need


def test_results_written_again_from_another_stream():
    """A result's buffers may be written by a call on another stream that waits for the first."""
    c = T.head_case(200, 3001, 96, "bf16", 5)
    want = {k: v.clone() for k, v in T.check_head(c).items()}
    out = lib.head_logprobs(c["h"], c["w"], c["targets"], temperature=c["temperature"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for v in out.values():
            v.zero_()
        assert lib.head_logprobs(c["h"], c["w"], c["targets"], temperature=c["temperature"], out=out) is out
    # the first stream's next allocations may take the first call's workspace, not the second's
    junk = [torch.full((lib.head_workspace(200, 3001),), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert len(junk) == 3
    for k in want:
        assert torch.equal(out[k].view(torch.int32), want[k].view(torch.int32)), k
