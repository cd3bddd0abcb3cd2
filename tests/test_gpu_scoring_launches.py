"""smp_token_logprobs in each of its launch shapes: rows of medium length in CTAs of 128
threads, once 2 x 3 x (number of SMs) of them share a call, chains of up to three
launches for one call, and masked rows in the ring without alternatives."""
import pytest
import torch

import top_selection_stats_gb300 as lib
import test_gpu_scoring as T

pytestmark = pytest.mark.gpu


def rows(loads, slots, more):
    """Rows that fill `loads` times all places for CTAs of 128 threads and `slots` times
    those for CTAs of 256, and `more`."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return (2 * loads + slots) * 3 * sms + more


@pytest.mark.parametrize("dtype,V,loads,slots,more,n,masked", [
    ("bf16", 9001, 1, 0, 0, 0, False), ("bf16", 9001, 1, 0, 1, 5, True), ("f16", 9001, 1, 0, 0, 32, True),
    ("f16", 20000, 1, 1, 0, 0, True), ("bf16", 20000, 1, 1, 44, 5, False), ("f16", 20011, 1, 1, 44, 32, True),
    ("bf16", 40000, 1, 0, 40, 5, True), ("f32", 4501, 1, 0, 0, 5, True), ("f32", 4501, 1, 0, 1, 0, False),
    ("f32", 9999, 1, 1, 44, 7, True), ("f32", 9999, 1, 1, 0, 0, True), ("f16", 9001, 1, 0, 30, 0, False)])
def test_rows_of_medium_length(dtype, V, loads, slots, more, n, masked):
    T.check_forward(T.make(rows(loads, slots, more), V, dtype, V + n, pad=3, shift=1, masked=masked,
                           neg_inf=0.02 if masked else 0.0), n)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,V", [(3, 70001), (40, 200003), (460, 70001)])
def test_masked_rows_in_the_ring_without_alternatives(B, V, dtype):
    T.check_forward(T.make(B, V, dtype, B, pad=1, masked=True, neg_inf=0.02), 0)


@pytest.mark.parametrize("n", [0, 6])
def test_three_launches_follow_and_are_followed(n):
    """Calls of three launches between writes of their logits and copies of their results,
    one after another and in a graph."""
    B, V = rows(1, 1, 44), 20000
    sets = [T.make(B, V, "bf16", 20 + k) for k in range(2)]
    want = [{k: v.clone() for k, v in T.run(c, n).items()} for c in sets]
    x = torch.empty_like(sets[0]["x"])
    out = {k: torch.zeros_like(v) for k, v in want[0].items()}

    def turn(c):
        x.copy_(c["x"])
        lib.token_logprobs(x, c["targets"], temperature=c["temperature"], n_top=n, out=out)
        copy = {k: v.clone() for k, v in out.items()}
        x.fill_(7.0)
        return copy

    got = [turn(sets[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        for k in r:
            assert torch.equal(r[k].view(torch.int32), want[i % 2][k].view(torch.int32)), (i, k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [turn(c) for c in sets]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for r, w in zip(got, want):
        for k in r:
            assert torch.equal(r[k].view(torch.int32), w[k].view(torch.int32)), k
