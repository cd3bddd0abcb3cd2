"""smp_token_logprobs where its launch changes: more rows than CTAs fit at once (the rows
left over take a second launch), long rows in many pieces, searches that find more
candidates than they hold, and calls with only some of the outputs."""
import numpy as np
import pytest
import torch

import top_selection_stats_gb300 as lib
import test_gpu_scoring as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B", [456, 470, 700])
def test_rows_past_one_load(B, dtype):
    V = 9001 if dtype == "f32" else 18003
    T.check_forward(T.make(B, V, dtype, B, pad=5, masked=B == 470), 7)


def test_rows_past_one_load_in_a_graph():
    c = T.make(500, 20000, "bf16", 3)
    want = {k: v.clone() for k, v in T.run(c, 4).items()}
    out = {k: torch.zeros_like(v) for k, v in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            lib.token_logprobs(c["x"], c["targets"], temperature=c["temperature"], n_top=4, out=out)
            # what follows on the stream sees every row
            copy = {k: v.clone() for k, v in out.items()}
    for _ in range(2):
        for v in out.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k].view(torch.int32), want[k].view(torch.int32)), k
            assert torch.equal(copy[k].view(torch.int32), want[k].view(torch.int32)), k


@pytest.mark.parametrize("B", [3, 500])
@pytest.mark.parametrize("order", ["equal", "falling", "rising", "block"])
def test_searches_that_overflow(B, order):
    """Every token a candidate: all equal, sorted by id, the best ones side by side."""
    V = 20011
    c = T.make(B, V, "f32", 5, temps=[1.0])
    j = torch.arange(V, device="cuda", dtype=torch.float32)
    c["x"][:] = {"equal": 0 * j, "falling": -j * 1e-3, "rising": j * 1e-3,
                 "block": torch.where((j > 7000) & (j < 9000), 5 + j * 1e-4, -j * 1e-4)}[order]
    T.check_forward(c, 32)


def test_a_very_long_row():
    T.check_forward(T.make(2, 3000001, "f32", 9, pad=2, temps=[1.0]), 9)
    T.check_forward(T.make(2, 2500003, "bf16", 10, temps=[1.0]), 32)


def test_some_outputs():
    c = T.make(20, 30000, "bf16", 6)
    full = T.run(c)
    L = lib.load_library()
    B, V = 20, 30000
    x, t, temp = c["x"].data_ptr(), c["targets"].data_ptr(), c["temperature"].data_ptr()
    lp, st = torch.zeros(B, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    ent = torch.zeros(B, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    # the log probability alone; then the entropy alone, without targets
    assert L.smp_token_logprobs(x, 1, B, V, V, None, temp, t, lp.data_ptr(), None, None, None, st.data_ptr(), 0,
                                None, None, stream) == 0
    assert L.smp_token_logprobs(x, 1, B, V, V, None, temp, None, None, ent.data_ptr(), None, None, st.data_ptr(), 0,
                                None, None, stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(lp, full["logprobs"]) and torch.equal(ent, full["entropy"]) and not st.any()


def test_head_with_some_outputs():
    c = T.head_case(130, 700, 64, "f16", 4)
    full = T.check_head(c)
    L = lib.load_library()
    ws = torch.empty(lib.head_workspace(130, 700), dtype=torch.uint8, device="cuda")
    st = torch.zeros(130, dtype=torch.int32, device="cuda")
    ent = torch.zeros(130, device="cuda")
    assert L.smp_head_logprobs(c["h"].data_ptr(), 64, c["w"].data_ptr(), 64, 2, 130, 700, 64,
                               c["temperature"].data_ptr(), None, None, ent.data_ptr(), None, st.data_ptr(),
                               ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(ent, full["entropy"]) and not st.any()


@pytest.mark.parametrize("N,V,D", [(257, 1000, 2048), (1300, 300, 64), (513, 40000, 72)])
def test_head_more_tiles(N, V, D):
    T.check_head(T.head_case(N, V, D, "bf16", N))


def test_grad_skips_rows_without_gradient():
    """A padded row's gradient is zero whatever its logits hold."""
    c = T.make(6, 5000, "bf16", 7)
    c["targets"][2] = -1
    f = T.run(c)
    c["x"][2] = float("nan")
    g = torch.ones(6, device="cuda")
    d = lib.token_logprobs_grad(c["x"], c["targets"], f["stats"], grad_logprobs=g, temperature=c["temperature"])
    torch.cuda.synchronize()
    assert not d[2].any() and torch.isfinite(d.float()).all() and d[0].any()
    assert np.isclose(d.float().sum(1).cpu().numpy(), 0.0, atol=0.05).all()  # sum of the gradient is 0


@pytest.mark.parametrize("N", [1, 21, 100, 130])
def test_head_does_not_depend_on_what_ran_before(N):
    """Rows of a tile that no state has hold what earlier work left on the SM."""
    c = T.head_case(N, 24514, 2764, "bf16", N, pad=4)
    first = {k: v.clone() for k, v in T.check_head(c).items()}
    other = T.head_case(256, 24514, 2764, "bf16", 9, pad=4)
    for value in (float("nan"), float("inf"), 3e38, 0.0):
        other["h"][:] = value
        lib.head_logprobs(other["h"], other["w"], other["targets"], D=2764)
        lib.head_logprobs(other["h"][:128].contiguous(), other["w"], other["targets"][:128].contiguous(), D=2764)
        out = lib.head_logprobs(c["h"], c["w"], c["targets"], temperature=c["temperature"], D=c["D"])
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(out[k].view(torch.int32), first[k].view(torch.int32)), (k, value)


@pytest.mark.parametrize("B,V", [(1, 128256), (64, 32000), (300, 5003), (300, 300), (600, 20000)])
def test_calls_follow_the_work_before_them(B, V):
    """Launches may start under the end of earlier work; what it writes is what they read.
    Each turn overwrites the logits, scores them, replaces them by their gradient and
    scores that, with nothing in between that waits."""
    g = torch.ones(B, device="cuda")
    sets = [T.make(B, V, "bf16", k, temps=[1.0]) for k in range(3)]
    want = []
    for c in sets:
        f = T.run(c, 5)
        x = c["x"].clone()
        lib.token_logprobs_grad(x, c["targets"], f["stats"], grad_logprobs=g, out=x)
        torch.cuda.synchronize()
        f2 = T.run(dict(c, x=x), 5)
        want.append({k: v.clone() for k, v in f.items()} | {"2" + k: v.clone() for k, v in f2.items()})
    x = torch.empty_like(sets[0]["x"])
    got = []
    for turn in range(30):
        c = sets[turn % 3]
        x.copy_(c["x"])
        f = lib.token_logprobs(x, c["targets"], n_top=5)
        lib.token_logprobs_grad(x, c["targets"], f["stats"], grad_logprobs=g, out=x)
        f2 = lib.token_logprobs(x, c["targets"], n_top=5)
        x.fill_(7.0)
        got.append(f | {"2" + k: v for k, v in f2.items()})
    torch.cuda.synchronize()
    for turn, r in enumerate(got):
        for k, v in want[turn % 3].items():
            assert torch.equal(r[k].view(torch.int32), v.view(torch.int32)), (turn, k)


def test_head_follows_the_work_before_it():
    c = [T.head_case(20, 5000, 512, "bf16", k) for k in range(3)]
    want = [{k: v.clone() for k, v in T.check_head(x).items()} for x in c]
    h, w = torch.empty_like(c[0]["h"]), torch.empty_like(c[0]["w"])
    got = []
    for turn in range(30):
        x = c[turn % 3]
        h.copy_(x["h"])
        w.copy_(x["w"])
        got.append(lib.head_logprobs(h, w, x["targets"], temperature=x["temperature"]))
        w.zero_()
    torch.cuda.synchronize()
    for turn, r in enumerate(got):
        for k, v in want[turn % 3].items():
            assert torch.equal(r[k].view(torch.int32), v.view(torch.int32)), (turn, k)
