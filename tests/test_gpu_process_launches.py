"""Each way that smp_process_logits cuts a call: tables and counts by cell, one to many segments,
rows that start and end inside a vector, results aligned unlike their logits, and in place.
Bounds and cases are test_gpu_process's."""
import pytest
import torch

import test_gpu_process as G
import top_selection_stats_gb300 as lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("H,NB", [(1000, 48), (2000, 48), (2000, 49), (2049, 0), (0, 2048), (0, 2049), (5000, 2500)])
def test_on_both_sides_of_the_table_s_size(H, NB, in_place):
    for V, masked in ((20011, False), (40005, True)):
        G.check(G.make(3, V, H, NB, "bf16", H + NB, pad=3, masked=masked), "bf16", in_place=in_place)


@pytest.mark.parametrize("dtype,out", [("f32", "same"), ("bf16", "same"), ("f16", "f32")])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 0), (3, 1), (4, 4), (7, 5)])
def test_ends_and_alignments(dtype, out, shift, pad):
    """Tokens in a row's first and last values, seen, biased and masked, at every alignment, for
    results that start alike and unlike."""
    for V, H in ((5, 8), (15, 20), (16, 20), (17, 20), (8191, 40), (8193, 40), (33001, 3000)):
        c = G.make(4, V, H, 6, dtype, V, pad=pad, shift=shift, masked=True)
        ends = torch.tensor([0, 1, 2, 3, V - 1, V - 2, V - 3, V // 2]).clamp(0, V - 1).int()
        c["history"][:, :8] = ends.cuda()
        c["lengths"][:] = H
        c["bias_ids"][:, 0], c["bias_ids"][:, 1] = 0, V - 1
        G.check(c, dtype, out)
        if out == "same":
            G.check(c, dtype, in_place=True)


@pytest.mark.parametrize("B,V,H", [(1, 260001, 10), (1, 1000003, 3000), (2, 140001, 0), (900, 9000, 200), (160, 40000, 4000)])
def test_one_to_many_segments(B, V, H):
    c = G.make(B, V, H, 9, "bf16", V, masked=B == 2)
    G.check(c, "bf16")
    G.check(c, "bf16", in_place=True)


def test_crowded_tables():
    """All entries different, and all tokens of a short row in the history."""
    for V, H in ((2048, 2048), (300, 2000), (1500, 2000)):
        c = G.make(3, V, H, 0, "f32", V)
        c["history"][:, :min(V, H)] = torch.randperm(V, device="cuda")[:min(V, H)].int()
        c["lengths"][:] = H
        G.check(c, "f32")
        G.check(c, "f32", in_place=True)


def test_the_same_bias_many_times():
    c = G.make(3, 5000, 0, 400, "f32", 5)
    c["bias_ids"][0] = 17
    c["bias_ids"][1, ::2] = 4999
    c["bias"][:] = torch.where(torch.isinf(c["bias"]), torch.ones_like(c["bias"]), c["bias"])
    G.check(c, "f32")
    G.check(c, "f32", in_place=True)


def test_row_parameters_written_right_before_the_call():
    for H, masked, in_place in ((300, True, False), (5000, False, False), (300, False, True)):
        c = G.make(200, 30000, H, 20, "bf16", 5, masked=masked)
        keep = {k: v.clone() for k, v in c.items() if torch.is_tensor(v)}
        want = G.call(dict(c, x=c["x"].clone()), in_place=in_place)["logits"].clone()
        for _ in range(10):
            for k, v in keep.items():
                c[k].zero_()
                c[k].copy_(v)
            got = G.call(c, in_place=in_place)["logits"]
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), (H, in_place)


def test_two_captured_calls_and_two_streams():
    """Calls keep nothing between them: two at once, and two graphs replayed in turn."""
    a, b = G.make(50, 40000, 500, 10, "bf16", 1), G.make(60, 30000, 4000, 0, "f16", 2, masked=True)
    want = [G.call(c)["logits"].clone() for c in (a, b)]
    outs, graphs = [G.call(c) for c in (a, b)], []
    for c, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            G.call(c, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s, o in zip(graphs, streams, outs):
            with torch.cuda.stream(s):
                o["logits"].zero_()
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o["logits"], w)


def test_in_place_leaves_the_rest_alone():
    """Only what changes is written: values of other types of NaN keep their bits."""
    x = torch.full((3, 9000), float("nan"), dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16)[:] = torch.arange(9000, device="cuda").to(torch.int16) | 0x7f80
    raw = x.clone()
    h = torch.tensor([[5], [8999], [-1]], dtype=torch.int32, device="cuda")
    lib.process_logits(x, history=h, repetition=torch.full((3,), 2.0, device="cuda"), in_place=True)
    same = x.view(torch.int16) == raw.view(torch.int16)
    assert bool(same[2].all()) and int((~same).sum()) <= 2
    y = lib.process_logits(raw, history=h, repetition=torch.full((3,), 2.0, device="cuda"))["logits"]
    assert bool((y.view(torch.int16) == raw.view(torch.int16))[2].all())
