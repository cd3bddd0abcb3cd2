"""Each launch shape of smp_distill_loss and smp_distill_loss_grad: rows that fill the SMs with
and without a warp for the slots, the rest of them in clusters of every size, CTAs of 2, 4 and 8
warps, segments of 1 to 8 steps, results aligned unlike their logits; and waits that run out.
Bounds and cases are test_gpu_distill's."""
import numpy as np
import pytest
import torch

import test_gpu_distill as G
import top_selection_stats_gb300 as lib

pytestmark = pytest.mark.gpu


def some_rows(c, rows):
    """The rows `rows` of a case, to compare a large batch by."""
    pick = lambda v: v[rows].contiguous() if torch.is_tensor(v) else v  # noqa: E731
    return {k: pick(v) for k, v in c.items()}


def repeated(c, B):
    """A batch of B rows from a small case's, shuffled the same way each time."""
    order = torch.from_numpy(np.random.Generator(np.random.PCG64(B)).integers(0, c["x"].shape[0], B)).cuda()
    return {k: v[order].contiguous() if torch.is_tensor(v) else v for k, v in c.items()}, order


@pytest.mark.parametrize("kind", G.KINDS)
@pytest.mark.parametrize("V,K,B", [(20000, 20, 460), (20000, 100, 460), (40000, 33, 470), (17000, 256, 920), (100000, 64, 600),
                                   (70000, 5, 914)])
def test_rows_that_fill_the_sms(kind, V, K, B):
    """A full round of CTAs (456 on 152 SMs) and a rest of 2 to 144 rows."""
    small = G.make(6, V, K, "bf16", V + K, kind, masked=K == 33, unused=0.1)
    if K > 32:
        small["ids"][5, K - 1] = small["ids"][5, 0] = 7  # the same id twice, in two warps' slots
    far = torch.tensor([-(1 << 31), (1 << 31) - 1, 1 << 30, V, -2], dtype=torch.int32, device="cuda")
    small["ids"][4, :min(K, 5)] = far[:min(K, 5)]
    G.check_forward(small)
    c, order = repeated(small, B)
    got, want = G.run(c), G.run(small)
    ref = G.reference(small)
    assert list(got["status"].cpu()) == [ref[i]["status"] for i in order.tolist()]
    assert ref[4]["status"] == 3 and (K <= 32 or ref[5]["status"] == 3)
    T = small["temperature"].cpu().numpy()
    for r, i in enumerate(order.tolist()):
        if ref[i]["status"] != 0 or r % 37 and r < B - 12:
            continue
        e = G.errors(ref[i], V, T[i], kind)
        G.close(got["loss"][r].item(), ref[i]["loss"], e["loss"], r)
        G.close(got["slot_logprobs"][r].cpu().numpy(), ref[i]["slot_logprobs"], e["slot_logprobs"], r)
        G.close(got["slot_grads"][r].cpu().numpy(), ref[i]["slot_grads"], e["slot_grads"] + 2.0 ** -126, r)
        G.close(got["stats"][r, 2].item(), ref[i]["stats"][2], e["A"] + 2.0 ** -126, r)
    g = torch.rand(6, device="cuda")
    ds = lib.distill_loss_grad(small["x"], small["ids"], want["slot_logprobs"], want["slot_grads"], want["stats"], g,
                               temperature=small["temperature"], bitmask=small["bitmask"])
    f = {k: v[order].contiguous() for k, v in want.items()}
    db = lib.distill_loss_grad(c["x"], c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"], g[order].contiguous(),
                               temperature=c["temperature"], bitmask=c["bitmask"])
    assert torch.equal(db, ds[order])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B", [1, 3, 40, 100, 200])
def test_clusters(B, dtype):
    c = G.make(B, 66001, 40, dtype, B, "reverse", masked=B == 40, pad=3)
    G.check_forward(c)
    G.check_grad(c, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift,pad", [(1, 0), (2, 1), (3, 2), (5, 0), (7, 5)])
def test_results_aligned_unlike_their_logits(dtype, shift, pad):
    """Fresh results of logits that start inside a 16-byte unit, against the aligned ones' bits."""
    for V in (9, 31, 1000, 20003):
        c = G.make(5, V, 6, dtype, V, pad=pad, shift=shift, masked=True)
        f = G.run(c)
        a = (c["ids"], f["slot_logprobs"], f["slot_grads"], f["stats"], torch.rand(5, device="cuda"))
        more = dict(targets=c["targets"], logprobs=f["logprobs"], grad_logprobs=a[4], temperature=c["temperature"],
                    bitmask=c["bitmask"], V=V)
        got = lib.distill_loss_grad(c["x"], *a, **more)
        want = lib.distill_loss_grad(c["x"].clone(), *a, **more)
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), V
        G.check_grad(c, dtype)


def test_row_parameters_written_right_before_the_call():
    """The launches get ready under the work before them, and read nothing of it too early."""
    c = G.make(300, 30000, 20, "bf16", 5)
    want = {k: v.clone() for k, v in G.run(c).items()}
    keep = {k: c[k].clone() for k in ("x", "ids", "teacher", "targets", "temperature")}
    out = {k: torch.empty_like(v) for k, v in want.items()}
    for _ in range(20):
        for k in keep:
            c[k].zero_()
        for k, v in keep.items():
            c[k].copy_(v)
        lib.distill_loss(c["x"], c["ids"], c["teacher"], targets=c["targets"], temperature=c["temperature"], out=out)
        d = lib.distill_loss_grad(c["x"], c["ids"], out["slot_logprobs"], out["slot_grads"], out["stats"],
                                  temperature=c["temperature"], grad_loss=keep["temperature"], out=c["x"])
        assert d.data_ptr() == c["x"].data_ptr()
    for k in want:
        assert torch.equal(want[k].view(torch.int32), out[k].view(torch.int32)), k


@pytest.mark.parametrize("B,V,K,masked", [(3, 128256, 20, False), (40, 50001, 64, True), (600, 20000, 20, False), (600, 20000, 100, False),
                                          (2000, 3000, 8, False), (2000, 6000, 40, True)])
def test_expired_waits(B, V, K, masked):
    """Under bounds from one cycle on a row either has the bits of the normal call or the status;
    the calls after them are whole."""
    c = G.make(7, V, K, "bf16", V, masked=masked)
    c, _ = repeated(c, B)
    want = {k: v.clone() for k, v in G.run(c).items()}
    try:
        for cycles in (1, 300, 3000, 30000):
            lib.set_scoring_wait_limit(cycles)
            got = G.run(c)
            late = got["status"] == lib.SMP_ERR_TIMEOUT
            for k in want:
                same = (got[k].view(B, -1).view(torch.int32) == want[k].view(B, -1).view(torch.int32)).all(1)
                assert bool((same | late).all()), (cycles, k)
            assert torch.isnan(got["loss"][late]).all() and torch.isnan(got["slot_grads"][late]).all()
            if cycles == 1 and B == 600 and K == 20:
                # warps that look as soon as they have asked (elsewhere the slots are looked up
                # first, which may take as long as the copies)
                assert late.any()
    finally:
        lib.set_scoring_wait_limit(0)
    again = G.run(c)
    for k in want:
        assert torch.equal(again[k].view(torch.int32), want[k].view(torch.int32)), k


def test_loss_larger_than_its_terms():
    """Slots in several parts, each far from the others, and a teacher with most of its mass on
    tokens that the student finds unlikely."""
    for kind in G.KINDS:
        c = G.make(6, 5000, 128, "f32", 3, kind, temps=[1.0], unused=0.0)
        for p in range(4):
            rows = torch.arange(6, device="cuda").unsqueeze(1)
            c["x"][rows, c["ids"][:, 32 * p:32 * p + 32].long()] += 30.0 * (p - 2)
        G.check_forward(c)
        G.check_grad(c, "f32")
