"""Refusals of the processing and distillation calls that come before any CUDA call (no GPU
needed; the pointers are never followed)."""
import os
import shutil

import pytest
import torch

import top_selection_stats_gb300 as pkg

P = 4096  # an address that nothing reads


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from top_selection_stats_gb300 import binding, build
    build.build()
    return binding.load_library()


def changed(args, *pairs):
    a = list(args)
    for i, v in pairs:
        a[i] = v
    return a


def test_process_logits(lib):
    # logits dtype B V ld | history H hld | lengths prompts theta pres freq | ids bias NB | mask | out dtype ld status st
    ok = [P, 1, 4, 64, 64, P, 8, 8, P, P, P, P, P, P, P, 3, P, 2 * P, 1, 64, P, None]
    for pairs in (((0, None),), ((1, 3),), ((1, -1),), ((2, -1),), ((3, 0),), ((4, 63),), ((5, None),), ((6, -1),),
                  ((7, 7),), ((13, None),), ((14, None),), ((15, -1),), ((17, None),), ((18, 2),), ((1, 0),), ((19, 63),),
                  ((20, None),), ((17, P), (18, 0)), ((17, P), (19, 72))):
        assert lib.smp_process_logits(*changed(ok, *pairs)) == pkg.SMP_ERR_INVALID_PARAM, pairs
    big = (1 << 24) + 1
    for pairs in (((3, big), (4, big), (19, big)), ((6, big), (7, big)), ((15, 4097),)):
        assert lib.smp_process_logits(*changed(ok, *pairs)) == pkg.SMP_ERR_CAPACITY, pairs
    assert lib.smp_process_logits(*changed(ok, (2, 0))) == pkg.SMP_OK  # no rows: no work


def test_distill_loss(lib):
    # logits dtype B V ld mask T ids teacher K kind targets loss logprobs slot_lp slot_g stats status st
    ok = [P, 0, 4, 64, 64, None, None, P, P, 5, 0, P, P, P, P, P, P, P, None]
    for i, v in ((0, None), (1, 3), (2, -1), (3, 0), (4, 63), (7, None), (8, None), (9, 0), (9, -1), (10, 3), (10, -1),
                 (12, None), (13, None), (17, None)):
        assert lib.smp_distill_loss(*changed(ok, (i, v))) == pkg.SMP_ERR_INVALID_PARAM, (i, v)
    big = (1 << 24) + 1
    for pairs in (((9, 257),), ((3, big), (4, big))):
        assert lib.smp_distill_loss(*changed(ok, *pairs)) == pkg.SMP_ERR_CAPACITY, pairs
    assert lib.smp_distill_loss(*changed(ok, (2, 0))) == pkg.SMP_OK


def test_distill_loss_grad(lib):
    # logits dtype B V ld mask T ids K slot_lp slot_g stats g_loss targets logprobs g_lp grad ld st
    ok = [P, 1, 4, 64, 64, None, None, P, 5, P, P, P, P, P, P, P, P, 64, None]
    for i, v in ((0, None), (1, 9), (2, -1), (3, 0), (4, 60), (7, None), (8, 0), (9, None), (10, None), (11, None),
                 (13, None), (14, None), (16, None), (17, 60), (17, 72)):  # the last: in place with another row length
        assert lib.smp_distill_loss_grad(*changed(ok, (i, v))) == pkg.SMP_ERR_INVALID_PARAM, (i, v)
    assert lib.smp_distill_loss_grad(*changed(ok, (8, 257))) == pkg.SMP_ERR_CAPACITY
    assert lib.smp_distill_loss_grad(*changed(ok, (2, 0))) == pkg.SMP_OK


def test_wrappers_refuse_host_tensors():
    x, ids, q = torch.zeros(2, 8), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    with pytest.raises(ValueError):
        pkg.process_logits(x)
    with pytest.raises(ValueError):
        pkg.distill_loss(x, ids, q)
    with pytest.raises(ValueError):
        pkg.distill_loss_grad(x, ids, q, q, torch.zeros(2, 4))
