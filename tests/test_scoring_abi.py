"""Refusals of the scoring calls that come before any CUDA call (no GPU needed; the
pointers are never followed)."""
import os
import shutil

import pytest
import torch

import top_selection_stats_gb300 as pkg
from top_selection_stats_gb300 import binding

P = 4096  # a 16-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from top_selection_stats_gb300 import build
    build.build()
    return binding.load_library()


def changed(args, i, v):
    a = list(args)
    a[i] = v
    return a


def test_token_logprobs(lib):
    ok = [P, 0, 4, 64, 64, None, None, P, P, P, P, P, P, 2, P, P, None]
    for i, v in ((0, None), (1, 3), (1, -1), (2, -1), (3, 0), (4, 63), (8, None), (12, None), (13, -1),
                 (14, None), (15, None)):
        assert lib.smp_token_logprobs(*changed(ok, i, v)) == pkg.SMP_ERR_INVALID_PARAM, (i, v)
    assert lib.smp_token_logprobs(*changed(ok, 13, 33)) == pkg.SMP_ERR_CAPACITY
    big = changed(changed(ok, 3, (1 << 24) + 1), 4, (1 << 24) + 1)
    assert lib.smp_token_logprobs(*big) == pkg.SMP_ERR_CAPACITY
    assert lib.smp_token_logprobs(*changed(ok, 2, 0)) == pkg.SMP_OK  # no rows: no work


def test_token_logprobs_grad(lib):
    ok = [P, 1, 4, 64, 64, None, None, P, P, P, P, P, P, 64, None]
    for i, v in ((0, None), (1, 7), (2, -1), (3, 0), (4, 60), (7, None), (8, None), (9, None), (12, None),
                 (13, 60), (13, 72)):  # the last: in place with another row length
        a = changed(ok, i, v)
        assert lib.smp_token_logprobs_grad(*a) == pkg.SMP_ERR_INVALID_PARAM, (i, v)
    assert lib.smp_token_logprobs_grad(*changed(ok, 2, 0)) == pkg.SMP_OK


def test_head_logprobs(lib):
    need = lib.smp_head_workspace(4, 100)
    assert need > 0 and lib.smp_head_workspace(0, 100) == 0 and lib.smp_head_workspace(4, 0) == 0
    # the workspace holds 16-byte states: more rows or tokens never need less
    assert lib.smp_head_workspace(4096, 128256) >= lib.smp_head_workspace(4095, 128256)
    ok = [P, 64, P, 64, binding.SMP_BF16, 4, 100, 64, None, P, P, P, P, P, P, need, None]
    for i, v in ((0, None), (0, P + 2), (1, 60), (1, 68), (2, P + 8), (3, 68), (4, binding.SMP_F32), (4, 9),
                 (5, -1), (6, 0), (7, 0), (7, 72), (10, None), (13, None), (14, None), (14, P + 4),
                 (15, need - 1)):
        assert lib.smp_head_logprobs(*changed(ok, i, v)) == pkg.SMP_ERR_INVALID_PARAM, (i, v)
    assert lib.smp_head_logprobs(*changed(ok, 5, 0)) == pkg.SMP_OK
    for i, v in ((5, (1 << 20) + 1), (6, (1 << 24) + 1)):
        assert lib.smp_head_logprobs(*changed(ok, i, v)) == pkg.SMP_ERR_CAPACITY, (i, v)


def test_wrappers_refuse_host_tensors():
    x, t = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkg.token_logprobs(x, t)
    with pytest.raises(ValueError):
        pkg.token_logprobs_grad(x, t, torch.zeros(2, 2))
    with pytest.raises(ValueError):
        pkg.head_logprobs(x.bfloat16(), x.bfloat16(), t)
