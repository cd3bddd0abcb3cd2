"""Scoring calls whose device waits run out (smp_set_scoring_wait_limit with a bound far
below a copy's latency): every row either has the bits of a call with the default bound
or returns SMP_ERR_TIMEOUT with NaN, rank -1 and ids -1, and the next call with the
default bound is whole again.  No wait is made to hang: each gives up after its bound, what
is in flight is waited for, and the kernel reports the status."""
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


def host(out):
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}


def check_rows(got, want):
    late = got["status"] == lib.SMP_ERR_TIMEOUT
    for k in got:
        a, b = got[k], want[k]
        assert np.array_equal(a[~late].view(np.int32), b[~late].view(np.int32)), k
        if k in ("rank", "top_ids"):
            assert np.all(a[late] == -1), k
        elif k != "status":
            assert np.all(np.isnan(a[late])), k
    return int(late.sum())


def big(B, V, dtype, seed, masked):
    """Logits past L2 in size, without the oracle's work; masks leave one token in twenty or all."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn((B, V), generator=g, device="cuda") * 2).to(T.DT[dtype])
    t = torch.randint(0, V, (B,), generator=g, device="cuda").to(torch.int32)
    bits = None
    if masked:
        bits = torch.full((B, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
        bits[::2] = torch.randint(-2**31, 2**31, bits[::2].shape, generator=g, device="cuda").to(torch.int32)
        bits[::3] = 1 << 7
    return dict(x=x, V=V, targets=t, temperature=None, bitmask=bits)


@pytest.mark.parametrize("dtype,B,V,n,masked", [
    ("bf16", 1000, 128256, 0, False), ("bf16", 1000, 128256, 20, False), ("f32", 700, 128256, 5, False),
    ("f16", 1000, 151936, 8, True), ("f16", 700, 151936, 0, True), ("bf16", 1412, 40000, 5, False),
    ("f32", 1412, 20000, 0, True), ("bf16", 100, 128256, 20, False),
    ("bf16", 20, 262143, 32, True), ("bf16", 3, 2500003, 32, False)])
def test_expired_waits(dtype, B, V, n, masked):
    c = big(B, V, dtype, V + n, masked)
    want = host(T.run(c, n))
    assert not (want["status"] == lib.SMP_ERR_TIMEOUT).any()
    expired = []
    other = torch.empty(1 << 28, device="cuda")
    for limit in (1, 1000, 4000, 10000):
        lib.set_scoring_wait_limit(limit)
        other.fill_(limit)  # the logits are not in L2
        expired.append(check_rows(host(T.run(c, n)), want))
    print(f"{dtype} {B} x {V}, {n}: {expired} of {B} rows timed out")
    if B >= 100:  # of a few rows on an idle device, every copy may be there when it is looked for
        assert expired[0] > 0
    lib.set_scoring_wait_limit(0)
    for _ in range(2):
        assert check_rows(host(T.run(c, n)), want) == 0
