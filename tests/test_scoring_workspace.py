"""smp_head_workspace for every V that an int can hold (no GPU needed)."""
import os
import shutil

import pytest

from top_selection_stats_gb300 import binding


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from top_selection_stats_gb300 import build
    build.build()
    return binding.load_library()


@pytest.mark.parametrize("N", [1, 128, 129, (1 << 31) - 1])
def test_never_shrinks_as_the_vocabulary_grows(lib, N):
    sizes = [lib.smp_head_workspace(N, V) for V in (1, 1000, 1 << 24, (1 << 31) - 256, (1 << 31) - 200, (1 << 31) - 1)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] > 0, sizes
    # two 16-byte states for each row and each tile of at most 256 tokens
    assert sizes[-1] >= 32 * N * ((1 << 31) // 256)
