"""smp_set_scoring_wait_limit takes any number and needs no GPU."""
import os
import shutil

import pytest

import top_selection_stats_gb300 as pkg
from top_selection_stats_gb300 import binding


def test_setter():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from top_selection_stats_gb300 import build
    build.build()
    L = binding.load_library()
    for cycles in (1, 1 << 40, -5, 0):
        assert L.smp_set_scoring_wait_limit(cycles) == pkg.SMP_OK
    pkg.set_scoring_wait_limit(7)
    pkg.set_scoring_wait_limit()
