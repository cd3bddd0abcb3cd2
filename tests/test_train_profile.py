"""profiles/processing_distillation_kernels.txt was taken on the kernels as they are: its source
hash is theirs, and its command leaves the clocks alone."""
import os
import re

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = ["top_selection_stats_gb300/csrc/" + f for f in (
    "smp_device.cuh", "smp_score.cuh", "smp_score_kernel.cuh", "smp_train.cuh", "smp_distill.cuh", "smp_distill_kernel.cuh",
    "smp_distill_f32.cu", "smp_distill_bf16.cu", "smp_distill_f16.cu", "smp_distill_grad.cu", "smp_process.cu")]


def test_counters_are_of_the_current_sources():
    with open(os.path.join(ROOT, "profiles", "processing_distillation_kernels.txt")) as f:
        text = f.read()
    assert re.findall(r"sha `([0-9a-f]{16})`", text) == [bench.kernel_source_hash(SOURCES)]
    commands = re.findall(r"^ {4}ncu --.*$", text, flags=re.M)
    assert commands and all("--clock-control none" in c for c in commands)
