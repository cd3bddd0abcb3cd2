"""The example runs all scoring operators beside the sampler: each step makes its
rewarded tokens more likely."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "policy_step.py")


def test_policy_steps_raise_the_rewarded_tokens():
    spec = importlib.util.spec_from_file_location("policy_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    lines = []
    history = m.run(log=lines.append)
    assert len(lines) == len(history) == 4
    for reward, before, after in history:
        assert 0 <= reward <= 1 and after > before
