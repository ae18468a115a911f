"""The rollout example runs, and its last step agrees with attention over the values read back (bf16 rounding of the
outputs and of the read-back values, 2^-9 each, bounds the difference by 2^-7 of the norm)."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rollout_example():
    spec = importlib.util.spec_from_file_location("rollout_nvfp4_cache", os.path.join(ROOT, "examples", "rollout_nvfp4_cache.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    err, flags = example.main(5)
    assert flags == 0
    assert err <= 2 ** -7
