"""The example of sampling, scoring and updating runs, and its updates do what they are for (needs a GB300)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_updates_raise_the_reward():
    from decode_step_token_gb300 import build
    build.build_library()
    spec = importlib.util.spec_from_file_location("rollout_update", os.path.join(ROOT, "examples", "rollout_update.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    rewards = mod.run(rounds=6)
    # half of the tokens are wanted by chance, +- 1/16 a round for 64 tokens
    assert rewards[0] < 0.75 and min(rewards[-2:]) > 0.85, rewards
